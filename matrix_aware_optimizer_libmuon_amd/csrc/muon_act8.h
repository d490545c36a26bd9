// Device helpers of the operators on 8-bit activations (gfx950).
//
// Work is dealt in vectors of 8 consecutive columns per lane; 4 lanes of a
// quad hold one group of 32, whose maximum they share by two quad
// permutations.  The vector accesses carry the alignment of one element:
// gfx950 global accesses may start at any byte, so rows of every stride take
// the same path.  A row's last, shorter vector is loaded with the elements before
// it, 8 up to the row's end, and shifted down in registers, so that it costs no
// further trip to memory; it is stored in pieces of 4, 2 and 1.
#pragma once
#include "muon_device.h"
#include "muon.h"

namespace muon {

typedef uint32_t u32x4_a2 __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x4_a4 __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u32x2_a1 __attribute__((ext_vector_type(2), aligned(1)));
typedef uint32_t u32x2_a2 __attribute__((ext_vector_type(2), aligned(2)));
typedef uint32_t u32x2_a4 __attribute__((ext_vector_type(2), aligned(4)));
typedef uint32_t u32_a1 __attribute__((aligned(1)));
typedef uint32_t u32_a2 __attribute__((aligned(2)));
typedef uint16_t u16_a1 __attribute__((aligned(1)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));

// Element types: raw 8-vectors as loaded, and their values.
template <class T>
struct Vec8;

template <>
struct Vec8<uint16_t> {            // bf16
  u32x4 r;
  __device__ __forceinline__ void zero() { r = u32x4{0, 0, 0, 0}; }
  __device__ __forceinline__ void load(const uint16_t* p) { r = gld<u32x4_a2>(p); }
  __device__ __forceinline__ void load(const uint16_t* p, int n) {
    uint32_t h[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = i < n ? gld<uint16_t>(p + i) : 0u;
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = h[2 * i] | (h[2 * i + 1] << 16);
  }
  // elements k .. 7 to the front, zeros behind them (0 < k < 8)
  __device__ __forceinline__ void drop(int k) {
    if (k & 4) r = u32x4{r[2], r[3], 0, 0};
    if (k & 2) r = u32x4{r[1], r[2], r[3], 0};
    if (k & 1)
      r = u32x4{(r[0] >> 16) | (r[1] << 16), (r[1] >> 16) | (r[2] << 16), (r[2] >> 16) | (r[3] << 16), r[3] >> 16};
  }
  __device__ __forceinline__ float get(int i) const {
    return __uint_as_float(i & 1 ? r[i >> 1] & 0xffff0000u : r[i >> 1] << 16);
  }
  static __device__ __forceinline__ void store(uint16_t* p, int n, const float (&v)[8]) {
    u32x4 o;
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = pack2(v[2 * i], v[2 * i + 1]);
    if (n >= 8) {
      gst<u32x4_a2>(p, o);
    } else if (n > 0) {
      if (n & 4) {
        gst<u32x2_a2>(p, u32x2_a2{o[0], o[1]});
        o[0] = o[2];
        o[1] = o[3];
        p += 4;
      }
      if (n & 2) {
        gst<u32_a2>(p, o[0]);
        o[0] = o[1];
        p += 2;
      }
      if (n & 1) gst<uint16_t>(p, static_cast<uint16_t>(o[0]));
    }
  }
};

template <>
struct Vec8<float> {
  u32x4 r[2];
  __device__ __forceinline__ void zero() { r[0] = r[1] = u32x4{0, 0, 0, 0}; }
  __device__ __forceinline__ void load(const float* p) {
    r[0] = gld<u32x4_a4>(p);
    r[1] = gld<u32x4_a4>(p + 4);
  }
  __device__ __forceinline__ void load(const float* p, int n) {
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i >> 2][i & 3] = i < n ? gld<uint32_t>(p + i) : 0u;
  }
  __device__ __forceinline__ void drop(int k) {
    if (k & 4) {
      r[0] = r[1];
      r[1] = u32x4{0, 0, 0, 0};
    }
    if (k & 2) {
      r[0] = u32x4{r[0][2], r[0][3], r[1][0], r[1][1]};
      r[1] = u32x4{r[1][2], r[1][3], 0, 0};
    }
    if (k & 1) {
      r[0] = u32x4{r[0][1], r[0][2], r[0][3], r[1][0]};
      r[1] = u32x4{r[1][1], r[1][2], r[1][3], 0};
    }
  }
  __device__ __forceinline__ float get(int i) const { return __uint_as_float(r[i >> 2][i & 3]); }
  static __device__ __forceinline__ void store(float* p, int n, const float (&v)[8]) {
    if (n >= 8) {
      gst<u32x4_a4>(p, u32x4{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])});
      gst<u32x4_a4>(p + 4, u32x4{__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7])});
    } else if (n > 0) {
      u32x4 o = u32x4{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])};
      if (n & 4) {
        gst<u32x4_a4>(p, o);
        o = u32x4{__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), 0};
        p += 4;
      }
      if (n & 2) {
        gst<u32x2_a4>(p, u32x2_a4{o[0], o[1]});
        o[0] = o[2];
        p += 2;
      }
      if (n & 1) gst<uint32_t>(p, o[0]);
    }
  }
};

// The 8 columns at p, columns c .. of a row, n of them inside (<= 0: none, zeros):
// fetch8 issues the load, settle8 puts a shorter vector in its place.  Several
// vectors are fetched before the first is settled.
template <class T>
__device__ __forceinline__ void fetch8(Vec8<T>& v, const T* p, int c, int n) {
  const int back = n < 8 ? 8 - n : 0;
  if (n <= 0) v.zero();
  else if (back <= c) v.load(p - back);
  else v.load(p, n);                 // a row of fewer than 8
}
template <class T>
__device__ __forceinline__ void settle8(Vec8<T>& v, int c, int n) {
  if (n > 0 && n < 8 && 8 - n <= c) v.drop(8 - n);
}
template <class T>
__device__ __forceinline__ void load8(Vec8<T>& v, const T* p, int c, int n) {
  fetch8(v, p, c, n);
  settle8(v, c, n);
}

template <int CTRL>
__device__ __forceinline__ uint32_t quad_perm(uint32_t x) {
  return static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(x), CTRL, 0xf, 0xf, true));
}

// Maximum over the 4 lanes of a quad (all of them active).
__device__ __forceinline__ uint32_t quad_max(uint32_t x) {
  uint32_t y = quad_perm<0xB1>(x);   // lanes 1 0 3 2
  x = x > y ? x : y;
  y = quad_perm<0x4E>(x);            // lanes 2 3 0 1
  return x > y ? x : y;
}

// ---------------------------------------------------------------------------
// 8-bit groups.  The scale's biased exponent is taken from the bits of the
// largest finite magnitude: 448 = 1.75 * 2^8, so e = exponent - 8, and one more
// where the mantissa is above 1.75 (adding 2^21 - 1 carries exactly then).
// Clamped to 10 .. 246: the smallest code, 2^-9, stays a normal fp32 and bf16
// number, and 448 * 2^119 the largest finite one of its binade.
// ---------------------------------------------------------------------------
__device__ __forceinline__ int act8_scale_byte(uint32_t amax_bits) {
  const int e = static_cast<int>((amax_bits + 0x1fffffu) >> 23) - 8;
  return e < 10 ? 10 : e > 246 ? 246 : e;
}
__device__ __forceinline__ float act8_scale(uint32_t byte) { return __uint_as_float(byte << 23); }
__device__ __forceinline__ float act8_inv_scale(int byte) {
  return __uint_as_float(static_cast<uint32_t>(254 - byte) << 23);
}

// One lane's 8 values (zeros where the row has ended): the group's scale byte
// and the lane's codes.  All 4 lanes of the quad take part.
__device__ __forceinline__ u32x2 act8_encode(const float (&v)[8], int& scale_byte) {
  uint32_t amax = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t a = __float_as_uint(v[i]) & 0x7fffffffu;
    const uint32_t f = a < 0x7f800000u ? a : 0u;
    amax = amax > f ? amax : f;
  }
  scale_byte = act8_scale_byte(quad_max(amax));
  const float inv = act8_inv_scale(scale_byte);
  float q[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    // the product is exact but for underflow far below the smallest code;
    // the clamp acts only where the exponent was clamped from above
    const bool finite = (__float_as_uint(v[i]) & 0x7fffffffu) < 0x7f800000u;
    q[i] = finite ? __builtin_amdgcn_fmed3f(v[i] * inv, -448.f, 448.f) : __uint_as_float(0x7fc00000u);
  }
  u32x2 c;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(q[4 * i], q[4 * i + 1], 0, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(q[4 * i + 2], q[4 * i + 3], w, true);
    c[i] = static_cast<uint32_t>(w);
  }
  return c;
}

__device__ __forceinline__ void act8_decode(u32x2 c, uint32_t scale_byte, float (&v)[8]) {
  const float s = act8_scale(scale_byte);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const f32x2_t lo = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(c[i]), false);
    const f32x2_t hi = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(c[i]), true);
    v[4 * i] = lo[0] * s;
    v[4 * i + 1] = lo[1] * s;
    v[4 * i + 2] = hi[0] * s;
    v[4 * i + 3] = hi[1] * s;
  }
}

// A lane's codes and their scale byte, columns c .. of row r, n of them inside:
// fetched and settled as above.
struct Codes8 {
  u32x2 c;
  uint32_t sb;
  __device__ __forceinline__ void fetch(const muon_act8_t& a, int64_t r, int col, int n) {
    const uint8_t* p = a.codes + r * a.ld_codes + col;
    const int back = n < 8 ? 8 - n : 0;
    c = u32x2{0, 0};
    sb = 127;
    if (n <= 0) return;
    sb = gld<uint8_t>(a.scales + r * a.ld_scales + (col >> 5));
    if (back <= col) {
      c = gld<u32x2_a1>(p - back);
    } else {                         // a row of fewer than 8
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < n) c[i >> 2] |= static_cast<uint32_t>(gld<uint8_t>(p + i)) << (8 * (i & 3));
    }
  }
  __device__ __forceinline__ void settle(int col, int n) {
    if (n > 0 && n < 8 && 8 - n <= col) {
      const uint64_t w = (static_cast<uint64_t>(c[1]) << 32 | c[0]) >> (8 * (8 - n));
      c = u32x2{static_cast<uint32_t>(w), static_cast<uint32_t>(w >> 32)};
    }
  }
  __device__ __forceinline__ void get(float (&v)[8]) const { act8_decode(c, sb, v); }
};

__device__ __forceinline__ void store_codes(uint8_t* p, int n, u32x2 c) {
  if (n >= 8) {
    gst<u32x2_a1>(p, c);
  } else if (n > 0) {
    uint32_t o = c[0];
    if (n & 4) {
      gst<u32_a1>(p, o);
      o = c[1];
      p += 4;
    }
    if (n & 2) {
      gst<u16_a1>(p, static_cast<uint16_t>(o));
      o >>= 16;
      p += 2;
    }
    if (n & 1) gst<uint8_t>(p, static_cast<uint8_t>(o));
  }
}

// A lane's 8 columns from c0 of row r, written to an 8-bit matrix.
__device__ __forceinline__ void act8_put(const muon_act8_t& a, int64_t r, int c0, int n, const float (&v)[8]) {
  int sb;
  const u32x2 c = act8_encode(v, sb);
  store_codes(a.codes + r * a.ld_codes + c0, n, c);
  if (n > 0 && (c0 & 31) == 0) gst<uint8_t>(a.scales + r * a.ld_scales + (c0 >> 5), static_cast<uint8_t>(sb));
}

}  // namespace muon
