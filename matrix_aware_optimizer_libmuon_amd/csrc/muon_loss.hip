// Losses over a row of logits with the gradient of the logits (gfx950):
// distillation from a teacher's top logits, and the clipped policy loss.
//
// Both need, of a token's row x = z / temperature, the softmax's maximum and sum
// and a few single entries, and their gradient is
//   dz = a softmax(x)  plus a value at each of those few entries.
// A block takes a row, or, of few long ones, its share of a row's gradient.  Up to 131072
// columns in bf16 and 65536 in fp32 the row stays in registers, so the logits are read once
// and the gradient written once; a longer row is read again for the gradient (from the
// caches, which hold the rows in work).  Bound by memory: distillation 16384 x 32000 bf16
// 409 us (4.9 TB/s), policy loss with 30 % of the rows masked 331 us (5.4); a large copy
// runs at 4.7 to 4.8.  A single row is bound by one CU's
// exponentials, a quarter of the rate of other instructions, 32000 of them twice in 9 us.
//
// Numbers.  x - max is taken before the factor log2(e) / temperature, so that rows
// of the type's lowest value stay finite, and a single log2 of a probability is
// halved, so that it does for a column of that value.  Sums run in fp32, in trees: a term
// goes through 19 roundings at most in a thread whose row is in registers, through 80 where
// it is read twice, then through the wave's and the waves' in a fixed order.  The gradient
// is rounded once, to the logits' type.
#include <type_traits>

#include "muon_act8.h"
#include "muon_ops.h"

namespace muon {

namespace {

constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;
constexpr float kNegInf = -__builtin_inff();

__device__ __forceinline__ float exp2_fast(float v) { return __builtin_amdgcn_exp2f(v); }   // 1 ulp
__device__ __forceinline__ float log2_fast(float v) { return __builtin_amdgcn_logf(v); }

__device__ __forceinline__ float wave_max(float v) {
  return wave_all(v, [](float x, float y) { return fmaxf(x, y); });
}
__device__ __forceinline__ float wave_add(float v) {
  return wave_all(v, [](float x, float y) { return x + y; });
}

// A maximum to subtract: 0 where there is nothing but -inf, so that exp gives 0.
__device__ __forceinline__ float base_of(float m) { return m == kNegInf ? 0.f : m; }
// What a sum taken against the maximum `from` is multiplied by for a larger one (a sum
// of nothing but -inf is 0 and stays it).
__device__ __forceinline__ float shrink(float from, float to, float k) {
  return from == kNegInf ? 0.f : exp2_fast((from - to) * k);
}

// Half of log2 of v's probability, (v - base) k - log2(sum): v may be the type's lowest value,
// which log2(e) takes past the largest number, and the half is as exact.
__device__ __forceinline__ float half_log2(float v, float base, float k, float log2_sum) {
  return (v - base) * 0.5f * k - 0.5f * log2_sum;
}

// Maximum and sum of 2^((v - m) k) over some values.
struct Soft {
  float m, s;
};

// Sum of two: the smaller one's is brought to the larger maximum.
__device__ __forceinline__ Soft wave_join(Soft a, float k) {
  const float m = wave_max(a.m);
  return {m, wave_add(a.s * shrink(a.m, m, k))};
}

template <int RT>
struct Shared {
  static constexpr int W = RT / 64;
  float m[2][W], s[2][W], part[W];
};

// Over the block's waves, from what each has left in shared memory.
template <int RT>
__device__ __forceinline__ Soft block_join(const Shared<RT>& sh, int which, float k) {
  float m = kNegInf, s = 0.f;
#pragma unroll
  for (int w = 0; w < RT / 64; ++w) m = fmaxf(m, sh.m[which][w]);
#pragma unroll
  for (int w = 0; w < RT / 64; ++w) s += sh.s[which][w] * shrink(sh.m[which][w], m, k);
  return {m, s};
}

// Columns behind the row's end count as -inf.
__device__ __forceinline__ void fill_behind(Vec8<float>& v, int n) {
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i >= n) v.r[i >> 2][i & 3] = 0xff800000u;
}
__device__ __forceinline__ void fill_behind(Vec8<uint16_t>& v, int n) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (2 * i >= n) v.r[i] = 0xff80ff80u;
    else if (2 * i + 1 >= n) v.r[i] = (v.r[i] & 0xffffu) | 0xff800000u;
  }
}
// The row stays as loaded: without this the compiler keeps the unpacked floats of the
// first pass for the second, in twice the registers.
__device__ __forceinline__ void keep_raw(Vec8<float>& v) { asm volatile("" : "+v"(v.r[0]), "+v"(v.r[1])); }
__device__ __forceinline__ void keep_raw(Vec8<uint16_t>& v) { asm volatile("" : "+v"(v.r)); }

template <class T>
__device__ __forceinline__ void settle_row(Vec8<T>& v, int c, int n) {
  if (n < 8) {
    settle8(v, c, n);
    fill_behind(v, n);
  }
}

template <class T>
__device__ __forceinline__ float value_at(const T* p) {
  if constexpr (sizeof(T) == 2) return bf2f(gld<uint16_t>(p));
  else return gld<float>(p);
}
template <class T>
__device__ __forceinline__ void put_value(T* p, float v) {
  if constexpr (sizeof(T) == 2) gst<uint16_t>(p, f2bf(v));
  else gst<float>(p, v);
}
__device__ __forceinline__ int64_t id_at(const void* ids, int64_t i, int32_t id_bytes) {
  return id_bytes == 8 ? gld<int64_t>(static_cast<const int64_t*>(ids) + i)
                       : static_cast<int64_t>(gld<int32_t>(static_cast<const int32_t*>(ids) + i));
}

// N vectors' maximum, and sum of 2^((x - base) k).
template <class T, int N>
__device__ __forceinline__ float top_of(const Vec8<T> (&x)[N]) {
  float m = kNegInf;
#pragma unroll
  for (int j = 0; j < N; ++j)
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, x[j].get(i));
  return m;
}
template <class T, int N>
__device__ __forceinline__ float sum_of(Vec8<T> (&x)[N], float base, float k) {
  float s = 0.f;
#pragma unroll
  for (int j = 0; j < N; ++j) {
    keep_raw(x[j]);
    float e[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = exp2_fast((x[j].get(i) - base) * k);
    s += ((e[0] + e[1]) + (e[2] + e[3])) + ((e[4] + e[5]) + (e[6] + e[7]));
  }
  return s;
}
// n (8 or more: all) of the vector's columns at out: a 2^((x - base) k)
template <class T>
__device__ __forceinline__ void put_scaled(T* out, int n, Vec8<T>& x, float base, float k, float a) {
  keep_raw(x);
  float g[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) g[i] = a * exp2_fast((x.get(i) - base) * k);
  Vec8<T>::store(out, n, g);
}

// A row in the registers of RT threads: `step` of them have VPL vectors each, vector
// t + j step the j-th of thread t.  All but the last lie inside the row (which has
// (VPL - 1)^2 + VPL vectors at least), so that one scalar address and one offset a lane
// do for them and only the last goes by its length.
template <class T, int RT, int VPL, bool SHARED>
struct Row {
  const T* p;
  int cols, t, step;
  Vec8<T> x[VPL];

  __device__ __forceinline__ Row(const T* p_, int cols_, int t_) : p(p_), cols(cols_), t(t_) {
    step = (((cols + 7) >> 3) + VPL - 1) / VPL;
  }
  __device__ __forceinline__ int last() const { return ((VPL - 1) * step + t) * 8; }
  __device__ __forceinline__ void fetch() {
#pragma unroll
    for (int j = 0; j < VPL; ++j) fill_behind(x[j], 0);
    if (t < step) {
#pragma unroll
      for (int j = 0; j < VPL - 1; ++j) x[j].load(p + j * step * 8 + static_cast<uint32_t>(t * 8));
      fetch8(x[VPL - 1], p + last(), last(), cols - last());
    }
  }
  // the thread's maximum and sum
  __device__ __forceinline__ Soft stats(float k) {
    if (t < step) settle_row(x[VPL - 1], last(), cols - last());
    const float m = wave_max(top_of(x));
    return {m, sum_of(x, base_of(m), k)};
  }
  // whether the block writes the vectors j of its row (uniform)
  static __device__ __forceinline__ bool mine(int j) {
    return !SHARED || static_cast<uint32_t>(j) * gridDim.y / VPL == blockIdx.y;
  }
  // out[c] = a 2^((x[c] - base) k), the block's share of it
  __device__ __forceinline__ void scaled(T* out, float base, float k, float a) {
    if (t >= step) return;
#pragma unroll
    for (int j = 0; j < VPL - 1; ++j)
      if (mine(j)) put_scaled(out + j * step * 8 + static_cast<uint32_t>(t * 8), 8, x[j], base, k, a);
    if (mine(VPL - 1)) put_scaled(out + last(), cols - last(), x[VPL - 1], base, k, a);
  }
  // whether this block, and of it this thread, has written column c
  __device__ __forceinline__ bool has(int c) const { return mine((c >> 3) / step); }
  __device__ __forceinline__ bool wrote(int c) const { return has(c) && (c >> 3) % step == t; }
};

// A row of any length, read twice: kPass vectors a thread at a time, then single ones.
constexpr int kPass = 4;
template <class T, int RT, bool SHARED>
struct Row<T, RT, 0, SHARED> {
  const T* p;
  int cols, t;
  Vec8<T> x[kPass];

  __device__ __forceinline__ Row(const T* p_, int cols_, int t_) : p(p_), cols(cols_), t(t_) {}
  __device__ __forceinline__ void fetch() {}
  __device__ __forceinline__ void load(int at) {
#pragma unroll
    for (int j = 0; j < kPass; ++j) x[j].load(p + at + j * RT * 8 + static_cast<uint32_t>(t * 8));
  }
  __device__ __forceinline__ Soft stats(float k) {
    Soft a{kNegInf, 0.f};
    auto add = [&](float top, auto sum) {
      const float m = fmaxf(a.m, top);
      a.s = a.s * shrink(a.m, m, k) + sum(base_of(m));
      a.m = m;
    };
    int at = 0;
    for (; at + kPass * RT * 8 <= cols; at += kPass * RT * 8) {
      load(at);
      add(top_of(x), [&](float base) { return sum_of(x, base, k); });
    }
#pragma unroll 1
    for (; at < cols; at += RT * 8) {
      Vec8<T> v[1];
      load8(v[0], p + at + t * 8, at + t * 8, cols - at - t * 8);
      if (cols - at - t * 8 < 8) fill_behind(v[0], cols - at - t * 8);
      add(top_of(v), [&](float base) { return sum_of(v, base, k); });
    }
    return a;
  }
  // (passes are dealt to the row's blocks in turn)
  static constexpr int kSpan = kPass * RT * 8;
  __device__ __forceinline__ bool has(int c) const {
    return !SHARED || static_cast<uint32_t>(c / kSpan) % gridDim.y == blockIdx.y;
  }
  __device__ __forceinline__ void scaled(T* out, float base, float k, float a) {
    int at = 0;
    for (; at + kSpan <= cols; at += kSpan) {
      if (!has(at)) continue;
      load(at);
#pragma unroll
      for (int j = 0; j < kPass; ++j) put_scaled(out + at + j * RT * 8 + static_cast<uint32_t>(t * 8), 8, x[j], base, k, a);
    }
#pragma unroll 1
    for (; at < cols && has(at); at += RT * 8) {
      const int c = at + t * 8;
      Vec8<T> v;
      load8(v, p + c, c, cols - c);
      put_scaled(out + c, cols - c, v, base, k, a);
    }
  }
  __device__ __forceinline__ bool wrote(int c) const { return has(c) && (c >> 3) % RT == t; }
};

// Waves a SIMD, by the registers that the row takes of the 64, 80 or 128 they leave (policy
// loss, 16384 x 32000 in bf16: 6 waves 338 us, 8 with some of the row spilled 359, 4 521).
// Also as it is some instances keep up to 8 values besides the row in scratch, written and
// read once a row; k_distill<*, 64, *> has 5 waves, for its LDS.
template <class T, int VPL>
constexpr int occupancy() {
  constexpr int row = (VPL ? VPL : kPass) * static_cast<int>(sizeof(T)) * 2;
  return row <= 16 ? 8 : row <= 32 ? 6 : 4;
}

template <class T, int RT>
__device__ __forceinline__ void zero_row(T* out, int cols, int t) {
  const float z[8] = {};
  for (int c = t * 8; c < cols; c += RT * 8) Vec8<T>::store(out + c, cols - c, z);
}

// ------------------------------------------------------------ distillation ----
// The entries' ids and teacher logits lie in LDS.  Their columns are written with
// all others and then once more, behind a barrier, by the thread that has the entry:
// softmax minus the sum of p over the entries of the same id, in their order (so
// threads of one id write the same value).
template <class T, int RT, int VPL, bool SHARED>
__global__ __launch_bounds__(RT, (occupancy<T, VPL>())) void k_distill(muon_distill_t op) {
  constexpr int top_max = MUON_DISTILL_MAX_TOP;
  __shared__ Shared<RT> sh;
  __shared__ __attribute__((aligned(16))) int id[top_max];
  __shared__ __attribute__((aligned(16))) float pt[top_max];   // teacher logits, then p
  const int t = static_cast<int>(threadIdx.x), wave = t >> 6, share = SHARED ? blockIdx.y : 0, top = static_cast<int>(op.top);
  const int padded = (top + 3) & ~3;
  const float k = kLog2e / op.temperature;
  for (int64_t row = blockIdx.x; row < op.tokens; row += gridDim.x) {
    const T* p = static_cast<const T*>(op.logits) + row * op.ld_logits;
    T* out = op.dlogits ? static_cast<T*>(op.dlogits) + row * op.ld_dlogits : nullptr;
    const float weight = op.weights ? gld<float>(op.weights + row) : 1.f;
    if (weight == 0.f) {
      if (out && share == 0) zero_row<T, RT>(out, static_cast<int>(op.vocab), t);
      if (t == 0 && share == 0) gst<float>(op.loss + row, 0.f);
      continue;
    }
    Row<T, RT, VPL, SHARED> x(p, static_cast<int>(op.vocab), t);
    x.fetch();
    Soft teach{kNegInf, 0.f};
    for (int e = t; e < padded; e += RT) {
      int64_t i = -1;
      float v = kNegInf;
      if (e < top) {
        i = id_at(op.ids, row * op.ld_ids + e, op.id_bytes);
        v = op.teacher_dtype == MUON_BF16 ? value_at(static_cast<const uint16_t*>(op.teacher) + row * op.ld_teacher + e)
                                          : value_at(static_cast<const float*>(op.teacher) + row * op.ld_teacher + e);
        if (i < 0 || i >= op.vocab || v == kNegInf) {
          i = -1;
          v = kNegInf;
        }
      }
      id[e] = static_cast<int>(i);
      pt[e] = v;
      const float m = fmaxf(teach.m, v);
      teach.s = teach.s * shrink(teach.m, m, k) + exp2_fast((v - base_of(m)) * k);
      teach.m = m;
    }
    teach = wave_join(teach, k);
    const Soft mine = wave_join(x.stats(k), k);
    if ((t & 63) == 0) {
      sh.m[0][wave] = mine.m;
      sh.s[0][wave] = mine.s;
      sh.m[1][wave] = teach.m;
      sh.s[1][wave] = teach.s;
    }
    __syncthreads();
    const Soft q = block_join<RT>(sh, 0, k);
    teach = block_join<RT>(sh, 1, k);
    const bool none = teach.s == 0.f;               // no entry, no loss
    const float base = base_of(q.m), lq = log2_fast(q.s), lt = log2_fast(teach.s), tbase = base_of(teach.m);
    float part = 0.f;
    for (int e = t; e < padded; e += RT) {
      const int i = id[e];
      float pe = 0.f;
      if (i >= 0) {
        const float le = (pt[e] - tbase) * k - lt;   // log2 of p
        pe = exp2_fast(le);
        if (pe != 0.f) part += pe * (le * 0.5f - half_log2(value_at(p + i), base, k, lq));
      }
      pt[e] = pe;
    }
    part = wave_add(part);
    if ((t & 63) == 0) sh.part[wave] = part;
    const float a = weight * op.temperature;
    if (out) {
      if (none) {
        if (share == 0) zero_row<T, RT>(out, x.cols, t);
      } else {
        x.scaled(out, base, k, a / q.s);
      }
    }
    __syncthreads();
    if (t == 0 && share == 0) {
      float sum = 0.f;
#pragma unroll
      for (int w = 0; w < RT / 64; ++w) sum += sh.part[w];
      gst<float>(op.loss + row, none ? 0.f : a * op.temperature * (2 * kLn2) * sum);
    }
    if (out && !none)
      for (int e = t; e < top; e += RT) {
        const int i = id[e];
        if (i < 0 || !x.has(i)) continue;
        float sum = 0.f;
        for (int f = 0; f < padded; f += 4) {
          const int4 ids = *reinterpret_cast<const int4*>(id + f);
          const float4 ps = *reinterpret_cast<const float4*>(pt + f);
          sum += ids.x == i ? ps.x : 0.f;
          sum += ids.y == i ? ps.y : 0.f;
          sum += ids.z == i ? ps.z : 0.f;
          sum += ids.w == i ? ps.w : 0.f;
        }
        put_value(out + i, a * (exp2_fast((value_at(p + i) - base) * k) / q.s - sum));
      }
    if (row + gridDim.x < op.tokens) __syncthreads();   // (uniform) before the next row's entries
  }
}

// ------------------------------------------------------------- policy loss ----
// exp(d) - 1 - d, which d^2 / 2 ... carries where the difference would cancel.
__device__ __forceinline__ float exp_less_linear(float d) {
  if (fabsf(d) > 0.25f) return expm1f(d) - d;
  return d * d * (0.5f + d * (1.f / 6 + d * (1.f / 24 + d * (1.f / 120 + d * (1.f / 720 + d * (1.f / 5040))))));
}

template <class T, int RT, int VPL, bool SHARED>
__global__ __launch_bounds__(RT, (occupancy<T, VPL>())) void k_policy(muon_policy_t op) {
  __shared__ Shared<RT> sh;
  const int t = static_cast<int>(threadIdx.x), wave = t >> 6, share = SHARED ? blockIdx.y : 0;
  const float k = kLog2e / op.temperature;
  for (int64_t row = blockIdx.x; row < op.tokens; row += gridDim.x) {
    const T* p = static_cast<const T*>(op.logits) + row * op.ld_logits;
    T* out = op.dlogits ? static_cast<T*>(op.dlogits) + row * op.ld_dlogits : nullptr;
    const float weight = op.weights ? gld<float>(op.weights + row) : 1.f;
    const int64_t act = id_at(op.actions, row, op.id_bytes);
    if (weight == 0.f || act < 0 || act >= op.vocab) {
      if (out && share == 0) zero_row<T, RT>(out, static_cast<int>(op.vocab), t);
      if (t == 0 && share == 0) {
        gst<float>(op.loss + row, 0.f);
        if (op.logp) gst<float>(op.logp + row, 0.f);
      }
      continue;
    }
    Row<T, RT, VPL, SHARED> x(p, static_cast<int>(op.vocab), t);
    x.fetch();
    const float xa = value_at(p + act), adv = gld<float>(op.advantages + row), old = gld<float>(op.old_logp + row),
                ref = op.ref_logp ? gld<float>(op.ref_logp + row) : 0.f;
    const Soft mine = wave_join(x.stats(k), k);
    if ((t & 63) == 0) {
      sh.m[0][wave] = mine.m;
      sh.s[0][wave] = mine.s;
    }
    __syncthreads();
    const Soft q = block_join<RT>(sh, 0, k);
    const float base = base_of(q.m), la = (xa - base) * k;
    const float logp = half_log2(xa, base, k, log2_fast(q.s)) * (2 * kLn2);
    const float ratio = expf(logp - old);
    // an advantage of 0 has no part, whatever the ratio
    const float free = adv == 0.f ? 0.f : ratio * adv;
    const float held = fminf(fmaxf(ratio, 1.f - op.clip_low), 1.f + op.clip_high) * adv;
    // a comparison that NaN fails lets it through
    float loss = held < free ? -held : -free, slope = held < free ? 0.f : -free;
    // a coefficient of 0 has no part either, whatever the reference (exp(d) may be infinite)
    if (op.ref_logp && op.kl_coef != 0.f) {
      const float d = ref - logp;
      loss += op.kl_coef * exp_less_linear(d);
      slope -= op.kl_coef * expm1f(d);
    }
    if (t == 0 && share == 0) {
      gst<float>(op.loss + row, weight * loss);
      if (op.logp) gst<float>(op.logp + row, logp);
    }
    if (out) {
      const float g = weight * slope / op.temperature;
      x.scaled(out, base, k, -g / q.s);
      // the action's column once more, by the thread that has just written it
      if (x.wrote(static_cast<int>(act))) put_value(out + act, g * (1.f - exp2_fast(la) / q.s));
    }
    if (row + gridDim.x < op.tokens) __syncthreads();   // (uniform) before the next row's sums
  }
}

// ---------------------------------------------------------------- dispatch ----
constexpr int64_t kFewRows = 512;   // two blocks a CU

// f(threads of a row, vectors of 8 columns a thread).  Few rows: as many threads to a
// row as have work, for its latency.  Many: as few as hold it beside the other rows of a
// CU, a wave up to 2048 columns, so that several rows are in flight (32768 x 5000 in
// bf16: 256 threads 175 us, 512 244; 1 x 32000: 1024 threads and 512 the same 8 us, 37 x
// 1000: 256 threads 4.0 us, a wave 5.4).
template <class T, class F>
int by_shape(int64_t rows, int64_t cols, F&& f) {
  auto with = [&](auto rt, auto vpl) { return f(rt, vpl); };
  using std::integral_constant;
#define MUON_ROW(RT, VPL) return with(integral_constant<int, RT>{}, integral_constant<int, VPL>{})
  if (cols <= 512) MUON_ROW(64, 1);
  if (rows <= kFewRows) {
    if (cols <= 2048) MUON_ROW(256, 1);
    if (cols <= 8192) MUON_ROW(1024, 1);
    if (cols <= 16384) MUON_ROW(1024, 2);
    if (cols <= 32768) MUON_ROW(1024, 4);
    if (cols <= 65536) MUON_ROW(1024, 8);
  }
  if (cols <= 2048) MUON_ROW(64, 4);
  if (cols <= 8192) MUON_ROW(256, 4);
  if (cols <= 16384) MUON_ROW(512, 4);
  if (cols <= 32768) MUON_ROW(512, 8);
  if constexpr (sizeof(T) == 2) {
    if (cols <= 65536) MUON_ROW(512, 16);
    if (cols <= 131072) MUON_ROW(1024, 16);
  } else {
    if (cols <= 65536) MUON_ROW(1024, 8);
  }
  MUON_ROW(1024, 0);
#undef MUON_ROW
}

constexpr int64_t kMaxGrid = int64_t(1) << 21;   // threads of a grid stay below 2^32

unsigned rows_grid(int64_t tokens) { return static_cast<unsigned>(tokens < kMaxGrid ? tokens : kMaxGrid); }

// Blocks of a long row: where the chip has more CUs than there are rows, several take the
// same one, each with statistics of its own, and share the writing of its gradient (and
// the second exponentials): no exchange between them, and the same bits.  One row of
// 200000 columns in bf16 27 us alone, 18 shared, of 131072 18, 12, 128 of them 24, 22, 20 of
// 200000 in fp32 35, 20, one of 32000 9 with and without; many rows would pay 1 to 2 % for
// the choice, so it is a kernel of its own.
constexpr bool shares(int rt, int vpl) { return rt == 1024 && (vpl == 0 || vpl >= 8); }
unsigned share_of(int64_t rows, int vpl, bool gradient) {
  unsigned share = 1;
  while (gradient && 2 * share <= static_cast<unsigned>(vpl ? vpl : 8) && rows * 2 * share <= 256) share *= 2;
  return share;
}

}  // namespace

int launch_distill(const muon_distill_t& op, void* stream) {
  auto run = [&](auto type) {
    using T = decltype(type);
    return by_shape<T>(op.tokens, op.vocab, [&](auto rt, auto vpl) {
      constexpr int RT = decltype(rt)::value, VPL = decltype(vpl)::value;
      const unsigned share = shares(RT, VPL) ? share_of(op.tokens, VPL, op.dlogits != nullptr) : 1;
      if (share > 1)
        hipLaunchKernelGGL((k_distill<T, RT, VPL, shares(RT, VPL)>), dim3(rows_grid(op.tokens), share), dim3(RT), 0, static_cast<hipStream_t>(stream), op);
      else
        hipLaunchKernelGGL((k_distill<T, RT, VPL, false>), dim3(rows_grid(op.tokens)), dim3(RT), 0, static_cast<hipStream_t>(stream), op);
      return static_cast<int>(hipGetLastError());
    });
  };
  return op.dtype == MUON_BF16 ? run(uint16_t{}) : run(float{});
}

int launch_policy(const muon_policy_t& op, void* stream) {
  auto run = [&](auto type) {
    using T = decltype(type);
    return by_shape<T>(op.tokens, op.vocab, [&](auto rt, auto vpl) {
      constexpr int RT = decltype(rt)::value, VPL = decltype(vpl)::value;
      const unsigned share = shares(RT, VPL) ? share_of(op.tokens, VPL, op.dlogits != nullptr) : 1;
      if (share > 1)
        hipLaunchKernelGGL((k_policy<T, RT, VPL, shares(RT, VPL)>), dim3(rows_grid(op.tokens), share), dim3(RT), 0, static_cast<hipStream_t>(stream), op);
      else
        hipLaunchKernelGGL((k_policy<T, RT, VPL, false>), dim3(rows_grid(op.tokens)), dim3(RT), 0, static_cast<hipStream_t>(stream), op);
      return static_cast<int>(hipGetLastError());
    });
  };
  return op.dtype == MUON_BF16 ? run(uint16_t{}) : run(float{});
}

}  // namespace muon
