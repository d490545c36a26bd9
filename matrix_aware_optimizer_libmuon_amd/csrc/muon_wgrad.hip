// Weight gradient of a linear layer from its 8-bit input (gfx950):
//   dW[i][j] = gain[j] sum_t dY[t][i] x[t][j],   x[t][j] = code[t][j] 2^e[t][j / 32].
//
// Both factors are summed over their rows, so both lie in LDS as in memory,
// [token][column], and the fragments of v_mfma_f32_16x16x32_bf16 are taken from
// there by transposing reads (the MN-contiguous form of muon_gemm.h).  A value
// of x8 is a 4-bit significand times a power of two: bf16 holds it exactly, so
// unpacking loses nothing, and the products are exact in fp32.
//
// The scale changes with the token, which is the summed index, so it cannot
// wait for the epilogue: x is unpacked between global memory and the matrix
// instruction.  Once per block (and not once per wave that reads a fragment):
// the codes and their scale bytes go straight into LDS; two steps later each
// wave turns the 8 tokens that it loaded itself into bf16 (two values of one
// group share an instruction) and writes them to a second LDS tile, from where
// on both operands are alike.
//
// Bounds.  Every load goes through a buffer descriptor that ends where the
// matrix ends: past it LDS receives zeros (whole dwords count, hence the
// alignment rule below), so tokens past the end add nothing and no address
// leaves the matrix.  Columns past a row's end read the next row and reach only
// outputs that are not stored.
#include <algorithm>

#include "muon_act8.h"
#include "muon_gemm.h"
#include "muon_ops.h"

namespace muon {

namespace {

// ---------------------------------------------------------------- loads ----
// 16 bytes (or one byte, zero-extended to a dword) per lane from buffer `srd` at
// voff + soff into LDS, at lds_dst + 16 (4) times the lane.  As dma16() of
// muon_gemm.h: an asm statement with explicit waits, whose scalar operands are
// formed by scalar instructions (tests/test_ops_isa.py checks the compiled code);
// the s_nop keeps the wait state between a scalar write of m0 and a load to LDS.
template <bool BYTE>
__device__ __forceinline__ void dma_bounded(u32x4 srd, uint32_t voff, uint32_t soff, const void* lds_dst) {
  const uint32_t m0 = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(
      (__attribute__((address_space(3))) void*)lds_dst));
  if constexpr (BYTE)
    asm volatile("s_nop 0\n\tbuffer_load_ubyte %0, %1, %2 offen lds" ::"v"(voff), "s"(srd), "s"(soff), "{m0}"(m0));
  else
    asm volatile("s_nop 0\n\tbuffer_load_dwordx4 %0, %1, %2 offen lds" ::"v"(voff), "s"(srd), "s"(soff), "{m0}"(m0));
}

// The descriptor of `rows` rows from row0, columns from byte col0, of a matrix:
// it ends with the last of them (wgrad_plan keeps that below 2^31 bytes).
__device__ __forceinline__ u32x4 window(const void* p, int64_t ld_bytes, int64_t row_bytes, int64_t row0, int64_t rows, int64_t col0) {
  const uint64_t b = reinterpret_cast<uint64_t>(p) + row0 * ld_bytes + col0;
  u32x4 srd;
  srd[0] = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(b));
  srd[1] = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(b >> 32) & 0xffffu);
  srd[2] = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>((rows - 1) * ld_bytes + row_bytes - col0));
  srd[3] = 0x00020000u;   // raw buffer of dwords
  return srd;
}

// TN x TK: the output tile, TN columns of dY by TK columns of x.
template <int TN, int TK>
struct Lds {
  static constexpr int PE = TN * BK * 2;                 // bytes of a stage: dY,
  static constexpr int BE = TK * BK * 2;                 // unpacked x,
  static constexpr int RE = TK * BK;                     // codes,
  static constexpr int SE = 4 * 64 * 4;                  // scales (a dword per wave and lane)
  static constexpr int B = 0;                            // 3 stages of unpacked x
  static constexpr int P = B + 3 * BE;                   // 4 stages of each load
  static constexpr int R = P + 4 * PE;
  static constexpr int S = R + 4 * RE;
  static constexpr int bytes = S + 4 * SE;
};
static_assert(Lds<256, 256>::bytes <= 160 * 1024 && 2 * Lds<128, 128>::bytes <= 160 * 1024, "LDS per CU");

// ------------------------------------------------------------ the product ----
// acc += dY[t0 .. + rows, i0 .. + TN]^T x[t0 .. + rows, j0 .. + TK], in steps of
// 32 tokens; 4 waves of TN / 2 x TK / 2, one MFMA per slot in the order of
// muon_gemm.h, operands exchanged (a lane ends up with four consecutive columns of
// one row).
//
// Step kt opens with a wait for this wave's loads of two steps before (dY of
// step kt + 1, codes and scales of kt + 2 have landed) and a barrier, and then
//   multiplies dY[kt] and x[kt], whose first fragments were read in step kt - 1,
//   loads dY of step kt + 3 and codes and scales of step kt + 4,
//   unpacks x of step kt + 2, into the tile whose fragments were read in step
//   kt - 2 and used in step kt - 1.
// So before the barrier only the wave's writes of the unpacked x have to be done,
// not its last fragment reads, which are used later: LDS finishes in order, and
// AFTER reads were issued after the last write.  (Waiting for them all, with two stages of x, left the matrix units idle for the length of an
// LDS read in each step.)
// Loads past the last token give zeros and read nothing.
//
// At 256 x 256 a SIMD has one wave, which issues an instruction every 4 cycles at
// best, 256 of them while its 64 MFMAs run: the loop has to stay below that.
// Hence descriptors that hold for the whole product, where a step is a scalar
// offset.
//
// The wave's codes of a step are 8 token rows; each lane unpacks 8 columns at a
// time, the lanes side by side along a row, so that 8 consecutive lanes write 128
// consecutive bytes (LDS takes a 16-byte write in such groups: with a lane on 32
// columns of its own the writes took four times as long).
template <int TN, int TK>
__device__ __forceinline__ void product(const muon_act8_wgrad_t& op, int64_t i0, int64_t j0, int64_t t0, int64_t rows,
                                        char* smem, f32x4_t (&acc)[TN / 32][TK / 32], int tid) {
  using L = Lds<TN, TK>;
  constexpr int NA = TN / 32, NB = TK / 32;              // MFMA blocks of a wave
  constexpr int H = NA / 2, PASS = H * NB, SLOTS = NA * NB;
  constexpr int LP = TN / 64, LR = TK / 128, LPS = LP + LR + 1;
  constexpr int LSS = (SLOTS - H) / LPS;                 // loads spread over the step
  const int lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int rowA = TN / 2 * (w >> 1), rowB = TK / 2 * (w & 1);
  const int steps = static_cast<int>((rows + BK - 1) / BK);

  const uint32_t ldp = static_cast<uint32_t>(op.ld_dy * 2), ldr = static_cast<uint32_t>(op.x8.ld_codes),
                 lds = static_cast<uint32_t>(op.x8.ld_scales);
  // rows end on a dword: in memory, or in the padding of an aligned copy
  const u32x4 dp = window(op.dy, op.ld_dy * 2, (op.n * 2 + 3) / 4 * 4, t0, rows, i0 * 2);
  const u32x4 dr = window(op.x8.codes, op.x8.ld_codes, (op.k + 3) / 4 * 4, t0, rows, j0);
  const u32x4 ds = window(op.x8.scales, op.x8.ld_scales, (op.k + 31) / 32, t0, rows, j0 / 32);
  // dY: the MN-contiguous form of DmaFeed (muon_gemm.h)
  constexpr int CPR = TN / 8, RPB = 512 / TN;            // chunks of a row, rows of a 1 KB load
  uint32_t vp[2];
#pragma unroll
  for (int par = 0; par < 2; ++par) {
    const int r = lane / CPR, c = (lane % CPR) ^ (2 * ((RPB * par + r) & 3) + 8 * (w & 1));
    vp[par] = r * ldp + 16 * c;
  }
  constexpr int RCPR = TK / 16, RRPB = 1024 / TK;        // the same of the codes
  const uint32_t vr = (lane / RCPR) * ldr + 16 * (lane % RCPR);
  constexpr int SPR = TK / 32;                           // scales of a row; lanes past 8 rows repeat
  const uint32_t vs = ((lane / SPR) & 7) * lds + lane % SPR;
  // the wave's share of the step to be loaded next: dY parts 0 .. LP - 1, codes, scales
  uint32_t sp = (w * LP * RPB) * ldp, sr = (w * LR * RRPB) * ldr, ss = (w * 8) * lds;
  auto load_p = [&](int st, auto part) __attribute__((always_inline)) {        // st: kt & 3
    constexpr int q = decltype(part)::value;
    dma_bounded<false>(dp, vp[q & 1], sp + q * (RPB * ldp), smem + L::P + st * L::PE + (w * LP + q) * 1024);
    if constexpr (q == LP - 1) sp += BK * ldp;
  };
  auto load_x = [&](int st, auto part) __attribute__((always_inline)) {
    constexpr int q = decltype(part)::value;
    if constexpr (q < LR) {
      dma_bounded<false>(dr, vr, sr + q * (RRPB * ldr), smem + L::R + st * L::RE + (w * LR + q) * 1024);
      if constexpr (q == LR - 1) sr += BK * ldr;
    } else {
      dma_bounded<true>(ds, vs, ss, smem + L::S + st * L::SE + w * 256);
      ss += BK * lds;
    }
  };

  // unpacking: piece q covers 1024 / TK rows of the wave's 8, 8 columns a lane
  constexpr int Q = 2 * LR, URP = 8 / Q, UL = 64 / URP;  // pieces, rows of a piece, lanes of a row
  const int ur = lane / UL, uc = lane % UL;
  const char* const raw_at = smem + L::R + (8 * w + ur) * TK + 8 * uc;
  const char* const sb_at = smem + L::S + w * 256 + (ur * SPR + (uc >> 2)) * 4;
  char* x_at[Q];
#pragma unroll
  for (int q = 0; q < Q; ++q) {
    const int r = URP * q + ur;
    x_at[q] = smem + L::B + (8 * w + r) * (TK * 2) + ((uc ^ (2 * (r & 3) + 8 * (w & 1))) << 4);
  }
  u32x2 raw[Q];
  uint32_t sb[Q];
  auto fetch = [&](int st, auto piece) __attribute__((always_inline)) {
    constexpr int q = decltype(piece)::value;
    raw[q] = *reinterpret_cast<const u32x2*>(raw_at + st * L::RE + URP * q * TK);
    sb[q] = *reinterpret_cast<const uint32_t*>(sb_at + st * L::SE + URP * q * SPR * 4);
  };
  u32x4 o;
  auto unpack = [&](int st, auto part) __attribute__((always_inline)) {        // a quarter of a piece; st: the tile's place
    constexpr int q = decltype(part)::value / 4, i = decltype(part)::value % 4;
    const float scale = act8_scale(sb[q]);
    o[i] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(raw[q][i >> 1], scale, (i & 1) != 0));
    if constexpr (i == 3) *reinterpret_cast<u32x4*>(x_at[q] + st) = o;
  };
  auto tile_p = [&](int st) { return reinterpret_cast<const uint16_t*>(smem + L::P + st * L::PE); };
  auto tile_b = [&](int st) { return reinterpret_cast<const uint16_t*>(smem + L::B + st); };

  // x8 of steps 0 .. 3 and dY of steps 0 .. 2, the share of the loop's step -1 last
  static_for<2>([&](auto k) { static_for<LR + 1>([&](auto part) { load_x(k, part); }); });
  static_for<3>([&](auto k) {
    static_for<LP>([&](auto part) { load_p(k, part); });
    if constexpr (decltype(k)::value > 0)
      static_for<LR + 1>([&](auto part) { load_x(k + 1, part); });
  });
  vm_wait<LPS>();
  static_for<2>([&](auto k) {
    static_for<Q>([&](auto q) { fetch(k, q); });
    static_for<4 * Q>([&](auto part) { unpack(k * L::BE, part); });
  });
  lds_barrier();
  bf16x8_t fa[NA], fb[NB];
#pragma unroll
  for (int r = 0; r < H; ++r) fa[r] = frag<true, TN>(tile_p(0), rowA + 16 * r, lane);
#pragma unroll
  for (int r = 0; r < NB; ++r) fb[r] = frag<true, TK>(tile_b(0), rowB + 16 * r, lane);

  // a wait that the compiler knows of: with reads pending on entry it would wait
  // for all of them at the top of every step
  __builtin_amdgcn_s_waitcnt(0xc07f);                     // lgkmcnt(0)
  // LDS operations issued after the step's last write: fragments of the next step
  constexpr int AFTER = 2 * (H + NB) < 15 ? 2 * (H + NB) : 15;
  constexpr int CPS = SLOTS == 16 ? 4 : 1, U0 = PASS - 4 * Q / CPS;   // conversions of a slot, first slot of them
  static_assert(U0 > H + Q, "after the codes");
  int b0 = 0, b1 = L::BE, b2 = 2 * L::BE;                 // places of x of steps kt, kt + 1, kt + 2
  for (int kt = 0; kt < steps; ++kt) {
    vm_wait<LPS>();
    asm volatile("s_waitcnt lgkmcnt(%0)\n\ts_barrier" ::"n"(AFTER) : "memory");
    const uint16_t* cu = tile_p(kt & 3);
    const uint16_t* nx = tile_p((kt + 1) & 3);
    const uint16_t* nb = tile_b(b1);
    static_for<SLOTS>([&](auto sc) __attribute__((always_inline)) {
      constexpr int s = decltype(sc)::value, pass = s / PASS, at = s % PASS;
      constexpr int bi = pass * H + at % H, bj = at / H;
      acc[bi][bj] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fb[bj], fa[bi], acc[bi][bj], 0, 0, 0);
      if constexpr (s < H) fa[H + s] = frag<true, TN>(cu, rowA + 16 * (H + s), lane);
      if constexpr (s >= PASS && s < PASS + H) fa[s - PASS] = frag<true, TN>(nx, rowA + 16 * (s - PASS), lane);
      if constexpr (pass == 1 && at % H == H - 1) fb[bj] = frag<true, TK>(nb, rowB + 16 * bj, lane);
      if constexpr (s >= H && (s - H) % LSS == 0 && (s - H) / LSS < LPS) {
        constexpr int part = (s - H) / LSS;
        if constexpr (part < LP) load_p((kt + 3) & 3, std::integral_constant<int, part>{});
        else load_x(kt & 3, std::integral_constant<int, part - LP>{});
      }
      // unpacking: codes and scales early, the conversions in the slots before the second pass
      if constexpr (s >= H && s < H + Q) fetch((kt + 2) & 3, std::integral_constant<int, s - H>{});
      if constexpr (s >= U0 && s < PASS)
        static_for<CPS>([&](auto k) { unpack(b2, std::integral_constant<int, (s - U0) * CPS + decltype(k)::value>{}); });
      __builtin_amdgcn_sched_barrier(0);
    });
    const int b = b0;
    b0 = b1;
    b1 = b2;
    b2 = b;
  }
  vm_wait<0>();
}

// ---------------------------------------------------------------- output ----
// Four consecutive elements from column j of row i, n of them inside.
template <class T>
__device__ __forceinline__ void put4(const muon_act8_wgrad_t& op, int64_t i, int64_t j, f32x4_t v) {
  const int n = static_cast<int>(min(op.k - j, int64_t(4)));
  T* p = static_cast<T*>(op.dw) + i * op.ld_dw + j;
  typedef float f32x4_a4 __attribute__((ext_vector_type(4), aligned(4)));
  typedef uint16_t u16x4_a2 __attribute__((ext_vector_type(4), aligned(2)));
  if (n == 4) {
    if (op.col_gain) v *= gld<f32x4_a4>(op.col_gain + j);
    if constexpr (sizeof(T) == 2) {
      if (op.accumulate) {
        const u16x4_a2 o = gld<u16x4_a2>(p);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] += bf2f(o[e]);
      }
      u16x4_a2 o;
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] = f2bf(v[e]);
      gst<u16x4_a2>(p, o);
    } else {
      if (op.accumulate) v += gld<f32x4_a4>(p);
      gst<f32x4_a4>(p, v);
    }
    return;
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if (e >= n) break;
    float x = v[e];
    if (op.col_gain) x *= gld<float>(op.col_gain + j + e);
    if constexpr (sizeof(T) == 2) {
      if (op.accumulate) x += bf2f(gld<uint16_t>(p + e));
      gst<uint16_t>(p + e, f2bf(x));
    } else {
      if (op.accumulate) x += gld<float>(p + e);
      gst<float>(p + e, x);
    }
  }
}

template <int TN, int TK>
__global__ __launch_bounds__(kGemmThreads) void k_wgrad(muon_act8_wgrad_t op, WgradPlan p, float* partial) {
  __shared__ __attribute__((aligned(16))) char smem[Lds<TN, TK>::bytes];
  const int tid = opaque_tid();
  // first the tiles that are one block's whole, then the others, range by range
  const uint32_t nwhole = static_cast<uint32_t>(p.whole), tiles = static_cast<uint32_t>(p.tiles_n * p.tiles_k);
  const bool whole = blockIdx.x < nwhole;
  const uint32_t unit = static_cast<uint32_t>(whole ? xcd_remap(blockIdx.x, nwhole)
                                                    : xcd_remap(blockIdx.x - nwhole, gridDim.x - nwhole));
  const uint32_t split = whole ? 0u : unit / (tiles - nwhole);
  int64_t ti, tj;
  decode_full(whole ? unit : nwhole + unit - split * (tiles - nwhole), p.tiles_n, p.tiles_k, ti, tj);
  const int64_t i0 = ti * TN, j0 = tj * TK, t0 = split * p.split_rows;
  const int64_t rows = whole ? op.tokens : min(p.split_rows, op.tokens - t0);
  const bool last = whole || p.splits == 1;
  partial += static_cast<int64_t>(unit) * (TN * TK);
  constexpr int NA = TN / 32, NB = TK / 32;
  f32x4_t acc[NA][NB];
#pragma unroll
  for (int bi = 0; bi < NA; ++bi)
#pragma unroll
    for (int bj = 0; bj < NB; ++bj) acc[bi][bj] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  product<TN, TK>(op, i0, j0, t0, rows, smem, acc, tid);
  // The sums leave through LDS, TN / 2 rows (two waves) at a time, whole rows
  // of the tile side by side: 16-byte pieces, piece c of row r at c ^ (r & 15) (the
  // 16 rows that one write instruction covers then fall on distinct banks).
  // Lane: row 16 bi + (lane & 15), columns 16 bj + 4 (lane >> 4) .. + 3.
  static_assert(TN / 2 * TK * 4 <= Lds<TN, TK>::bytes, "half a tile of fp32");
  const int lane = tid & 63, w = tid >> 6;
  constexpr int PPR = TK / 4;                       // pieces of a row
  for (int half = 0; half < 2; ++half) {
    lds_barrier();
    if ((w >> 1) == half) {
#pragma unroll
      for (int bi = 0; bi < NA; ++bi)
#pragma unroll
        for (int bj = 0; bj < NB; ++bj) {
          const int r = 16 * bi + (lane & 15), c = (TK / 8) * (w & 1) + 4 * bj + (lane >> 4);
          *reinterpret_cast<f32x4_t*>(smem + (r * PPR + (c ^ (r & 15))) * 16) = acc[bi][bj];
        }
    }
    lds_barrier();
#pragma unroll 4
    for (int u = tid; u < TN / 2 * PPR; u += kGemmThreads) {
      const int r = u / PPR, c = u % PPR;
      const int64_t i = i0 + half * (TN / 2) + r, j = j0 + 4 * c;
      if (i < op.n && j < op.k) {
        const f32x4_t v = *reinterpret_cast<const f32x4_t*>(smem + (r * PPR + (c ^ (r & 15))) * 16);
        if (!last) gst<f32x4_t>(partial + (half * (TN / 2) + r) * TK + 4 * c, v);
        else if (op.dw_dtype == MUON_BF16) put4<uint16_t>(op, i, j, v);
        else put4<float>(op, i, j, v);
      }
    }
  }
}

// The sums of the token ranges, added in order (no range: zero), 4 columns a
// thread.  partial: [range][tile of the rest][TN][TK].
template <int TN, int TK>
__global__ __launch_bounds__(256) void k_wgrad_join(muon_act8_wgrad_t op, WgradPlan p, const float* partial) {
  constexpr int PPR = TK / 4, PER = TN * PPR / 256;      // pieces of a row, shares of a tile
  const int64_t rest = p.tiles_n * p.tiles_k - p.whole;
  for (int64_t b = blockIdx.x; b < rest * PER; b += gridDim.x) {   // 256 pieces of one tile
    const int64_t tile = b / PER;
    const int u = static_cast<int>(b % PER) * 256 + threadIdx.x, r = u / PPR, c = u % PPR;
    int64_t ti, tj;
    decode_full(p.whole + tile, p.tiles_n, p.tiles_k, ti, tj);
    const int64_t i = ti * TN + r, j = tj * TK + 4 * c;
    if (i >= op.n || j >= op.k) continue;
    f32x4_t v{0.f, 0.f, 0.f, 0.f};
    const float* at = partial + tile * (TN * TK) + r * TK + 4 * c;
#pragma unroll 8
    for (int s = 0; s < static_cast<int>(p.splits); ++s) v += gld<f32x4_t>(at + s * rest * (TN * TK));
    if (op.dw_dtype == MUON_BF16) put4<uint16_t>(op, i, j, v);
    else put4<float>(op, i, j, v);
  }
}

// Matrices of `width`-byte rows at any place, copied to rows of ld_out bytes (a
// multiple of 16), zeros past each row's end; all of a call's in one launch.
struct Copy {
  const uint8_t* in;
  uint8_t* out;
  int64_t ld_in, width, ld_out;
  int64_t begin, end;         // blocks of this one, 256 pieces of 16 bytes each
};
struct Copies {
  Copy c[3];
  int n;
  int64_t rows;
};
__global__ __launch_bounds__(256) void k_wgrad_copy(Copies a) {
  typedef uint32_t u32x4_a1 __attribute__((ext_vector_type(4), aligned(1)));
  for (int64_t b = blockIdx.x; b < a.c[a.n - 1].end; b += gridDim.x) {
    int which = 0;
    while (b >= a.c[which].end) ++which;
    const Copy& k = a.c[which];
    const uint32_t per = static_cast<uint32_t>(k.ld_out / 16);
    const uint64_t first = static_cast<uint64_t>(b - k.begin) * 256, row0 = first / per;   // uniform
    const uint32_t u = static_cast<uint32_t>(first - row0 * per) + threadIdx.x, dr = u / per;
    const int64_t r = static_cast<int64_t>(row0 + dr), c = static_cast<int64_t>(u - dr * per) * 16;
    if (r >= a.rows) continue;
    const uint8_t* p = k.in + r * k.ld_in + c;
    u32x4 v{0, 0, 0, 0};
    if (c + 16 <= k.width) {
      v = gld<u32x4_a1>(p);
    } else {
#pragma unroll
      for (int e = 0; e < 16; ++e)
        if (c + e < k.width) v[e >> 2] |= static_cast<uint32_t>(gld<uint8_t>(p + e)) << (8 * (e & 3));
    }
    gst<u32x4>(k.out + r * k.ld_out + c, v);
  }
}

bool is_aligned(const void* p, int64_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
int64_t up(int64_t x, int64_t a) { return (x + a - 1) / a * a; }

}  // namespace

namespace {

// The tile sizes: blocks that the chip holds, and what a step of one takes with
// the chip full, or with one block to a CU (us).  Larger tiles read less from LDS
// per product, smaller ones waste less of a matrix and need fewer token ranges;
// measured, in the order of the table (us):
//   8192 x 4096 x 4096   231  281  310        16384 x 768 x 1536    56   54   59
//   8192 x 4096 x 1024    77   79   88        16001 x  80 x 1536    30   26   21
//   4096 x 2048 x 2048    53   49   51          256 x 256 x  768    25   16    9
// The estimate takes the fastest of the three but for 8192 x 4096 x 1024 (256 x 128,
// 2 % slower) and 4096 x 2048 x 2048 (128 x 128, 3 % slower): it overrates what
// token ranges cost.
struct WgradTile {
  int tn, tk;
  int64_t slots;
  double step_us, alone_us;
};
constexpr WgradTile kWgradTiles[] = {{256, 256, 256, 0.80, 0.80}, {256, 128, 256, 0.50, 0.50}, {128, 128, 512, 0.55, 0.40}};

// How a tile size would be dealt to the chip: `whole` tiles that one block makes
// alone, in full rounds of the chip, and the rest cut into token ranges such that
// they fill it too; and an estimate of the time, from measured figures.
struct WgradShape {
  int64_t whole, split_steps;
  double us;
};

WgradShape wgrad_shape(const muon_act8_wgrad_t& op, const WgradTile& t, int64_t steps, int64_t most) {
  const int64_t tiles = ((op.n + t.tn - 1) / t.tn) * ((op.k + t.tk - 1) / t.tk);
  // `units` blocks of `each` steps, 6 us to begin and end one
  auto run = [&](int64_t units, int64_t each) {
    const int64_t full = units / t.slots, left = units - full * t.slots;
    return full * (each * t.step_us + 6.0) + (left > 0 ? each * (left > 256 ? t.step_us : t.alone_us) + 6.0 : 0.0);
  };
  const bool fits = steps <= most;
  const int64_t whole = fits ? tiles / t.slots * t.slots : 0, cut = tiles - whole;
  WgradShape best{tiles, steps, fits ? run(tiles, steps) : 1e30};
  const double share = static_cast<double>(cut) / tiles * op.n * op.k * 4;   // bytes of the cut tiles' sums
  for (int64_t want = 2; want <= 64 && cut > 0; ++want) {
    const int64_t each = (steps + want - 1) / want, ranges = each ? (steps + each - 1) / each : 0;
    if (each < 4 && want > 2) break;
    if (each > most) continue;
    // the sums of the ranges are written and read once, at about 4 TB/s, and joined by one more launch
    const double us = run(whole, steps) + run(cut * ranges, each) + 2.0 * ranges * share / 4e6 + 5.0;
    if (us < best.us) best = {whole, each, us};
  }
  if (best.us >= 1e30) best = {0, most, 1e29};            // more than 64 ranges: by the bound alone
  return best;
}

}  // namespace

WgradPlan wgrad_plan(const muon_act8_wgrad_t& op) {
  WgradPlan p{};
  // the loads take 16 bytes at multiples of 16, rows that end on a dword, and
  // 32-bit offsets
  constexpr int64_t kMaxLd = int64_t(1) << 21;
  p.copy_dy = op.tokens > 0 && !(is_aligned(op.dy, 16) && op.ld_dy % 8 == 0 && op.ld_dy < kMaxLd && op.n % 2 == 0);
  p.copy_x = op.tokens > 0 && !(is_aligned(op.x8.codes, 16) && op.x8.ld_codes % 16 == 0 && op.x8.ld_codes < kMaxLd &&
                                op.x8.ld_scales < kMaxLd && op.k % 4 == 0);
  const int64_t ld = std::max({(p.copy_dy ? up(op.n, 8) : op.ld_dy) * 2, p.copy_x ? up(op.k, 16) : op.x8.ld_codes,
                               p.copy_x ? int64_t(1) : op.x8.ld_scales});
  const int64_t most = (int64_t(1) << 31) / ld / BK - 1;   // steps of a range below 2^31 bytes
  const int64_t steps = (op.tokens + BK - 1) / BK;
  WgradShape w{0, 0, 2e30};
  for (const WgradTile& t : kWgradTiles) {
    const WgradShape c = wgrad_shape(op, t, steps, most);
    if (c.us >= w.us) continue;
    w = c;
    p.tn = t.tn;
    p.tk = t.tk;
  }
  p.tiles_n = (op.n + p.tn - 1) / p.tn;
  p.tiles_k = (op.k + p.tk - 1) / p.tk;
  p.whole = w.whole;
  p.split_rows = std::max<int64_t>(1, w.split_steps) * BK;
  p.splits = p.whole == p.tiles_n * p.tiles_k ? 1 : (op.tokens + p.split_rows - 1) / p.split_rows;
  if (op.tokens == 0) p.whole = p.splits = 0;              // k_wgrad_join writes the zeros
  size_t off = 0;
  auto take = [&](int64_t bytes) {
    const size_t at = off;
    off += static_cast<size_t>(up(bytes, 256));
    return at;
  };
  if (p.splits > 1) p.partial_off = take(p.splits * (p.tiles_n * p.tiles_k - p.whole) * p.tn * p.tk * 4);
  if (p.copy_dy) p.dy_off = take(op.tokens * up(op.n, 8) * 2);
  if (p.copy_x) {
    p.x_off = take(op.tokens * up(op.k, 16));
    p.s_off = take(op.tokens * up((op.k + 31) / 32, 16));
  }
  p.bytes = off;
  return p;
}

int launch_wgrad_copy(muon_act8_wgrad_t& op, const WgradPlan& p, char* ws, void* stream) {
  Copies a{};
  a.rows = op.tokens;
  int64_t end = 0;
  auto add = [&](const void* in, int64_t ld_in, int64_t width, size_t off, int64_t ld_out) {
    const int64_t begin = end;
    end += (op.tokens * (ld_out / 16) + 255) / 256;
    a.c[a.n++] = {static_cast<const uint8_t*>(in), reinterpret_cast<uint8_t*>(ws + off), ld_in, width, ld_out, begin, end};
    return reinterpret_cast<uint8_t*>(ws + off);
  };
  if (p.copy_dy) {
    const int64_t ld = up(op.n, 8);
    op.dy = add(op.dy, op.ld_dy * 2, op.n * 2, p.dy_off, ld * 2);
    op.ld_dy = ld;
  }
  if (p.copy_x) {
    const int64_t ld = up(op.k, 16), groups = (op.k + 31) / 32, lds = up(groups, 16);
    op.x8.codes = add(op.x8.codes, op.x8.ld_codes, op.k, p.x_off, ld);
    op.x8.ld_codes = ld;
    op.x8.scales = add(op.x8.scales, op.x8.ld_scales, groups, p.s_off, lds);
    op.x8.ld_scales = lds;
  }
  hipLaunchKernelGGL(k_wgrad_copy, dim3(static_cast<unsigned>(std::min(end, int64_t(1) << 23))), dim3(256), 0, static_cast<hipStream_t>(stream), a);
  return static_cast<int>(hipGetLastError());
}

namespace {
// f(TN, TK) of the plan
template <class F>
void by_tile(const WgradPlan& p, F&& f) {
  using std::integral_constant;
  if (p.tk == 256) f(integral_constant<int, 256>{}, integral_constant<int, 256>{});
  else if (p.tn == 256) f(integral_constant<int, 256>{}, integral_constant<int, 128>{});
  else f(integral_constant<int, 128>{}, integral_constant<int, 128>{});
}
}  // namespace

int launch_wgrad(const muon_act8_wgrad_t& op, const WgradPlan& p, char* ws, void* stream) {
  const int64_t rest = p.tiles_n * p.tiles_k - p.whole;
  const dim3 grid(static_cast<unsigned>(p.whole + rest * p.splits));
  float* partial = reinterpret_cast<float*>(ws + p.partial_off);   // not used where there is one range
  by_tile(p, [&](auto tn, auto tk) {
    hipLaunchKernelGGL((k_wgrad<decltype(tn)::value, decltype(tk)::value>), grid, dim3(kGemmThreads), 0,
                       static_cast<hipStream_t>(stream), op, p, partial);
  });
  return static_cast<int>(hipGetLastError());
}

int launch_wgrad_join(const muon_act8_wgrad_t& op, const WgradPlan& p, const char* ws, void* stream) {
  const int64_t rest = p.tiles_n * p.tiles_k - p.whole;
  const dim3 grid(static_cast<unsigned>(std::min<int64_t>(rest * (p.tn * p.tk / 1024), int64_t(1) << 22)));
  const float* partial = reinterpret_cast<const float*>(ws + p.partial_off);
  by_tile(p, [&](auto tn, auto tk) {
    hipLaunchKernelGGL((k_wgrad_join<decltype(tn)::value, decltype(tk)::value>), grid, dim3(256), 0,
                       static_cast<hipStream_t>(stream), op, p, partial);
  });
  return static_cast<int>(hipGetLastError());
}

}  // namespace muon
