// Weight gradient of a linear layer from its 8-bit input (gfx950):
//   dW[i][j] = gain[j] sum_t dY[t][i] x[t][j].
//
// Both factors are summed over their rows, so both reach LDS as they lie in
// memory, [token][column], and the matrix instruction's fragments are taken
// from there by transposing reads (as in muon_gemm.h).  A value of x8 is a 4-bit
// significand times a power of two: bf16 holds it exactly, so the products are
// those of the bf16 matrix instruction and nothing is lost by unpacking.
#include <algorithm>

#include "muon_act8.h"
#include "muon_gemm.h"
#include "muon_ops.h"

namespace muon {

namespace {

constexpr int kTile = 128;
using G = Geo<kTile>;

// LDS place of the 16-byte chunk c of token row r (see muon_gemm.h).
__device__ __forceinline__ int chunk_at(int r, int c) {
  return r * kTile + ((c ^ (2 * (r & 3) + 8 * ((r >> 3) & 1))) << 3);
}

template <class T>
__device__ __forceinline__ void put_out(const muon_act8_wgrad_t& op, int64_t i, int64_t j, float v) {
  if (op.col_gain) v *= gld<float>(op.col_gain + j);
  T* p = static_cast<T*>(op.dw) + i * op.ld_dw + j;
  if constexpr (sizeof(T) == 2) {
    if (op.accumulate) v += bf2f(gld<uint16_t>(p));
    gst<uint16_t>(p, f2bf(v));
  } else {
    if (op.accumulate) v += gld<float>(p);
    gst<float>(p, v);
  }
}

__global__ __launch_bounds__(kGemmThreads) void k_wgrad(muon_act8_wgrad_t op, WgradPlan p, float* partial) {
  __shared__ __attribute__((aligned(16))) uint16_t sm[2 * G::TE];
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  const int64_t unit = blockIdx.x, tiles = p.tiles_n * p.tiles_k;
  const int64_t split = unit / tiles, tile = unit % tiles;
  const int64_t i0 = tile / p.tiles_k * kTile, j0 = tile % p.tiles_k * kTile;
  const int64_t t0 = split * p.split_rows;
  const int64_t t1 = t0 + p.split_rows < op.tokens ? t0 + p.split_rows : op.tokens;
  const uint16_t* dy = static_cast<const uint16_t*>(op.dy);
  f32x4_t acc[G::NB][G::NB];
  zero_acc<G::NB>(acc);
  const int rowA = G::WT * (w >> 1), rowB = G::WT * (w & 1);
  for (int64_t t = t0; t < t1; t += BK) {
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int v = tid + q * kGemmThreads, r = v >> 4, c = v & 15;
      const bool in = t + r < t1;
      Vec8<uint16_t> a;
      load8(a, dy + (t + r) * op.ld_dy + i0 + c * 8, in ? static_cast<int>(min(op.n - i0 - c * 8, int64_t(8))) : 0);
      *reinterpret_cast<u32x4*>(sm + chunk_at(r, c)) = a.r;
      const int n = in ? static_cast<int>(min(op.k - j0 - c * 8, int64_t(8))) : 0;
      u32x4 b{0, 0, 0, 0};
      if (n > 0) {
        const u32x2 code = load_codes(op.x8.codes + (t + r) * op.x8.ld_codes + j0 + c * 8, n);
        float f[8];
        act8_decode(code, gld<uint8_t>(op.x8.scales + (t + r) * op.x8.ld_scales + ((j0 + c * 8) >> 5)), f);
#pragma unroll
        for (int k = 0; k < 4; ++k) b[k] = pack2(f[2 * k], f[2 * k + 1]);
      }
      *reinterpret_cast<u32x4*>(sm + G::TE + chunk_at(r, c)) = b;
    }
    __syncthreads();
    bf16x8_t fa[G::NB], fb[G::NB];
#pragma unroll
    for (int k = 0; k < G::NB; ++k) {
      fa[k] = frag<true, kTile>(sm, rowA + 16 * k, lane);
      fb[k] = frag<true, kTile>(sm + G::TE, rowB + 16 * k, lane);
    }
#pragma unroll
    for (int bi = 0; bi < G::NB; ++bi)
#pragma unroll
      for (int bj = 0; bj < G::NB; ++bj)
        acc[bi][bj] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fb[bj], fa[bi], acc[bi][bj], 0, 0, 0);
    __syncthreads();
  }
  // lane: row 16 bi + (lane & 15), columns 16 bj + 4 (lane >> 4) .. + 3
#pragma unroll
  for (int bi = 0; bi < G::NB; ++bi) {
    const int64_t i = i0 + rowA + 16 * bi + (lane & 15);
    if (i >= op.n) continue;
#pragma unroll
    for (int bj = 0; bj < G::NB; ++bj)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int64_t j = j0 + rowB + 16 * bj + 4 * (lane >> 4) + e;
        if (j >= op.k) continue;
        if (p.splits > 1) gst<float>(partial + (split * op.n + i) * op.k + j, acc[bi][bj][e]);
        else if (op.dw_dtype == MUON_BF16) put_out<uint16_t>(op, i, j, acc[bi][bj][e]);
        else put_out<float>(op, i, j, acc[bi][bj][e]);
      }
  }
}

// The token ranges' sums, added in order (no range: zero).
__global__ __launch_bounds__(256) void k_wgrad_join(muon_act8_wgrad_t op, int64_t splits, const float* partial) {
  for (int64_t u = blockIdx.x * int64_t(256) + threadIdx.x; u < op.n * op.k; u += int64_t(gridDim.x) * 256) {
    float v = 0.f;
    for (int64_t s = 0; s < splits; ++s) v += gld<float>(partial + s * op.n * op.k + u);
    const int64_t i = u / op.k, j = u % op.k;
    if (op.dw_dtype == MUON_BF16) put_out<uint16_t>(op, i, j, v);
    else put_out<float>(op, i, j, v);
  }
}

}  // namespace

WgradPlan wgrad_plan(const muon_act8_wgrad_t& op) {
  WgradPlan p;
  p.tiles_n = (op.n + kTile - 1) / kTile;
  p.tiles_k = (op.k + kTile - 1) / kTile;
  const int64_t tiles = p.tiles_n * p.tiles_k, steps = (op.tokens + BK - 1) / BK;
  // token ranges until there are two blocks per CU, of 8 steps at least
  int64_t want = std::max<int64_t>(1, std::min<int64_t>(512 / tiles, steps / 8));
  p.split_rows = std::max<int64_t>(1, (steps + want - 1) / want) * BK;
  p.splits = (op.tokens + p.split_rows - 1) / p.split_rows;
  p.bytes = p.splits > 1 ? static_cast<size_t>(p.splits) * op.n * op.k * sizeof(float) : 0;
  return p;
}

int launch_wgrad(const muon_act8_wgrad_t& op, const WgradPlan& p, void* workspace, void* stream) {
  hipLaunchKernelGGL(k_wgrad, dim3(static_cast<unsigned>(p.splits * p.tiles_n * p.tiles_k)), dim3(kGemmThreads), 0,
                     static_cast<hipStream_t>(stream), op, p, static_cast<float*>(workspace));
  return static_cast<int>(hipGetLastError());
}

int launch_wgrad_join(const muon_act8_wgrad_t& op, const WgradPlan& p, const void* workspace, void* stream) {
  const int64_t blocks = std::min<int64_t>((op.n * op.k + 255) / 256, 8192);
  hipLaunchKernelGGL(k_wgrad_join, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, static_cast<hipStream_t>(stream),
                     op, p.splits, static_cast<const float*>(workspace));
  return static_cast<int>(hipGetLastError());
}

}  // namespace muon
