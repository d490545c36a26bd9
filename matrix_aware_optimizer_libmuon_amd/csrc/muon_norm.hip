// RMS norm with the residual's addition and its backward pass, on 8-bit
// activations (gfx950).
//
// A row is held in the registers of RT threads (a wave, or a block of 256 to
// 1024), VPL vectors of 8 columns each, thread t the vectors t, t + RT: one
// read of every input, one write of every output, the row's sums by wave
// permutations and, past a wave, through LDS.  Both passes are bound by memory.
#include "muon_act8.h"
#include "muon_ops.h"

namespace muon {

namespace {

// Rows per block: 4 waves with a row each, or the whole block on one.
template <int RT>
struct Rows {
  static constexpr int threads = RT < 128 ? 256 : RT;
  static constexpr int per_block = threads / RT;
};

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
  return v;
}

// Sum over the RT threads of a row, in every one of them.  `red` holds two
// sets of RT / 64 partial sums, used in turn so that one barrier is enough.
template <int RT>
__device__ __forceinline__ float row_sum(float v, float* red, int turn) {
  v = wave_sum(v);
  if constexpr (RT > 64) {
    constexpr int W = RT / 64;
    float* r = red + (turn & 1) * W;
    if ((threadIdx.x & 63) == 0) r[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) v += r[w];
  }
  return v;
}

template <class T, int RT, int VPL>
__global__ __launch_bounds__(Rows<RT>::threads) void k_rmsnorm(muon_rmsnorm_t op) {
  using R = Rows<RT>;
  __shared__ float red[2 * (RT / 64)];
  const int t = static_cast<int>(threadIdx.x) % RT;
  const int cols = static_cast<int>(op.cols);
  int turn = 0;
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * R::per_block + threadIdx.x / RT; row < op.rows;
       row += static_cast<int64_t>(gridDim.x) * R::per_block) {
    Vec8<T> x[VPL], r[VPL];
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      const int c = (t + j * RT) * 8;
      fetch8(x[j], static_cast<const T*>(op.x) + row * op.ld_x + c, c, cols - c);
      if (op.residual) fetch8(r[j], static_cast<const T*>(op.residual) + row * op.ld_residual + c, c, cols - c);
    }
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      const int c = (t + j * RT) * 8;
      settle8(x[j], c, cols - c);
      if (op.residual) settle8(r[j], c, cols - c);
    }
    float h[VPL][8], ss = 0.f;
#pragma unroll
    for (int j = 0; j < VPL; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        h[j][i] = op.residual ? x[j].get(i) + r[j].get(i) : x[j].get(i);
        ss = fmaf(h[j][i], h[j][i], ss);
      }
    ss = row_sum<RT>(ss, red, turn++);
    const float rstd = rsqrtf(ss / static_cast<float>(cols) + op.eps);
    if (op.rstd && t == 0) gst<float>(op.rstd + row, rstd);
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      const int c = (t + j * RT) * 8, n = cols - c;
      if (op.h) Vec8<T>::store(static_cast<T*>(op.h) + row * op.ld_h + c, n, h[j]);
#pragma unroll
      for (int i = 0; i < 8; ++i) h[j][i] *= rstd;
      if (op.n.codes) act8_put(op.n, row, c, n, h[j]);
      if (op.y) {
        if (op.gain) {
          Vec8<float> g;
          load8(g, op.gain + c, c, n);
#pragma unroll
          for (int i = 0; i < 8; ++i) h[j][i] *= g.get(i);
        }
        Vec8<T>::store(static_cast<T*>(op.y) + row * op.ld_y + c, n, h[j]);
      }
    }
  }
}

// The backward pass.  Block b takes rows b, b + gridDim.x, ...; each thread
// sums dy n of its columns over them, into dgain where there is one block,
// else into the block's row of `partial`, which k_dgain adds up in order.
template <class T, int RT, int VPL>
__global__ __launch_bounds__(Rows<RT>::threads) void k_rmsnorm_grad(muon_rmsnorm_grad_t op, float* partial) {
  using R = Rows<RT>;
  __shared__ float red[2 * (RT / 64)];
  __shared__ float cross[R::per_block > 1 ? R::per_block : 1][R::per_block > 1 ? RT * VPL * 8 : 1];
  const int t = static_cast<int>(threadIdx.x) % RT;
  const int cols = static_cast<int>(op.cols);
  float gain[VPL][8], dg[VPL][8];
#pragma unroll
  for (int j = 0; j < VPL; ++j) {
    const int c = (t + j * RT) * 8;
    Vec8<float> g;
    if (op.gain) load8(g, op.gain + c, c, cols - c);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      gain[j][i] = op.gain ? g.get(i) : 1.f;
      dg[j][i] = 0.f;
    }
  }
  int turn = 0;
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * R::per_block + threadIdx.x / RT; row < op.rows;
       row += static_cast<int64_t>(gridDim.x) * R::per_block) {
    Vec8<T> dy[VPL], dres[VPL];
    Codes8 code[VPL];
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      const int c = (t + j * RT) * 8, n = cols - c;
      fetch8(dy[j], static_cast<const T*>(op.dy) + row * op.ld_dy + c, c, n);
      if (op.dres) fetch8(dres[j], static_cast<const T*>(op.dres) + row * op.ld_dres + c, c, n);
      code[j].fetch(op.n, row, c, n);
    }
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      const int c = (t + j * RT) * 8, n = cols - c;
      settle8(dy[j], c, n);
      if (op.dres) settle8(dres[j], c, n);
      code[j].settle(c, n);
    }
    const float rstd = gld<float>(op.rstd + row);
    float gd[VPL][8], nv[VPL][8], s = 0.f;
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      code[j].get(nv[j]);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float d = dy[j].get(i);
        gd[j][i] = d * gain[j][i];
        s = fmaf(gd[j][i], nv[j][i], s);
        dg[j][i] = fmaf(d, nv[j][i], dg[j][i]);
      }
    }
    s = row_sum<RT>(s, red, turn++) / static_cast<float>(cols);
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      const int c = (t + j * RT) * 8;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float d = rstd * fmaf(-nv[j][i], s, gd[j][i]);
        gd[j][i] = op.dres ? d + dres[j].get(i) : d;
      }
      Vec8<T>::store(static_cast<T*>(op.dx) + row * op.ld_dx + c, cols - c, gd[j]);
    }
  }
  if (!op.dgain) return;
  float* out = gridDim.x == 1 ? op.dgain : partial + static_cast<int64_t>(blockIdx.x) * cols;
  if constexpr (R::per_block > 1) {   // the block's waves in order
    const int w = threadIdx.x / RT;
#pragma unroll
    for (int j = 0; j < VPL; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) cross[w][(t + j * RT) * 8 + i] = dg[j][i];
    __syncthreads();
    for (int c = threadIdx.x; c < cols; c += R::threads) {
      float v = 0.f;
#pragma unroll
      for (int k = 0; k < R::per_block; ++k) v += cross[k][c];
      gst<float>(out + c, v);
    }
  } else {
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      const int c = (t + j * RT) * 8;
      Vec8<float>::store(out + c, cols - c, dg[j]);
    }
  }
}

// dgain[c] = sum over blocks of partial[b][c]: 16 columns per block, the partial
// rows dealt in turn to its 64 groups of 16 threads.
constexpr int kDgainCols = 16, kDgainThreads = 1024;
__global__ __launch_bounds__(kDgainThreads) void k_dgain(const float* partial, int64_t blocks, int cols, float* dgain) {
  constexpr int kGroups = kDgainThreads / kDgainCols, kWaves = kDgainThreads / 64;
  __shared__ float red[kWaves][kDgainCols];
  const int t = static_cast<int>(threadIdx.x), g = t / kDgainCols;
  const int c = static_cast<int>(blockIdx.x) * kDgainCols + t % kDgainCols;
  float v = 0.f;
  if (c < cols) {
#pragma unroll 8
    for (int b = g; b < static_cast<int>(blocks); b += kGroups) v += gld<float>(partial + static_cast<int64_t>(b) * cols + c);
  }
  v += __shfl_xor(v, 16, 64);
  v += __shfl_xor(v, 32, 64);
  if ((t & 63) < kDgainCols) red[t >> 6][t & 63] = v;
  __syncthreads();
  if (t < kDgainCols && c < cols) {
    v = 0.f;
#pragma unroll
    for (int k = 0; k < kWaves; ++k) v += red[k][t];
    gst<float>(dgain + c, v);
  }
}

// f(RT, VPL) for the layout of a row: one vector a thread up to 8192 columns
// (two a thread, with half the threads, need twice the registers: 115 us instead
// of 90 for the backward pass of 16384 x 4096 bf16).  Past 8192 columns there are no
// more threads to take: two vectors each, where the backward pass needs more than the
// 128 registers a thread then has, and spills (80 bytes a lane in bf16, 120 in fp32).
template <class F>
int by_width(int64_t cols, F&& f) {
  if (cols <= 512) return f(std::integral_constant<int, 64>{}, std::integral_constant<int, 1>{});
  if (cols <= 1024) return f(std::integral_constant<int, 128>{}, std::integral_constant<int, 1>{});
  if (cols <= 2048) return f(std::integral_constant<int, 256>{}, std::integral_constant<int, 1>{});
  if (cols <= 4096) return f(std::integral_constant<int, 512>{}, std::integral_constant<int, 1>{});
  if (cols <= 8192) return f(std::integral_constant<int, 1024>{}, std::integral_constant<int, 1>{});
  return f(std::integral_constant<int, 1024>{}, std::integral_constant<int, 2>{});
}
static_assert(MUON_NORM_MAX_COLS == 1024 * 2 * 8, "widest layout");

// threads of a grid stay below 2^32
constexpr int64_t kMaxGrid = int64_t(1) << 21;
// Threads of the backward pass, all resident at once (half as many: 109 us, one
// and a half times: 103, this: 88 for 16384 x 4096 bf16); and 4 rows to a wave or
// block at least, or the partial sums of dgain cost as much as the rows (2048 x 768
// bf16: 15.4 us with one row, 11.5 with 4, 14.1 with 8).
constexpr int64_t kGradThreads = 1024 * 256;

}  // namespace

int launch_rmsnorm(const muon_rmsnorm_t& op, void* stream) {
  return by_width(op.cols, [&](auto rt, auto vpl) {
    constexpr int RT = decltype(rt)::value, VPL = decltype(vpl)::value;
    const int64_t need = (op.rows + Rows<RT>::per_block - 1) / Rows<RT>::per_block;
    const dim3 grid(static_cast<unsigned>(need < kMaxGrid ? need : kMaxGrid)), block(Rows<RT>::threads);
    if (op.dtype == MUON_BF16)
      hipLaunchKernelGGL((k_rmsnorm<uint16_t, RT, VPL>), grid, block, 0, static_cast<hipStream_t>(stream), op);
    else
      hipLaunchKernelGGL((k_rmsnorm<float, RT, VPL>), grid, block, 0, static_cast<hipStream_t>(stream), op);
    return static_cast<int>(hipGetLastError());
  });
}

int64_t rmsnorm_grad_blocks(int64_t rows, int64_t cols) {
  return by_width(cols, [&](auto rt, auto) {
    using R = Rows<decltype(rt)::value>;
    const int64_t need = (rows + 4 * R::per_block - 1) / (4 * R::per_block), most = kGradThreads / R::threads;
    return static_cast<int>(need < most ? need : most);
  });
}

int launch_rmsnorm_grad(const muon_rmsnorm_grad_t& op, float* partial, void* stream) {
  const dim3 grid(static_cast<unsigned>(rmsnorm_grad_blocks(op.rows, op.cols)));
  return by_width(op.cols, [&](auto rt, auto vpl) {
    constexpr int RT = decltype(rt)::value, VPL = decltype(vpl)::value;
    const dim3 block(Rows<RT>::threads);
    if (op.dtype == MUON_BF16)
      hipLaunchKernelGGL((k_rmsnorm_grad<uint16_t, RT, VPL>), grid, block, 0, static_cast<hipStream_t>(stream), op, partial);
    else
      hipLaunchKernelGGL((k_rmsnorm_grad<float, RT, VPL>), grid, block, 0, static_cast<hipStream_t>(stream), op, partial);
    return static_cast<int>(hipGetLastError());
  });
}

int launch_rmsnorm_dgain(const float* partial, int64_t blocks, int64_t cols, float* dgain, void* stream) {
  hipLaunchKernelGGL(k_dgain, dim3(static_cast<unsigned>((cols + kDgainCols - 1) / kDgainCols)), dim3(kDgainThreads), 0,
                     static_cast<hipStream_t>(stream), partial, blocks, static_cast<int>(cols), dgain);
  return static_cast<int>(hipGetLastError());
}

}  // namespace muon
