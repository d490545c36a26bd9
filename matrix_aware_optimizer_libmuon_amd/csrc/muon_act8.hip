// Elementwise operators on 8-bit activations (gfx950): pack, unpack, the gated
// unit and its backward pass.
//
// One lane handles 8 columns of one row; the vectors of a row are rounded up to
// a multiple of 4 so that a group of 32 columns never leaves its quad.  A block
// takes 256 consecutive vectors of the rows laid end to end.  All of these are
// bound by memory: each value is read once and written once.
#include "muon_act8.h"
#include "muon_ops.h"

namespace muon {

constexpr int kThreads = 256;

// The row and first column of this thread's vector in the block's b-th share;
// false past the last row (whole quads together).
struct Place {
  int64_t row;
  int col, n;   // n: valid columns of the vector (may be <= 0)
};
__device__ __forceinline__ bool place(int64_t b, int64_t rows, int cols, Place& p) {
  const uint32_t vpr = static_cast<uint32_t>((cols + 31) >> 5) * 4;   // vectors per row
  const uint64_t first = static_cast<uint64_t>(b) * kThreads;
  const uint64_t row0 = first / vpr;                                  // uniform
  const uint32_t u = static_cast<uint32_t>(first - row0 * vpr) + threadIdx.x;
  const uint32_t dr = u / vpr;
  p.row = static_cast<int64_t>(row0 + dr);
  p.col = static_cast<int>(u - dr * vpr) * 8;
  p.n = cols - p.col;
  return p.row < rows;
}

// f(place) for every vector of this block: one, unless the matrix has more
// shares than a grid has blocks.
template <class F>
__device__ __forceinline__ void each_vector(int64_t blocks, int64_t rows, int cols, F&& f) {
  for (int64_t b = blockIdx.x; b < blocks; b += gridDim.x) {
    Place p;
    if (place(b, rows, cols, p)) f(p);
  }
}

template <class T>
__global__ __launch_bounds__(kThreads) void k_act8_pack(int64_t blocks, const T* x, int64_t ld, int64_t rows, int cols,
                                                        muon_act8_t out) {
  each_vector(blocks, rows, cols, [&](const Place& p) __attribute__((always_inline)) {
    Vec8<T> raw;
    load8(raw, x + p.row * ld + p.col, p.col, p.n);
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = raw.get(i);
    act8_put(out, p.row, p.col, p.n, v);
  });
}

template <class T>
__global__ __launch_bounds__(kThreads) void k_act8_unpack(int64_t blocks, muon_act8_t in, int64_t rows, int cols, T* out,
                                                          int64_t ld) {
  each_vector(blocks, rows, cols, [&](const Place& p) __attribute__((always_inline)) {
    Codes8 c;
    c.fetch(in, p.row, p.col, p.n);
    c.settle(p.col, p.n);
    float v[8];
    c.get(v);
    Vec8<T>::store(out + p.row * ld + p.col, p.n, v);
  });
}

// sigma(g) = 1 / (1 + exp(-g)).  Where the exponential is infinite (g below
// about -88.7) it is 0, its limit, and the products with g stay finite.  The
// reciprocal instruction gives 0 for denominators above 2^126, hence the scaling
// by 2^-24 around it, which is exact.
__device__ __forceinline__ float sigmoid(float g) {
  return __builtin_amdgcn_rcpf((1.f + __expf(-g)) * 0x1p-24f) * 0x1p-24f;
}

template <class T>
__global__ __launch_bounds__(kThreads) void k_swiglu(int64_t blocks, muon_swiglu_t op) {
  each_vector(blocks, op.rows, static_cast<int>(op.cols), [&](const Place& p) __attribute__((always_inline)) {
    Vec8<T> rg, ru;
    fetch8(rg, static_cast<const T*>(op.gate) + p.row * op.ld_gate + p.col, p.col, p.n);
    fetch8(ru, static_cast<const T*>(op.up) + p.row * op.ld_up + p.col, p.col, p.n);
    settle8(rg, p.col, p.n);
    settle8(ru, p.col, p.n);
    float g[8], u[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      g[i] = rg.get(i);
      u[i] = ru.get(i);
    }
    if (op.a) {
      float a[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) a[i] = g[i] * sigmoid(g[i]) * u[i];
      Vec8<T>::store(static_cast<T*>(op.a) + p.row * op.ld_a + p.col, p.n, a);
    }
    if (op.gate8.codes) {
      act8_put(op.gate8, p.row, p.col, p.n, g);
      act8_put(op.up8, p.row, p.col, p.n, u);
    }
  });
}

template <class T>
__global__ __launch_bounds__(kThreads) void k_swiglu_grad(int64_t blocks, muon_swiglu_grad_t op) {
  each_vector(blocks, op.rows, static_cast<int>(op.cols), [&](const Place& p) __attribute__((always_inline)) {
    Vec8<T> rd;
    Codes8 cg, cu;
    fetch8(rd, static_cast<const T*>(op.da) + p.row * op.ld_da + p.col, p.col, p.n);
    cg.fetch(op.gate8, p.row, p.col, p.n);
    cu.fetch(op.up8, p.row, p.col, p.n);
    settle8(rd, p.col, p.n);
    cg.settle(p.col, p.n);
    cu.settle(p.col, p.n);
    float g[8], u[8], dg[8], du[8];
    cg.get(g);
    cu.get(u);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float d = rd.get(i), s = sigmoid(g[i]), act = g[i] * s;
      dg[i] = d * u[i] * fmaf(act, 1.f - s, s);   // s (1 + g (1 - s))
      du[i] = d * act;
      g[i] = act * u[i];
    }
    Vec8<T>::store(static_cast<T*>(op.dgate) + p.row * op.ld_dgate + p.col, p.n, dg);
    Vec8<T>::store(static_cast<T*>(op.dup) + p.row * op.ld_dup + p.col, p.n, du);
    if (op.a8.codes) act8_put(op.a8, p.row, p.col, p.n, g);
  });
}

namespace {
// threads of a grid stay below 2^32
constexpr int64_t kMaxGrid = int64_t(1) << 23;

template <class K, class... A>
int go(K k, int64_t rows, int64_t cols, void* stream, A... a) {
  const int64_t vpr = (cols + 31) / 32 * 4;
  const int64_t blocks = (rows * vpr + kThreads - 1) / kThreads;
  hipLaunchKernelGGL(k, dim3(static_cast<unsigned>(blocks < kMaxGrid ? blocks : kMaxGrid)), dim3(kThreads), 0,
                     static_cast<hipStream_t>(stream), blocks, a...);
  return static_cast<int>(hipGetLastError());
}
}  // namespace

int launch_act8_pack(const void* x, int64_t ld_x, int32_t dtype, int64_t rows, int64_t cols,
                     const muon_act8_t& out, void* stream) {
  const int c = static_cast<int>(cols);
  if (dtype == MUON_BF16)
    return go(k_act8_pack<uint16_t>, rows, cols, stream, static_cast<const uint16_t*>(x), ld_x, rows, c, out);
  return go(k_act8_pack<float>, rows, cols, stream, static_cast<const float*>(x), ld_x, rows, c, out);
}

int launch_act8_unpack(const muon_act8_t& in, int64_t rows, int64_t cols, void* out, int64_t ld_out,
                       int32_t dtype, void* stream) {
  const int c = static_cast<int>(cols);
  if (dtype == MUON_BF16)
    return go(k_act8_unpack<uint16_t>, rows, cols, stream, in, rows, c, static_cast<uint16_t*>(out), ld_out);
  return go(k_act8_unpack<float>, rows, cols, stream, in, rows, c, static_cast<float*>(out), ld_out);
}

int launch_swiglu(const muon_swiglu_t& op, void* stream) {
  return op.dtype == MUON_BF16 ? go(k_swiglu<uint16_t>, op.rows, op.cols, stream, op)
                               : go(k_swiglu<float>, op.rows, op.cols, stream, op);
}

int launch_swiglu_grad(const muon_swiglu_grad_t& op, void* stream) {
  return op.dtype == MUON_BF16 ? go(k_swiglu_grad<uint16_t>, op.rows, op.cols, stream, op)
                               : go(k_swiglu_grad<float>, op.rows, op.cols, stream, op);
}

}  // namespace muon
