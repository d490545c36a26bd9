// Embedding lookup and its gradient (gfx950).
//
// The gradient adds the rows of dy by id without atomics: the tokens are sorted
// by id with a stable radix sort (8-bit digits, least significant first), so
// each row of the table finds its tokens side by side and in their own order,
// and its sum does not depend on scheduling.  Tokens whose id is outside the
// table take the key `vocab` and end up past every row.
#include <algorithm>

#include "muon_act8.h"
#include "muon_ops.h"

namespace muon {

namespace {

constexpr int kDigits = 256;
constexpr int kSortThreads = 1024;
constexpr int kSortWaves = kSortThreads / 64;
constexpr int kPerWave = 256;                       // tokens of a wave per step
constexpr int kStep = kSortWaves * kPerWave;        // tokens of a block per step
constexpr int kRowThreads = 256;

__device__ __forceinline__ int64_t load_id(const void* ids, int id_bytes, int64_t i) {
  return id_bytes == 8 ? gld<int64_t>(static_cast<const char*>(ids) + 8 * i)
                       : static_cast<int64_t>(gld<int32_t>(static_cast<const char*>(ids) + 4 * i));
}

// ------------------------------------------------------------------ lookup ----
// One lane per 8 columns; rows of 8-vectors laid end to end.
template <class S, class T>
__global__ __launch_bounds__(kRowThreads) void k_embed(muon_embed_t op, int64_t blocks) {
  const uint32_t vpr = static_cast<uint32_t>((op.cols + 7) >> 3);
  for (int64_t b = blockIdx.x; b < blocks; b += gridDim.x) {
    const uint64_t first = static_cast<uint64_t>(b) * kRowThreads;
    const uint64_t row0 = first / vpr;
    const uint32_t u = static_cast<uint32_t>(first - row0 * vpr) + threadIdx.x;
    const uint32_t dr = u / vpr;
    const int64_t row = static_cast<int64_t>(row0 + dr);
    if (row >= op.tokens) continue;
    const int c = static_cast<int>(u - dr * vpr) * 8, n = static_cast<int>(op.cols) - c;
    const int64_t id = load_id(op.ids, op.id_bytes, row);
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 0.f;
    if (id >= 0 && id < op.vocab) {
      Vec8<S> raw;
      load8(raw, static_cast<const S*>(op.table) + id * op.ld_table + c, n);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = raw.get(i) * op.scale;
    }
    Vec8<T>::store(static_cast<T*>(op.out) + row * op.ld_out + c, n, v);
  }
}

// -------------------------------------------------------------------- sort ----
struct SortArgs {
  const void* ids;
  int id_bytes;
  int64_t tokens, vocab;
  int64_t block_tokens;
  int shift;
  const uint32_t* keys_in;    // null in the first pass: from the ids
  const uint32_t* toks_in;
  uint32_t* keys_out;
  uint32_t* toks_out;
  uint32_t* count;            // [block][digit]
};

__device__ __forceinline__ uint32_t key_of(const SortArgs& a, int64_t i) {
  if (a.keys_in) return gld<uint32_t>(a.keys_in + i);
  const int64_t id = load_id(a.ids, a.id_bytes, i);
  return static_cast<uint32_t>(id >= 0 && id < a.vocab ? id : a.vocab);
}

// Tokens of each digit in each block's share.
__global__ __launch_bounds__(kSortThreads) void k_embed_count(SortArgs a) {
  __shared__ uint32_t hist[kDigits];
  if (threadIdx.x < kDigits) hist[threadIdx.x] = 0;
  __syncthreads();
  const int64_t begin = blockIdx.x * a.block_tokens;
  const int64_t end = begin + a.block_tokens < a.tokens ? begin + a.block_tokens : a.tokens;
  for (int64_t i = begin + threadIdx.x; i < end; i += kSortThreads)
    atomicAdd(&hist[(key_of(a, i) >> a.shift) & (kDigits - 1)], 1u);
  __syncthreads();
  if (threadIdx.x < kDigits) gst<uint32_t>(a.count + blockIdx.x * kDigits + threadIdx.x, hist[threadIdx.x]);
}

// Moves each block's share to its place.  A digit's tokens of earlier blocks
// come first, then those of earlier waves, then in order within the wave: the
// lanes with one digit find each other by a ballot per digit bit.
__global__ __launch_bounds__(kSortThreads) void k_embed_scatter(SortArgs a) {
  __shared__ uint32_t base[kDigits];                // next place of each digit
  __shared__ uint32_t part[kDigits];
  __shared__ uint32_t wcnt[kSortWaves][kDigits];
  const int t = static_cast<int>(threadIdx.x), lane = t & 63, w = t >> 6;
  uint32_t before = 0, total = 0;
  if (t < kDigits) {
    for (unsigned b = 0; b < gridDim.x; ++b) {
      const uint32_t n = gld<uint32_t>(a.count + b * kDigits + t);
      if (b < blockIdx.x) before += n;
      total += n;
    }
    part[t] = total;
  }
  __syncthreads();
  for (int o = 1; o < kDigits; o <<= 1) {           // inclusive scan over the digits
    uint32_t v = 0;
    if (t < kDigits && t >= o) v = part[t - o];
    __syncthreads();
    if (t < kDigits) part[t] += v;
    __syncthreads();
  }
  if (t < kDigits) base[t] = part[t] - total + before;
  const int64_t begin = blockIdx.x * a.block_tokens;
  const int64_t end = begin + a.block_tokens < a.tokens ? begin + a.block_tokens : a.tokens;
  for (int64_t at = begin; at < end; at += kStep) {
    for (int i = t; i < kSortWaves * kDigits; i += kSortThreads) (&wcnt[0][0])[i] = 0;
    __syncthreads();
    uint32_t key[kPerWave / 64], tok[kPerWave / 64], rank[kPerWave / 64];
#pragma unroll
    for (int r = 0; r < kPerWave / 64; ++r) {
      const int64_t i = at + w * kPerWave + r * 64 + lane;
      key[r] = i < end ? key_of(a, i) : 0u;
      tok[r] = i < end ? (a.toks_in ? gld<uint32_t>(a.toks_in + i) : static_cast<uint32_t>(i)) : 0u;
    }
#pragma unroll
    for (int r = 0; r < kPerWave / 64; ++r) {
      const bool valid = at + w * kPerWave + r * 64 + lane < end;
      const uint32_t d = (key[r] >> a.shift) & (kDigits - 1);
      uint64_t same = __ballot(valid);
#pragma unroll
      for (int bit = 0; bit < 8; ++bit) {
        const uint64_t on = __ballot((d >> bit) & 1);
        same &= (d >> bit) & 1 ? on : ~on;
      }
      const uint32_t seen = wcnt[w][d];
      rank[r] = seen + __popcll(same & ((uint64_t(1) << lane) - 1));
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
      if (valid && (same >> lane) == 1) wcnt[w][d] = rank[r] + 1;   // the digit's last lane
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
    }
    __syncthreads();
    if (t < kDigits) {
      uint32_t run = base[t];
#pragma unroll
      for (int k = 0; k < kSortWaves; ++k) {
        const uint32_t n = wcnt[k][t];
        wcnt[k][t] = run;
        run += n;
      }
      base[t] = run;
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kPerWave / 64; ++r) {
      if (at + w * kPerWave + r * 64 + lane < end) {
        const uint32_t p = wcnt[w][(key[r] >> a.shift) & (kDigits - 1)] + rank[r];
        gst<uint32_t>(a.keys_out + p, key[r]);
        gst<uint32_t>(a.toks_out + p, tok[r]);
      }
    }
    __syncthreads();
  }
}

// -------------------------------------------------------------------- rows ----
// First place whose key is >= v, by a whole wave: 64 probes a step.  (c probes
// below v: the place is past the c-th and at most at the next one.)
__device__ __forceinline__ uint32_t lower_bound(const uint32_t* keys, uint32_t n, uint32_t v, int lane) {
  uint32_t lo = 0, hi = n;
  while (lo < hi) {
    const uint32_t step = (hi - lo + 63) >> 6;
    const uint32_t p = lo + (lane + 1) * step - 1;
    bool less = false;
    if (p < hi) less = gld<uint32_t>(keys + p) < v;
    lo += static_cast<uint32_t>(__popcll(__ballot(less))) * step;
    hi = min(hi, lo + step - 1);
  }
  return lo;
}

// One wave per row of the table.
template <class S, class T>
__global__ __launch_bounds__(kRowThreads) void k_embed_rows(muon_embed_grad_t op, const uint32_t* keys, const uint32_t* toks) {
  const int lane = threadIdx.x & 63;
  const int cols = static_cast<int>(op.cols);
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6); row < op.vocab;
       row += static_cast<int64_t>(gridDim.x) * 4) {
    const uint32_t v = static_cast<uint32_t>(row);
    const uint32_t first = lower_bound(keys, static_cast<uint32_t>(op.tokens), v, lane);
    for (int c = lane * 8; c < cols; c += 512) {
      const int n = cols - c;
      float s[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) s[i] = 0.f;
      for (int64_t i = first; i < op.tokens && gld<uint32_t>(keys + i) == v; ++i) {
        Vec8<S> raw;
        load8(raw, static_cast<const S*>(op.dy) + static_cast<int64_t>(gld<uint32_t>(toks + i)) * op.ld_dy + c, n);
#pragma unroll
        for (int k = 0; k < 8; ++k) s[k] += raw.get(k);
      }
      T* out = static_cast<T*>(op.dtable) + row * op.ld_dtable + c;
      Vec8<T> old;
      if (op.accumulate) load8(old, out, n);
#pragma unroll
      for (int i = 0; i < 8; ++i) s[i] = op.accumulate ? fmaf(op.scale, s[i], old.get(i)) : op.scale * s[i];
      Vec8<T>::store(out, n, s);
    }
  }
}

// threads of a grid stay below 2^32
constexpr int64_t kMaxGrid = int64_t(1) << 23;
size_t up256(size_t x) { return (x + 255) / 256 * 256; }

SortArgs sort_args(const muon_embed_grad_t& op, const EmbedSortPlan& p, int pass, char* ws) {
  SortArgs a;
  a.ids = op.ids;
  a.id_bytes = op.id_bytes;
  a.tokens = op.tokens;
  a.vocab = op.vocab;
  a.block_tokens = p.block_tokens;
  a.shift = 8 * pass;
  const int in = (pass + 1) & 1, out = pass & 1;
  a.keys_in = pass ? reinterpret_cast<const uint32_t*>(ws + p.keys_off[in]) : nullptr;
  a.toks_in = pass ? reinterpret_cast<const uint32_t*>(ws + p.toks_off[in]) : nullptr;
  a.keys_out = reinterpret_cast<uint32_t*>(ws + p.keys_off[out]);
  a.toks_out = reinterpret_cast<uint32_t*>(ws + p.toks_off[out]);
  a.count = reinterpret_cast<uint32_t*>(ws + p.count_off);
  return a;
}

// f.operator()<input type, output type>()
template <class F>
int by_types(int32_t in, int32_t out, F&& f) {
  if (in == MUON_BF16) return out == MUON_BF16 ? f(uint16_t{}, uint16_t{}) : f(uint16_t{}, float{});
  return out == MUON_BF16 ? f(float{}, uint16_t{}) : f(float{}, float{});
}

}  // namespace

EmbedSortPlan embed_sort_plan(int64_t tokens, int64_t vocab, int64_t cols) {
  EmbedSortPlan p;
  p.passes = 0;
  for (int64_t top = vocab; top > 0; top >>= 8) ++p.passes;
  // at most 256 blocks, whole steps each
  p.block_tokens = kStep * std::max<int64_t>(1, (tokens + kStep * 256 - 1) / (kStep * 256));
  p.blocks = (tokens + p.block_tokens - 1) / p.block_tokens;
  size_t off = 0;
  for (int k = 0; k < 2; ++k) {
    p.keys_off[k] = off;
    off = up256(off + static_cast<size_t>(tokens) * 4);
    p.toks_off[k] = off;
    off = up256(off + static_cast<size_t>(tokens) * 4);
  }
  p.count_off = off;
  off = up256(off + static_cast<size_t>(p.blocks) * kDigits * 4);
  p.bytes = off;
  (void)cols;
  return p;
}

int launch_embed(const muon_embed_t& op, void* stream) {
  const int64_t vpr = (op.cols + 7) / 8, blocks = (op.tokens * vpr + kRowThreads - 1) / kRowThreads;
  return by_types(op.table_dtype, op.out_dtype, [&](auto s, auto t) {
    hipLaunchKernelGGL((k_embed<decltype(s), decltype(t)>), dim3(static_cast<unsigned>(std::min(blocks, kMaxGrid))),
                       dim3(kRowThreads), 0, static_cast<hipStream_t>(stream), op, blocks);
    return static_cast<int>(hipGetLastError());
  });
}

int launch_embed_count(const muon_embed_grad_t& op, const EmbedSortPlan& p, int pass, char* ws, void* stream) {
  hipLaunchKernelGGL(k_embed_count, dim3(static_cast<unsigned>(p.blocks)), dim3(kSortThreads), 0,
                     static_cast<hipStream_t>(stream), sort_args(op, p, pass, ws));
  return static_cast<int>(hipGetLastError());
}

int launch_embed_scatter(const muon_embed_grad_t& op, const EmbedSortPlan& p, int pass, char* ws, void* stream) {
  hipLaunchKernelGGL(k_embed_scatter, dim3(static_cast<unsigned>(p.blocks)), dim3(kSortThreads), 0,
                     static_cast<hipStream_t>(stream), sort_args(op, p, pass, ws));
  return static_cast<int>(hipGetLastError());
}

int launch_embed_rows(const muon_embed_grad_t& op, const EmbedSortPlan& p, char* ws, void* stream) {
  const int last = (p.passes - 1) & 1;
  const uint32_t* keys = reinterpret_cast<const uint32_t*>(ws + p.keys_off[last]);
  const uint32_t* toks = reinterpret_cast<const uint32_t*>(ws + p.toks_off[last]);
  const int64_t blocks = (op.vocab + 3) / 4;
  return by_types(op.dy_dtype, op.table_dtype, [&](auto s, auto t) {
    hipLaunchKernelGGL((k_embed_rows<decltype(s), decltype(t)>), dim3(static_cast<unsigned>(std::min(blocks, kMaxGrid))),
                       dim3(kRowThreads), 0, static_cast<hipStream_t>(stream), op, keys, toks);
    return static_cast<int>(hipGetLastError());
  });
}

}  // namespace muon
