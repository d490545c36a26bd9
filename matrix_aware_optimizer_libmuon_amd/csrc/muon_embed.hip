// Embedding lookup and its gradient (gfx950).
//
// The gradient adds the rows of dy by id without atomics, so that its sums do
// not depend on scheduling.  The tokens are sorted by id, which puts each row's
// side by side and in their own order: up to 32768 of them, in tables of up to
// 261631 rows, in one launch (k_embed_buckets); else with a stable radix sort (9-bit
// digits, least significant first: two passes up to 262143 rows) and k_starts, which
// notes where each row's begin.  Tokens whose id is outside the table take the key
// `vocab`, which is no row's.
//
// Ids are as frequent as words: a few have thousands of tokens, most none.
//   Rows of up to kRun tokens (and empty ones, which are written as zeros unless the
//   sums are added to what is there) are a wave's or a block's, one each (4 or 8 each
//   were 4 and 8 % slower: too few independent loads).
//   Longer runs are cut where the sorted order passes a multiple of kRun: each
//   piece is summed into the workspace (by blocks of the same launch, k_sums), and
//   k_join adds a run's pieces in order.  A piece lies in one chunk of kRun
//   places; a chunk can hold two of them, the end of one run and the beginning of
//   another.
// Up to kDirect tokens none of that is needed: each wave of k_direct finds its
// rows' tokens by comparing all ids; it walks the whole table, also when it adds to
// what is there and leaves the other rows alone.
//
// Bound by memory: dy is read once, the table's gradient written once.
#include <algorithm>

#include "muon_act8.h"
#include "muon_ops.h"

namespace muon {

namespace {

constexpr int kDigitBits = 9;
constexpr int kDigits = 1 << kDigitBits;
constexpr int kSortThreads = 1024;                  // tokens of a block per step
constexpr int kSortWaves = kSortThreads / 64;
constexpr int kRowThreads = 256;
constexpr int kRun = 32;                            // longest run that one wave adds up (at most 64)
constexpr int kDirect = 256;                        // tokens that are not sorted
constexpr int kRowsEach = 4;                        // rows of a wave (or block) of k_direct

__device__ __forceinline__ int64_t load_id(const void* ids, int id_bytes, int64_t i) {
  return id_bytes == 8 ? gld<int64_t>(static_cast<const char*>(ids) + 8 * i)
                       : static_cast<int64_t>(gld<int32_t>(static_cast<const char*>(ids) + 4 * i));
}

// ------------------------------------------------------------------ lookup ----
// Rows of 8-column vectors laid end to end, kVecs of them 256 apart for each
// thread: the ids, then the rows, are loaded for all of them at once (one each:
// 43 us, two: 37.2, four: 37.7 for 16384 tokens of 4096 bf16).
constexpr int kVecs = 2;
template <class S, class T>
__global__ __launch_bounds__(kRowThreads) void k_embed(muon_embed_t op, int64_t blocks) {
  const uint32_t vpr = static_cast<uint32_t>((op.cols + 7) >> 3);
  const int cols = static_cast<int>(op.cols);
  for (int64_t b = blockIdx.x; b < blocks; b += gridDim.x) {
    const uint64_t first = static_cast<uint64_t>(b) * (kRowThreads * kVecs);
    const uint64_t row0 = first / vpr;
    const uint32_t u0 = static_cast<uint32_t>(first - row0 * vpr) + threadIdx.x;
    int64_t row[kVecs], id[kVecs];
    int c[kVecs];
#pragma unroll
    for (int k = 0; k < kVecs; ++k) {
      const uint32_t u = u0 + k * kRowThreads, dr = u / vpr;
      row[k] = static_cast<int64_t>(row0 + dr);
      c[k] = static_cast<int>(u - dr * vpr) * 8;
      id[k] = row[k] < op.tokens ? load_id(op.ids, op.id_bytes, row[k]) : -1;
    }
    Vec8<S> raw[kVecs];
#pragma unroll
    for (int k = 0; k < kVecs; ++k) {
      const bool in = id[k] >= 0 && id[k] < op.vocab;
      fetch8(raw[k], static_cast<const S*>(op.table) + (in ? id[k] : 0) * op.ld_table + c[k], c[k], in ? cols - c[k] : 0);
    }
#pragma unroll
    for (int k = 0; k < kVecs; ++k) {
      if (row[k] >= op.tokens) continue;
      settle8(raw[k], c[k], id[k] >= 0 && id[k] < op.vocab ? cols - c[k] : 0);
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = raw[k].get(i) * op.scale;
      Vec8<T>::store(static_cast<T*>(op.out) + row[k] * op.ld_out + c[k], cols - c[k], v);
    }
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

__device__ __forceinline__ uint32_t key_of(const void* ids, int id_bytes, int64_t vocab, int64_t i) {
  const uint64_t id = static_cast<uint64_t>(load_id(ids, id_bytes, i));   // negative: past any table
  return static_cast<uint32_t>(id >> 32) == 0 && static_cast<uint32_t>(id) < static_cast<uint32_t>(vocab)
             ? static_cast<uint32_t>(id) : static_cast<uint32_t>(vocab);
}
__device__ __forceinline__ uint32_t key_in(const SortArgs& a, int64_t i) {
  return a.keys_in ? gld<uint32_t>(a.keys_in + i) : key_of(a.ids, a.id_bytes, a.vocab, i);
}

// The wave's valid lanes with this lane's digit, by a ballot per digit bit.
__device__ __forceinline__ uint64_t same_digit(bool valid, uint32_t d) {
  uint64_t same = __ballot(valid);
#pragma unroll
  for (int bit = 0; bit < kDigitBits; ++bit) {
    const uint64_t on = __ballot((d >> bit) & 1);
    same &= (d >> bit) & 1 ? on : ~on;
  }
  return same;
}

// Whether that is all of them (lane 0 is valid if any is).
__device__ __forceinline__ bool one_digit(bool valid, uint32_t d) {
  return __ballot(valid && d != static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(d))) == 0;
}

// v of this lane and the lanes before it.
__device__ __forceinline__ uint32_t wave_scan(uint32_t v, int lane) {
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const uint32_t u = __shfl_up(v, o, 64);
    v += lane >= o ? u : 0u;
  }
  return v;
}

// Tokens of each digit in each block's share.
__global__ __launch_bounds__(kSortThreads) void k_embed_count(SortArgs a) {
  __shared__ uint32_t hist[kDigits];
  if (threadIdx.x < kDigits) hist[threadIdx.x] = 0;
  __syncthreads();
  const int64_t begin = blockIdx.x * a.block_tokens;
  const int64_t end = min(begin + a.block_tokens, a.tokens);
  for (int64_t i = begin + threadIdx.x; i < end; i += kSortThreads)
    atomicAdd(&hist[(key_in(a, i) >> a.shift) & (kDigits - 1)], 1u);
  __syncthreads();
  if (threadIdx.x < kDigits) gst<uint32_t>(a.count + blockIdx.x * kDigits + threadIdx.x, hist[threadIdx.x]);
}

// Moves each block's share to its place.  A digit's tokens of earlier blocks
// come first, then those of earlier waves, then in order within the wave.
__global__ __launch_bounds__(kSortThreads) void k_embed_scatter(SortArgs a) {
  __shared__ uint32_t base[kDigits];                // next place of each digit
  __shared__ uint32_t wcnt[kSortWaves][kDigits];    // a step's tokens by wave, then their places
  __shared__ uint32_t half[2][kDigits], wsum[kSortWaves];
  const int t = static_cast<int>(threadIdx.x), lane = t & 63, w = t >> 6;
  // tokens of digit d in the blocks before this one, and in all: two halves of
  // the threads take every other block
  {
    const int d = t & (kDigits - 1), h = t / kDigits;
    uint32_t before = 0, total = 0;
#pragma unroll 4
    for (unsigned b = h; b < gridDim.x; b += 2) {
      const uint32_t n = gld<uint32_t>(a.count + b * kDigits + d);
      before += b < blockIdx.x ? n : 0u;
      total += n;
    }
    half[h][d] = total;
    if (h == 1) base[d] = before;
    __syncthreads();
    uint32_t sum = 0;
    if (t < kDigits) {
      sum = half[0][t] + half[1][t];
      before += base[t];
    }
    // exclusive scan of the totals over the digits
    const uint32_t scan = wave_scan(sum, lane);
    if (lane == 63) wsum[w] = scan;
    __syncthreads();
    if (t < kDigits) {
      uint32_t first = scan - sum;
      for (int k = 0; k < w; ++k) first += wsum[k];
      base[t] = first + before;
    }
  }
  const int64_t begin = blockIdx.x * a.block_tokens;
  const int64_t end = min(begin + a.block_tokens, a.tokens);
  for (int64_t at = begin; at < end; at += kSortThreads) {
#pragma unroll
    for (int i = t; i < kSortWaves * kDigits; i += kSortThreads) (&wcnt[0][0])[i] = 0;
    __syncthreads();
    const int64_t i = at + t;
    const bool valid = i < end;
    uint32_t key = 0, tok = 0;
    if (valid) {
      key = key_in(a, i);
      tok = a.toks_in ? gld<uint32_t>(a.toks_in + i) : static_cast<uint32_t>(i);
    }
    const uint32_t d = (key >> a.shift) & (kDigits - 1);
    const uint64_t same = same_digit(valid, d);
    const uint32_t rank = __popcll(same & ((uint64_t(1) << lane) - 1));
    if (valid && (same >> lane) == 1) wcnt[w][d] = rank + 1;   // the digit's last lane
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
    if (valid) {
      const uint32_t p = wcnt[w][d] + rank;
      gst<uint32_t>(a.keys_out + p, key);
      gst<uint32_t>(a.toks_out + p, tok);
    }
    __syncthreads();
  }
}

// The whole sort in one launch: block b takes the ids whose low bits are b.  It
// goes over all ids once, noting its own and counting those of lower blocks, so
// that it knows where its places begin, and orders its own by their high bits.
// A row's tokens are side by side all the same, and each block writes the starts
// of its rows, [block][high bits], as it has them.
//   Against one block alone (up to 4096 tokens) or the launches above and k_starts:
// 1000 tokens 6.3 for 10.2 us, 4000 6.9 for 16.4, 10010 8.5 for 21.6, 32768 13.0 for
// 27.3.  An id that has them all is the worst case, one block's work: the sort then
// costs 7 us more than by digits at 32768 tokens (and would cost more with more).
constexpr int64_t kBucketTokens = 32 * kSortThreads;   // 32 loads of 64 tokens for a wave: 64 lanes hold their masks
constexpr uint32_t kHighs = kDigits - 1;               // (what LDS has room for)
constexpr int kLogBuckets = 8;                         // a block to a CU; for larger tables twice as many
constexpr int64_t kBucketVocab = (int64_t(1) << (kLogBuckets + 1)) * kHighs - 1;
template <int ID_BYTES>
__global__ __launch_bounds__(kSortThreads) void k_embed_buckets(SortArgs a, int log_buckets, uint32_t highs, uint32_t* start) {
  __shared__ uint16_t list[kBucketTokens], high[kBucketTokens];   // the block's tokens in order, their high bits
  __shared__ uint32_t wcnt[kSortWaves * kHighs];    // [wave][high]: counts, then places
  __shared__ uint32_t wsum[kSortWaves];
  const int t = static_cast<int>(threadIdx.x), lane = t & 63, w = __builtin_amdgcn_readfirstlane(t >> 6);
  const int n = static_cast<int>(a.tokens);
  const uint32_t low = (1u << log_buckets) - 1;
  const uint64_t below = (uint64_t(1) << lane) - 1;
  for (uint32_t i = t; i < kSortWaves * highs; i += kSortThreads) wcnt[i] = 0;
  // the ids, each wave's share side by side: lanes 2 e and 2 e + 1 keep the mask of
  // load e's tokens that are the block's
  const int loads = (n + kSortThreads - 1) / kSortThreads, begin = w * 64 * loads;
  uint32_t hits = 0, less = 0;
  auto note = [&](uint32_t key, bool valid, int e) __attribute__((always_inline)) {
    const uint32_t b = key & low;
    const uint64_t m = __ballot(valid && b == blockIdx.x);
    less += __popcll(__ballot(valid && b < blockIdx.x));
    if (lane >> 1 == e) hits = static_cast<uint32_t>(lane & 1 ? m >> 32 : m);
  };
  const int full = min(loads, max(0, n - begin) / 64);   // then a short one, if any
  constexpr int kAtOnce = 8, kGather = 4;
  for (int e = 0; e < full; e += kAtOnce) {
    uint32_t key[kAtOnce];
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) key[k] = key_of(a.ids, ID_BYTES, a.vocab, begin + 64 * min(e + k, full - 1) + lane);
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k)
      if (k == 0 || e + k < full) note(key[k], true, e + k);
  }
  if (full < loads && begin + 64 * full < n) {
    const int i = begin + 64 * full + lane;
    note(key_of(a.ids, ID_BYTES, a.vocab, min(i, n - 1)), i < n, full);
  }
  uint32_t before = wave_scan(__popc(hits), lane);  // tokens of this lane and the lanes before it
  if (lane == 63) wsum[w] = before << 16 | less;    // (2048 at most)
  before -= __popc(hits);
  __syncthreads();
  uint32_t base = 0, count = 0;                     // the block's first place, its tokens
#pragma unroll
  for (int k = 0; k < kSortWaves; ++k) {
    const uint32_t v = wsum[k];
    base += v & 0xffffu;
    before += k < w ? v >> 16 : 0u;
    count += v >> 16;
  }
  for (; hits; hits &= hits - 1) list[before++] = static_cast<uint16_t>(begin + 32 * lane + __builtin_ctz(hits));
  __syncthreads();
  // the list by high bits, each wave's share of it side by side: counted, then placed
  const uint32_t each = (count + kSortThreads - 1) / kSortThreads, first = w * 64 * each + lane;
  uint32_t* const mine = wcnt + w * highs;
  for (uint32_t e = 0; e < each; e += kGather) {
    uint32_t d[kGather];
#pragma unroll
    for (uint32_t k = 0; k < kGather; ++k)
      d[k] = key_of(a.ids, ID_BYTES, a.vocab, list[min(first + 64 * (e + k), count - 1)]) >> log_buckets;
#pragma unroll
    for (uint32_t k = 0; k < kGather; ++k) {
      if (k > 0 && e + k >= each) break;
      const uint32_t i = first + 64 * (e + k);
      const uint64_t valid = __ballot(i < count);
      const bool one = one_digit(i < count, d[k]);  // frequent ids: no atomics in one place
      if (i < count) {
        high[i] = static_cast<uint16_t>(d[k]);
        if (!one) atomicAdd(&mine[d[k]], 1u);
        else if ((valid >> lane) == 1) atomicAdd(&mine[d[k]], static_cast<uint32_t>(__popcll(valid)));
      }
    }
  }
  __syncthreads();
  uint32_t cnt[kSortWaves], sum = 0;
  if (t < static_cast<int>(highs))
#pragma unroll
    for (int k = 0; k < kSortWaves; ++k) sum += cnt[k] = wcnt[k * highs + t];
  uint32_t run = wave_scan(sum, lane);
  if (lane == 63) wsum[w] = run;
  __syncthreads();
  if (t < static_cast<int>(highs)) {
    run += base - sum;
#pragma unroll
    for (int k = 0; k < kDigits / 64; ++k) run += k < w ? wsum[k] : 0u;
    gst<uint32_t>(start + blockIdx.x * highs + t, run);
#pragma unroll
    for (int k = 0; k < kSortWaves; ++k) {
      wcnt[k * highs + t] = run;
      run += cnt[k];
    }
  }
  if (blockIdx.x == gridDim.x - 1 && t == 0) gst<uint32_t>(start + gridDim.x * highs, static_cast<uint32_t>(n));
  __syncthreads();
  for (uint32_t e = 0; e < each; ++e) {
    const uint32_t i = first + 64 * e;
    const bool valid = i < count;
    const uint32_t d = valid ? high[i] : 0u;
    const uint64_t same = one_digit(valid, d) ? __ballot(valid) : same_digit(valid, d);
    const uint32_t p = mine[d] + __popcll(same & below);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    if (valid) {
      if ((same >> lane) == 1) mine[d] = p + 1;     // the digit's last lane
      gst<uint32_t>(a.keys_out + p, d << log_buckets | blockIdx.x);
      gst<uint32_t>(a.toks_out + p, static_cast<uint32_t>(list[i]));
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  }
}

// start[v] = first place whose key is >= v, for v = 0 .. vocab.
__global__ __launch_bounds__(kRowThreads) void k_starts(const uint32_t* keys, uint32_t tokens, uint32_t vocab, uint32_t* start) {
  const uint32_t v = blockIdx.x * kRowThreads + threadIdx.x;
  if (v > vocab) return;
  uint32_t lo = 0, hi = tokens;
  while (lo < hi) {
    const uint32_t mid = (lo + hi) >> 1;
    if (gld<uint32_t>(keys + mid) < v) lo = mid + 1;
    else hi = mid;
  }
  gst<uint32_t>(start + v, lo);
}

// ------------------------------------------------------------------ sums ----
// s += dy[token] for the tokens held by lanes first .. first + n - 1 of the wave
// (all lanes active), in order; this thread's columns c .. c + 7.
template <class S>
__device__ __forceinline__ void add_rows(const muon_embed_grad_t& op, uint32_t held, int first, int n, int c, float (&s)[8]) {
  const int valid = static_cast<int>(op.cols) - c;
  const S* dy = static_cast<const S*>(op.dy) + c;
  auto row = [&](int i) { return dy + static_cast<int64_t>(static_cast<uint32_t>(__builtin_amdgcn_readlane(held, i))) * op.ld_dy; };
  auto batch = [&](auto size, int i) __attribute__((always_inline)) {
    constexpr int N = decltype(size)::value;
    Vec8<S> v[N];
#pragma unroll
    for (int k = 0; k < N; ++k) fetch8(v[k], row(i + k), c, valid);
#pragma unroll
    for (int k = 0; k < N; ++k) {
      settle8(v[k], c, valid);
#pragma unroll
      for (int j = 0; j < 8; ++j) s[j] += v[k].get(j);
    }
  };
  int i = first;
  const int end = first + n;
  for (; i + 8 <= end; i += 8) batch(std::integral_constant<int, 8>{}, i);
  if (i + 4 <= end) {
    batch(std::integral_constant<int, 4>{}, i);
    i += 4;
  }
  if (i + 2 <= end) {
    batch(std::integral_constant<int, 2>{}, i);
    i += 2;
  }
  if (i < end) batch(std::integral_constant<int, 1>{}, i);
}

// dtable[row] (+)= scale s, columns c .. c + 7.
template <class T>
__device__ __forceinline__ void put_row(const muon_embed_grad_t& op, int64_t row, int c, float (&s)[8]) {
  const int n = static_cast<int>(op.cols) - c;
  T* out = static_cast<T*>(op.dtable) + row * op.ld_dtable + c;
  Vec8<T> old;
  if (op.accumulate) load8(old, static_cast<const T*>(out), c, n);
#pragma unroll
  for (int j = 0; j < 8; ++j) s[j] = op.accumulate ? fmaf(op.scale, s[j], old.get(j)) : op.scale * s[j];
  Vec8<T>::store(out, n, s);
}

// Few tokens: kRowsEach rows for each group of TPR threads (a wave, or the
// block), whose tokens are found by comparing all ids.
template <class S, class T, int TPR>
__global__ __launch_bounds__(kRowThreads) void k_direct(muon_embed_grad_t op) {
  const int lane = threadIdx.x & 63;
  // uniform over a wave: taken from its first lane
  const int group = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) / TPR);
  const int t = static_cast<int>(threadIdx.x) % TPR;
  const int cols = static_cast<int>(op.cols);
  uint32_t key[kDirect / 64];
#pragma unroll
  for (int q = 0; q < kDirect / 64; ++q) {
    const int64_t i = q * 64 + lane;
    key[q] = i < op.tokens ? key_of(op.ids, op.id_bytes, op.vocab, i) : 0xffffffffu;
  }
  for (int64_t row0 = (static_cast<int64_t>(blockIdx.x) * (kRowThreads / TPR) + group) * kRowsEach; row0 < op.vocab;
       row0 += static_cast<int64_t>(gridDim.x) * (kRowThreads / TPR) * kRowsEach)
    for (int r = 0; r < kRowsEach && row0 + r < op.vocab; ++r) {
      if (op.accumulate) {   // a row without tokens is neither read nor written
        bool mine = false;
#pragma unroll
        for (int q = 0; q < kDirect / 64; ++q) mine |= key[q] == static_cast<uint32_t>(row0 + r);
        if (!__ballot(mine)) continue;
      }
      for (int c0 = 0; c0 < cols; c0 += TPR * 8) {
        const int c = c0 + t * 8;
        float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int q = 0; q < kDirect / 64; ++q) {
          const bool mine = key[q] == static_cast<uint32_t>(row0 + r);
          const uint64_t m = __ballot(mine);
          if (!m) continue;
          // the row's tokens, in order, to the first lanes; the others' go past them
          const int n = __popcll(m), before = __popcll(m & ((uint64_t(1) << lane) - 1));
          const int to = mine ? before : n + lane - before;
          add_rows<S>(op, static_cast<uint32_t>(__builtin_amdgcn_ds_permute(4 * to, q * 64 + lane)), 0, n, c, s);
        }
        put_row<T>(op, row0 + r, c, s);
      }
    }
}

// What the sums of sorted tokens work on.
struct Sorted {
  const uint32_t* keys;
  const uint32_t* toks;
  const uint32_t* start;        // [low bits of the row][high bits]
  int log_buckets;              // low bits (0: in the order of the rows)
  uint32_t highs;
  float* pieces;                // [chunk][left, right][cols]
  int64_t chunks;
  unsigned piece_blocks;        // the launch's first blocks: pieces, the others: rows
};
// Where a row's tokens begin and end in the sorted order.
__device__ __forceinline__ void run_of(const Sorted& a, uint32_t row, uint32_t& begin, uint32_t& end) {
  const uint32_t* p = a.start + ((row & ((1u << a.log_buckets) - 1)) * a.highs + (row >> a.log_buckets));
  begin = gld<uint32_t>(p);
  end = gld<uint32_t>(p + 1);
}

// The long runs that touch chunk `chunk` of the sorted order, one place per
// lane: `left`, lanes of a run that began in an earlier chunk, and `right`, lanes
// of one that begins here (it goes on in the next chunk).
struct Chunk {
  uint64_t left, right;
  uint32_t key, begin, end;     // of this lane's run
};
__device__ __forceinline__ Chunk chunk_runs(const Sorted& a, int64_t tokens, int64_t vocab, int64_t chunk, int lane) {
  const int64_t i = chunk * kRun + lane;
  Chunk c;
  c.key = lane < kRun && i < tokens ? gld<uint32_t>(a.keys + i) : static_cast<uint32_t>(vocab);
  c.begin = c.end = 0;
  if (c.key < vocab) run_of(a, c.key, c.begin, c.end);
  const bool is_long = c.end - c.begin > kRun;
  c.left = __ballot(is_long && c.begin < chunk * kRun);
  c.right = __ballot(is_long && c.begin >= chunk * kRun);
  return c;
}

// Sums of the pieces of one chunk, the wave's 512 columns from c - 8 lane.
template <class S>
__device__ __forceinline__ void sum_pieces(const muon_embed_grad_t& op, const Sorted& a, int64_t chunk, int c, int lane) {
  const int cols = static_cast<int>(op.cols);
  const Chunk r = chunk_runs(a, op.tokens, op.vocab, chunk, lane);
  if (!(r.left | r.right)) return;
  const int64_t i = chunk * kRun + lane;
  const uint32_t held = i < op.tokens ? gld<uint32_t>(a.toks + i) : 0u;
#pragma unroll
  for (int side = 0; side < 2; ++side) {
    const uint64_t m = side ? r.right : r.left;
    if (!m) continue;
    float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    add_rows<S>(op, held, __builtin_ctzll(m), __popcll(m), c, s);
    Vec8<float>::store(a.pieces + (chunk * 2 + side) * cols + c, cols - c, s);
  }
}

// One row without a long run, by the TPR threads of a group, t of them this one.
// A row without tokens (most of them) is written in 16-byte pieces side by side,
// past the caches (222 us with the stores of put_row, 198 side by side, 190 past
// the caches: 32768 tokens into 32000 x 4096 in fp32).
template <class S, class T, int TPR>
__device__ __forceinline__ void sum_row(const muon_embed_grad_t& op, const Sorted& a, int64_t row, int t, int lane) {
  const int cols = static_cast<int>(op.cols);
  uint32_t first, end;
  run_of(a, static_cast<uint32_t>(row), first, end);
  const int len = static_cast<int>(end - first);
  if (len > kRun) return;                         // k_join's
  if (len == 0) {
    if (op.accumulate) return;
    constexpr int E = 16 / sizeof(T);
    T* out = static_cast<T*>(op.dtable) + row * op.ld_dtable;
    int c = t * E;
    for (; c + E <= cols; c += TPR * E)
      __builtin_nontemporal_store(u32x4_a2{0, 0, 0, 0}, (__attribute__((address_space(1))) u32x4_a2*)(out + c));
    for (int e = c; e < min(c + E, cols); ++e) gst<T>(out + e, T(0));
    return;
  }
  const uint32_t held = lane < len ? gld<uint32_t>(a.toks + first + lane) : 0u;
  for (int c0 = 0; c0 < cols; c0 += TPR * 8) {
    float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    add_rows<S>(op, held, 0, len, c0 + t * 8, s);
    put_row<T>(op, row, c0 + t * 8, s);
  }
}

// The pieces of the long runs (a wave per chunk and 512 columns) and, in the
// blocks behind them, the other rows.
template <class S, class T, int TPR>
__global__ __launch_bounds__(kRowThreads) void k_sums(muon_embed_grad_t op, Sorted a) {
  const int lane = threadIdx.x & 63;
  // uniform over a wave: taken from its first lane
  const int w = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) >> 6);
  if (blockIdx.x < a.piece_blocks) {
    const int per = static_cast<int>((op.cols + 511) / 512);   // waves of a chunk
    const int64_t n = a.chunks * per;
    for (int64_t u = static_cast<int64_t>(blockIdx.x) * 4 + w; u < n; u += static_cast<int64_t>(a.piece_blocks) * 4) {
      const int64_t chunk = u / per;
      sum_pieces<S>(op, a, chunk, static_cast<int>(u - chunk * per) * 512 + lane * 8, lane);
    }
    return;
  }
  constexpr int GPB = kRowThreads / TPR;
  const int64_t step = static_cast<int64_t>(gridDim.x - a.piece_blocks) * GPB;
  for (int64_t row = static_cast<int64_t>(blockIdx.x - a.piece_blocks) * GPB + (GPB > 1 ? w : 0); row < op.vocab; row += step)
    sum_row<S, T, TPR>(op, a, row, static_cast<int>(threadIdx.x) % TPR, lane);
}

// The long runs that begin among 64 places of the sorted order: their pieces,
// 512 columns from 512 blockIdx.y.  The waves take consecutive shares of a run's
// pieces, which are added in order.  8 waves where a row is one block's: a run of all
// of 32768 x 64 takes 59 us (with 4: 76) for the whole gradient, 10010 x 150 43 (58);
// 4 for wider rows, where the many blocks without a run count (32768 x 4096: 182 us,
// with 8: 185).
template <class T, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void k_join(muon_embed_grad_t op, Sorted a) {
  __shared__ float red[WAVES][512];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int cols = static_cast<int>(op.cols);
  const int c = static_cast<int>(blockIdx.y) * 512 + lane * 8;
  for (int64_t at = static_cast<int64_t>(blockIdx.x) * 64; at < op.tokens; at += static_cast<int64_t>(gridDim.x) * 64) {
    const int64_t i = at + lane;
    uint32_t key = static_cast<uint32_t>(op.vocab), begin = 0, end = 0;
    if (i < op.tokens) key = gld<uint32_t>(a.keys + i);
    if (key < op.vocab) run_of(a, key, begin, end);
    // (the same in all waves)
    for (uint64_t m = __ballot(end - begin > kRun && begin == i); m; m &= m - 1) {
      const int src = __builtin_ctzll(m);
      const int64_t row = static_cast<uint32_t>(__builtin_amdgcn_readlane(key, src));
      const int64_t chunk = (at + src) / kRun;
      const int64_t last = (static_cast<int64_t>(static_cast<uint32_t>(__builtin_amdgcn_readlane(end, src))) - 1) / kRun;
      const int n = static_cast<int>(last - chunk + 1), per = (n + WAVES - 1) / WAVES;
      const int to = min((w + 1) * per, n);
      float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
      for (int k = w * per; k < to; ++k) {
        Vec8<float> v;
        load8(v, static_cast<const float*>(a.pieces) + ((chunk + k) * 2 + (k == 0)) * cols + c, c, cols - c);
#pragma unroll
        for (int j = 0; j < 8; ++j) s[j] += v.get(j);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) red[w][j * 64 + lane] = s[j];
      __syncthreads();
      if (w == 0) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          s[j] = 0.f;
          for (int k = 0; k < WAVES; ++k) s[j] += red[k][j * 64 + lane];
        }
        put_row<T>(op, row, c, s);
      }
      __syncthreads();                               // before red is used again
    }
  }
}

// Blocks of a grid of `threads` each: its threads stay below 2^32, whatever the block.
constexpr int64_t max_grid(int64_t threads) { return (int64_t(1) << 31) / threads; }
size_t up256(size_t x) { return (x + 255) / 256 * 256; }

SortArgs sort_args(const muon_embed_grad_t& op, const EmbedSortPlan& p, int pass, char* ws) {
  SortArgs a;
  a.ids = op.ids;
  a.id_bytes = op.id_bytes;
  a.tokens = op.tokens;
  a.vocab = op.vocab;
  a.block_tokens = p.block_tokens;
  a.shift = kDigitBits * pass;
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
  EmbedSortPlan p{};
  if (tokens <= kDirect) return p;
  if (tokens <= kBucketTokens && vocab <= kBucketVocab) {
    p.passes = 1;
    p.log_buckets = kLogBuckets + ((vocab >> kLogBuckets) >= kHighs ? 1 : 0);
  } else {
    for (int64_t top = vocab; top > 0; top >>= kDigitBits) ++p.passes;
  }
  p.highs = static_cast<uint32_t>((vocab >> p.log_buckets) + 1);
  // at most 256 blocks, whole steps each
  p.block_tokens = kSortThreads * ((tokens + kSortThreads * 256 - 1) / (kSortThreads * 256));
  p.blocks = (tokens + p.block_tokens - 1) / p.block_tokens;
  p.chunks = (tokens + kRun - 1) / kRun;
  size_t off = 0;
  auto take = [&](int64_t n) {
    const size_t at = off;
    off = up256(off + static_cast<size_t>(n) * 4);
    return at;
  };
  for (int k = 0; k < std::min(p.passes, 2); ++k) {
    p.keys_off[k] = take(tokens);
    p.toks_off[k] = take(tokens);
  }
  if (!p.log_buckets) p.count_off = take(p.blocks * kDigits);
  p.start_off = take((int64_t(p.highs) << p.log_buckets) + 1);
  p.pieces_off = take(p.chunks * 2 * cols);
  p.bytes = off;
  return p;
}

int launch_embed(const muon_embed_t& op, void* stream) {
  const int64_t vpr = (op.cols + 7) / 8, blocks = (op.tokens * vpr + kRowThreads * kVecs - 1) / (kRowThreads * kVecs);
  return by_types(op.table_dtype, op.out_dtype, [&](auto s, auto t) {
    hipLaunchKernelGGL((k_embed<decltype(s), decltype(t)>), dim3(static_cast<unsigned>(std::min(blocks, max_grid(kRowThreads)))),
                       dim3(kRowThreads), 0, static_cast<hipStream_t>(stream), op, blocks);
    return static_cast<int>(hipGetLastError());
  });
}

int launch_embed_buckets(const muon_embed_grad_t& op, const EmbedSortPlan& p, char* ws, void* stream) {
  const dim3 grid(1u << p.log_buckets), block(kSortThreads);
  hipStream_t st = static_cast<hipStream_t>(stream);
  const SortArgs a = sort_args(op, p, 0, ws);
  if (op.id_bytes == 8) hipLaunchKernelGGL((k_embed_buckets<8>), grid, block, 0, st, a, p.log_buckets, p.highs, p.starts(ws));
  else hipLaunchKernelGGL((k_embed_buckets<4>), grid, block, 0, st, a, p.log_buckets, p.highs, p.starts(ws));
  return static_cast<int>(hipGetLastError());
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

int launch_embed_starts(const muon_embed_grad_t& op, const EmbedSortPlan& p, char* ws, void* stream) {
  hipLaunchKernelGGL(k_starts, dim3(static_cast<unsigned>((op.vocab + kRowThreads) / kRowThreads)), dim3(kRowThreads), 0,
                     static_cast<hipStream_t>(stream), p.keys(ws), static_cast<uint32_t>(op.tokens),
                     static_cast<uint32_t>(op.vocab), p.starts(ws));
  return static_cast<int>(hipGetLastError());
}

namespace {
Sorted sorted(const EmbedSortPlan& p, char* ws) {
  Sorted a;
  a.keys = p.keys(ws);
  a.toks = p.toks(ws);
  a.start = p.starts(ws);
  a.log_buckets = p.log_buckets;
  a.highs = p.highs;
  a.pieces = p.pieces(ws);
  a.chunks = p.chunks;
  a.piece_blocks = 0;
  return a;
}
}  // namespace

int launch_embed_sums(const muon_embed_grad_t& op, const EmbedSortPlan& p, char* ws, void* stream) {
  const bool direct = p.passes == 0, wide = op.cols > 512;
  const int64_t per_block = (wide ? 1 : 4) * (direct ? kRowsEach : 1);
  const int64_t row_blocks = std::min((op.vocab + per_block - 1) / per_block, max_grid(kRowThreads) / 2);
  return by_types(op.dy_dtype, op.table_dtype, [&](auto s, auto t) {
    using S = decltype(s);
    using T = decltype(t);
    hipStream_t st = static_cast<hipStream_t>(stream);
    if (direct) {
      const dim3 grid(static_cast<unsigned>(row_blocks));
      if (wide) hipLaunchKernelGGL((k_direct<S, T, 256>), grid, dim3(kRowThreads), 0, st, op);
      else hipLaunchKernelGGL((k_direct<S, T, 64>), grid, dim3(kRowThreads), 0, st, op);
    } else {
      Sorted a = sorted(p, ws);
      a.piece_blocks = static_cast<unsigned>(std::min((p.chunks * ((op.cols + 511) / 512) + 3) / 4, max_grid(kRowThreads) / 2));
      const dim3 grid(a.piece_blocks + static_cast<unsigned>(row_blocks));
      if (wide) hipLaunchKernelGGL((k_sums<S, T, 256>), grid, dim3(kRowThreads), 0, st, op, a);
      else hipLaunchKernelGGL((k_sums<S, T, 64>), grid, dim3(kRowThreads), 0, st, op, a);
    }
    return static_cast<int>(hipGetLastError());
  });
}

int launch_embed_join(const muon_embed_grad_t& op, const EmbedSortPlan& p, char* ws, void* stream) {
  const int threads = 64 * (op.cols > 512 ? 4 : 8);
  const dim3 grid(static_cast<unsigned>(std::min((op.tokens + 63) / 64, max_grid(threads))), static_cast<unsigned>((op.cols + 511) / 512));
  return by_types(op.dy_dtype, op.table_dtype, [&](auto, auto t) {
    hipStream_t st = static_cast<hipStream_t>(stream);
    if (op.cols > 512) hipLaunchKernelGGL((k_join<decltype(t), 4>), grid, dim3(threads), 0, st, op, sorted(p, ws));
    else hipLaunchKernelGGL((k_join<decltype(t), 8>), grid, dim3(threads), 0, st, op, sorted(p, ws));
    return static_cast<int>(hipGetLastError());
  });
}

}  // namespace muon
