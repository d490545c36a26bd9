// Attention over sequences of any lengths, and its backward pass (gfx950):
//   S = scale Q K^T (masked),  P = softmax(S),  O = P V,  lse = log sum exp S
//   dP = dO V^T,  dS = P (dP - rowsum(dO O)),  dQ = scale dS K,
//   dK = scale dS^T Q,  dV = P^T dO.
// S and P never leave the registers.  The backward pass recomputes P from lse, in
// two kernels, one that owns queries (dQ) and one that owns keys (dK, dV): seven
// products instead of five, but no sums across blocks, so no atomics, and the same
// bits every time.
//
// Rounded to bf16: P and dS as operands of the second products, whose sums are fp32 (half
// a step, 2^-8, of each term, as the inputs have), and the outputs, once.
//
// 4 x 4096 tokens, 32 heads of 128 over 8 of K and V, causal: forward 553 to 590 us (930
// to 990 TFLOP/s), backward 1720 to 1810 (760 to 800, five products counted; dQ 728 and dK,
// dV 958); 8192 tokens of 16 heads without a mask 1020 and 841; heads of 64: 904 and 764.
// A library product of 8192^3 reaches 1309 to 1409.  50 to 57 % of the cycles have a matrix
// instruction (38 at 64 columns, where vector instructions take as long as matrix ones; the
// exponentials run at a quarter of other instructions' rate).  Two waves share a SIMD, and in
// the forward pass each spends 37 % of its time ready but not issued and 21 % at waits and
// barriers: the softmax of a step stands between its two products.  No LDS conflicts.
//
// Layout.  A wave owns 32 queries (or keys), one per lane and half: it forms the
// transposed product S^T = K Q^T with v_mfma_f32_32x32x16_bf16, whose result leaves
// lane l with 16 of 32 keys of query l & 31.  A row's maximum and sum are then one
// exchange between the wave's halves, its rescaling is one factor a lane, and P,
// rounded to bf16, is already the second operand of O^T = V^T P^T: the instruction
// sums over keys, so they may come in the order in which the lane holds them,
//   element e of half h of 16-key step s  <->  key 16 s + 8 (e / 4) + 4 h + e % 4,
// if V^T is read in the same order, which the transposing LDS read does at no cost.
// The other products are of the same two kinds.
//
// Tiles of 64 rows lie in LDS as in memory, 16-byte chunk c of row r at c ^ swz(r):
// the 16 rows that a 16-byte read serves in one cycle, and the 4 rows by 4 chunks of a
// transposing read, then fall on distinct banks.  They are loaded straight into LDS
// while the tile before is in work.  Rows past a sequence's end and columns past dim
// are zeros there, so that nothing of a neighbour reaches a sum.
#include <algorithm>
#include <type_traits>

#include "muon_act8.h"
#include "muon_gemm.h"
#include "muon_ops.h"

namespace muon {

namespace {

typedef __attribute__((ext_vector_type(16))) float f32x16_t;
typedef short s16x4 __attribute__((ext_vector_type(4)));

constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;
constexpr float kInf = __builtin_inff();
constexpr int BN = 64;             // rows of a staged tile
constexpr int BM = 128;            // rows that a block owns, 32 a wave
constexpr int kThreads = 256;
constexpr int64_t kMaxParts = 16, kMaxForwardParts = 64;  // of a block's steps

// DB blocks of 32 columns are computed: dim up to 64, 96 or 128.
template <int DB>
struct Geo {
  static constexpr int KS = 2 * DB;                       // 16-column steps
  static constexpr int COLS = 32 * DB;                    // columns of a row in LDS
  static constexpr int ROWB = COLS * 2, CPR = COLS / 8;   // its bytes and chunks
  static constexpr int TILE = BN * ROWB;
};

// What the index of a chunk of row `row` is XORed with.  Rows of 192 bytes are a quarter of
// the banks apart by themselves.
template <int COLS>
__device__ __forceinline__ int swz(int row) {
  return COLS == 128 ? ((row & 3) << 2) | ((row >> 2) & 3) : COLS == 96 ? (row >> 2) & 3 : ((row & 2) << 1) | ((row >> 2) & 3);
}

__device__ __forceinline__ f32x16_t mfma(bf16x8_t a, bf16x8_t b, f32x16_t c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ float exp2_fast(float v) { return __builtin_amdgcn_exp2f(v); }
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __builtin_amdgcn_readfirstlane(v); }

// The kernel's first argument, read where it is used: scalar registers do not hold all of
// it over the loop.
template <class Op>
__device__ __forceinline__ const __attribute__((address_space(4))) Op* late() {
  const uint64_t at = reinterpret_cast<uint64_t>(__builtin_amdgcn_kernarg_segment_ptr());
  uint32_t lo = static_cast<uint32_t>(at), hi = static_cast<uint32_t>(at >> 32);
  asm volatile("" : "+v"(lo), "+v"(hi));
  return (const __attribute__((address_space(4))) Op*)(static_cast<uint64_t>(uniform(hi)) << 32 | uniform(lo));
}
__device__ __forceinline__ muon_heads_t copy(const __attribute__((address_space(4))) muon_heads_t& t) {
  return {t.data, t.ld_token, t.ld_head};
}

// Both halves' values in every lane.
__device__ __forceinline__ u32x2 halves(float v) {
  return __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false));
}
__device__ __forceinline__ float halves_max(float v) {
  const u32x2 r = halves(v);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float halves_sum(float v) {
  const u32x2 r = halves(v);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

__device__ __forceinline__ void block_barrier() { asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// 16 (4) bytes a lane from buffer `srd` at voff + soff into LDS at lds_dst + 16 (4)
// times the lane; zeros past the buffer's end.  An asm statement, because the
// compiler would wait for all of them before every later LDS read; block_barrier()
// waits.  The s_nop keeps the 5 wait states between a vector instruction's write of
// a scalar register and this read of it (and the one after a write of m0).
template <int BYTES>
__device__ __forceinline__ void dma(u32x4 srd, uint32_t voff, uint32_t soff, uint32_t lds_dst) {
  if constexpr (BYTES == 16)
    asm volatile("s_nop 4\n\tbuffer_load_dwordx4 %0, %1, %2 offen lds" ::"v"(voff), "s"(srd), "s"(soff), "{m0}"(lds_dst));
  else
    asm volatile("s_nop 4\n\tbuffer_load_dword %0, %1, %2 offen lds" ::"v"(voff), "s"(srd), "s"(soff), "{m0}"(lds_dst));
}
__device__ __forceinline__ uint32_t lds_at(const void* p) {
  return static_cast<uint32_t>(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) const void*)p));
}
__device__ __forceinline__ u32x4 buffer(const void* p, uint32_t bytes) {
  const uint64_t b = reinterpret_cast<uint64_t>(p);
  u32x4 srd;
  srd[0] = uniform(static_cast<uint32_t>(b));
  srd[1] = uniform(static_cast<uint32_t>(b >> 32) & 0xffffu);
  srd[2] = uniform(bytes);
  srd[3] = 0x00020000u;   // raw buffer of dwords
  return srd;
}

// Tiles of one head's rows of a sequence, into LDS.  ALIGNED: rows begin on 16
// bytes and 64 of them span less than 2^31 (attn_aligned): loads without registers,
// in flight until block_barrier().  Else through registers at once.
template <int DB, bool ALIGNED, int WAVES = 4>
struct Feed {
  using G = Geo<DB>;
  static constexpr int LOADS = G::TILE / 1024 / WAVES;    // 1 KB loads of a wave
  const uint16_t* p;
  int64_t ld;
  int rows, dim;                   // of the sequence; columns
  uint32_t voff[LOADS];
  int w, tid;

  __device__ __forceinline__ Feed(const muon_heads_t& t, int64_t row0, int nrows, int head, int dim_, int tid_)
      : p(static_cast<const uint16_t*>(t.data) + row0 * t.ld_token + head * t.ld_head), ld(t.ld_token), rows(nrows), dim(dim_), tid(tid_) {
    w = uniform(tid >> 6);
    if constexpr (ALIGNED) {
#pragma unroll
      for (int q = 0; q < LOADS; ++q) {
        const int at = (w * LOADS + q) * 64 + (tid & 63), r = at / G::CPR, c = (at % G::CPR) ^ swz<G::COLS>(r);
        voff[q] = c * 8 < dim ? static_cast<uint32_t>(r * ld * 2 + c * 16) : 0x80000000u;   // past every end
      }
    }
  }
  __device__ __forceinline__ void load(int row, char* dst) const {
    const int left = min(rows - row, BN);
    if (left <= 0) return;         // (uniform) no such tile: nobody reads it
    const uint16_t* at = p + row * ld;
    if constexpr (ALIGNED) {
      const uint32_t ldb = static_cast<uint32_t>(ld * 2);
      const u32x4 srd = buffer(at, (left - 1) * ldb + dim * 2);
      const uint32_t to = lds_at(dst);
#pragma unroll
      for (int q = 0; q < LOADS; ++q) {
        dma<16>(srd, voff[q], 0, to + (w * LOADS + q) * 1024);
      }
    } else {
#pragma unroll 1
      for (int i = tid; i < BN * G::CPR; i += 64 * WAVES) {
        const int r = i / G::CPR, c = (i % G::CPR) ^ swz<G::COLS>(r);
        u32x4 v{0, 0, 0, 0};
        if (r < left && c * 8 < dim) v = gld<u32x4_a2>(at + r * ld + c * 8);
        *reinterpret_cast<u32x4*>(dst + i * 16) = v;
      }
    }
  }
};

// Fragments of a staged tile.  rows(): row rb + (lane & 31), columns 16 ks + 8 h ..;
// cols(): column 32 db + (lane & 31), the rows of 16-row step s in the order above.
// FRESH: addresses are formed at each read, for a kernel whose registers do not hold
// those of all steps.
template <int DB, bool FRESH = false>
struct Frags {
  using G = Geo<DB>;
  int r0, t0;
  static __device__ __forceinline__ int flip(int v, int bits) {
    if constexpr (!FRESH) return v ^ bits;
    int r;
    asm volatile("v_xor_b32 %0, %1, %2" : "=v"(r) : "n"(bits), "v"(v));
    return r;
  }
  __device__ __forceinline__ explicit Frags(int lane) {
    const int l = lane & 31, h = lane >> 5, j = lane & 15;
    r0 = l * G::ROWB + ((h ^ swz<G::COLS>(l)) << 4);
    const int row = 4 * h + (j >> 2), c = 2 * ((lane >> 4) & 1) + ((j & 3) >> 1);
    t0 = row * G::ROWB + ((c ^ swz<G::COLS>(row)) << 4) + (j & 1) * 8;
  }
  __device__ __forceinline__ bf16x8_t rows(const char* tile, int rb, int ks) const {
    // (rows of 192 bytes: only the two low bits of a chunk change)
    constexpr bool low = G::COLS == 96;
    return *reinterpret_cast<const bf16x8_t*>(tile + rb * G::ROWB + (low ? (ks >> 1) * 64 : 0) + flip(r0, (low ? ks & 1 : ks) << 5));
  }
  __device__ __forceinline__ bf16x8_t cols(const char* tile, int s, int db) const {
    // 8 rows on, bit 1 of the swizzle is set
    constexpr bool low = G::COLS == 96;
    const char* at = tile + s * 16 * G::ROWB + (low ? db * 64 : 0);
    const int bits = low ? 0 : db << 6;
    const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)(at + flip(t0, bits)));
    const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)(at + 8 * G::ROWB + flip(t0, bits ^ 32)));
    return __builtin_bit_cast(bf16x8_t, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
  }
};

// The wave's own 32 rows as a second operand: row lane & 31, columns 16 ks + 8 h ..
template <int DB>
__device__ __forceinline__ void own_rows(const muon_heads_t& t, int64_t row0, int row, int nrows, int head, int dim, int h,
                                         bf16x8_t (&f)[2 * DB]) {
  const uint16_t* p = static_cast<const uint16_t*>(t.data) + (row0 + row) * t.ld_token + head * t.ld_head;
#pragma unroll
  for (int ks = 0; ks < 2 * DB; ++ks) {
    const int c = 16 * ks + 8 * h;
    u32x4 v{0, 0, 0, 0};
    if (row < nrows && c < dim) v = gld<u32x4_a2>(p + c);
    f[ks] = __builtin_bit_cast(bf16x8_t, v);
  }
}

// Fragments that have arrived.  Before a loop that issues loads of its own, or the
// compiler waits for those too, at each use inside it that may be the first.
template <int N>
__device__ __forceinline__ void arrived(bf16x8_t (&f)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    u32x4 v = __builtin_bit_cast(u32x4, f[i]);
    asm volatile("" : "+v"(v));
    f[i] = __builtin_bit_cast(bf16x8_t, v);
  }
}

// Two values rounded to bf16 by one instruction; a lane's 8 as an operand.
__device__ __forceinline__ uint32_t pack(float lo, float hi) {
  typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2;
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2_t{lo, hi}), bf16x2));
}
__device__ __forceinline__ bf16x8_t pack8(const f32x16_t& v, int from) {
  u32x4 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) r[i] = pack(v[from + 2 * i], v[from + 2 * i + 1]);
  return __builtin_bit_cast(bf16x8_t, r);
}

// Transposed sums (rows d, the lane's own row as column) times f, to the row: the
// halves trade registers, so that each stores 16 bytes at a time.
template <int DB>
__device__ __forceinline__ void store_row(const muon_heads_t& t, int64_t row, int head, int dim, int h, bool live,
                                          const f32x16_t (&acc)[DB], float f) {
  uint16_t* p = static_cast<uint16_t*>(t.data) + row * t.ld_token + head * t.ld_head;
#pragma unroll
  for (int db = 0; db < DB; ++db)
#pragma unroll
    for (int a = 0; a < 16; a += 8) {
      u32x4 o;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t x = pack(acc[db][a + 2 * i] * f, acc[db][a + 2 * i + 1] * f);
        const uint32_t y = pack(acc[db][a + 4 + 2 * i] * f, acc[db][a + 4 + 2 * i + 1] * f);
        const auto r = __builtin_amdgcn_permlane32_swap(x, y, false, false);
        o[i] = r[0];
        o[2 + i] = r[1];
      }
      const int d = 32 * db + 2 * a + 8 * h;
      if (live && d < dim) gst<u32x4_a2>(p + d, o);
    }
}

// The same in fp32, to `to` (columns side by side).
template <int DB>
__device__ __forceinline__ void store_part(float* to, int dim, int h, bool live, const f32x16_t (&acc)[DB], float f) {
#pragma unroll
  for (int db = 0; db < DB; ++db)
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const int d = 32 * db + 8 * g + 4 * h;
      if (live && d < dim)
        gst<f32x4_t>(to + d, f32x4_t{acc[db][4 * g] * f, acc[db][4 * g + 1] * f, acc[db][4 * g + 2] * f, acc[db][4 * g + 3] * f});
    }
}

// ------------------------------------------------------------ a block's rows ----
// Neighbouring blocks of an XCD share a head where the heads can be dealt to the XCDs
// evenly, and so its keys and values in the L2; else every head's tiles go to all of them,
// the heaviest first.
struct Deal {
  int head, unit;
};
struct Blocks {
  uint32_t block, blocks, units;   // this one, of units x heads
  uint32_t part, parts;            // of a block's steps
  __device__ __forceinline__ Deal deal() const {
    const uint32_t heads = uniform(blocks / units);
    if (heads % 8 == 0) {
      const uint32_t at = static_cast<uint32_t>(xcd_remap(block, blocks)), head = uniform(at / units);
      return {static_cast<int>(head), static_cast<int>(at - head * units)};
    }
    const uint32_t unit = uniform(block / heads);
    return {static_cast<int>(block - unit * heads), static_cast<int>(unit)};
  }
  // this part of n steps: from .. to - 1
  __device__ __forceinline__ int2 range(int n) const {
    const uint32_t each = uniform(static_cast<uint32_t>(n) / parts), more = n - each * parts;
    auto cut = [&](uint32_t i) { return static_cast<int>(uniform(i * each + min(i, more))); };
    return {cut(part), cut(part + 1)};
  }
};
__device__ __forceinline__ Blocks grid(uint32_t units) { return {blockIdx.x, gridDim.x, units, blockIdx.y, gridDim.y}; }

struct Place {
  int q0, nq, k0, nk;   // the sequence's first query and queries, first key and keys
  int tile;             // the block's tile of them
  bool found;
  bool rest;            // rows behind the last sequence
};

// Unit `unit` of the tiles of OWN queries (KEYS: keys) of all sequences, a query counted as
// `each` rows; those behind the last sequence are one more, without keys (queries), if they
// are to be written.  Starts
// are brought into range and order first, so that bad ones cannot lead outside the
// tensors.
//
// Under a causal mask and with fewer than 64 sequences, units are numbered by their work, the
// most first: the last queries and the first keys of all sequences (backward pass of 4 x
// 4096 tokens, 32 and 8 heads of 128: 1916 us, 2306 with one sequence after the other).
// Else tile t of sequence i, which begins at row a, is unit a / OWN + i + t: the numbers
// rise and none is used twice, so that a search of the starts finds it, 64 at a time.
template <bool KEYS, int OWN>
__device__ __forceinline__ Place place_of(const int32_t* starts, const int32_t* k_starts, int64_t sequences, int tokens, int k_tokens,
                                          bool rest, bool causal, int unit, int lane, int each = 1) {
  constexpr Place none{0, 0, 0, 0, 0, false, false};
  // the tile with `work` tiles of its sequence at or behind it (KEYS: before it)
  auto tile_of = [](int tiles, int work) { return KEYS ? tiles - work : work - 1; };
  auto tiles_of = [](int rows) { return (rows + OWN - 1) / OWN; };
  if (!starts) {
    const int tiles = tiles_of(KEYS ? k_tokens : tokens * each);
    return {0, tokens * each, 0, k_tokens, tile_of(tiles, tiles - unit), unit < tiles, false};
  }
  if (!k_starts) k_starts = starts;
  auto q_at = [&](int64_t i) { return min(max(gld<int32_t>(starts + i), 0), tokens) * each; };
  auto k_at = [&](int64_t i) { return min(max(gld<int32_t>(k_starts + i), 0), k_tokens); };
  auto sequence = [&](int64_t i) {        // its rows; the one behind the last: the rest
    Place p = none;
    const int64_t next = i < sequences ? i + 1 : i;
    p.q0 = q_at(i);
    p.k0 = k_at(i);
    p.nq = max(q_at(next) - p.q0, 0);
    p.nk = max(k_at(next) - p.k0, 0);
    p.rest = i == sequences;
    if (p.rest && rest) (KEYS ? p.nk : p.nq) = KEYS ? k_tokens - p.k0 : tokens * each - p.q0;
    return p;
  };
  if (causal && sequences < 64) {
    const Place p = lane <= sequences ? sequence(lane) : none;
    const int tiles = tiles_of(KEYS ? p.nk : p.nq);
    // the largest `work` of which fewer than unit + 1 tiles have more
    auto above = [&](int v) { return wave_all(max(tiles - v, 0), [](int x, int y) { return x + y; }); };
    if (above(0) <= unit) return none;
    int lo = 0, work = wave_all(tiles, [](int x, int y) { return max(x, y); });     // above(work) == 0 <= unit
    while (lo + 1 < work) {
      const int mid = lo + (work - lo) / 2;
      (above(mid) <= unit ? work : lo) = mid;
    }
    uint64_t with = __ballot(tiles >= work);
    for (int skip = unit - above(work); skip > 0; --skip) with &= with - 1;
    const int f = __builtin_ctzll(with);
    auto of = [&](int v) { return __builtin_amdgcn_readlane(v, f); };
    return {of(p.q0), of(p.nq), of(p.k0), of(p.nk), tile_of(of(tiles), work), true, f == sequences};
  }
  int64_t at = 0, left = sequences + 1;
  int first = 0;                            // the number of the sequence's first tile
  while (true) {
    const int64_t step = (left + 63) / 64, i = at + lane * step;
    const int number = lane * step < left ? static_cast<int>((KEYS ? k_at(i) : q_at(i)) / OWN + i) : 0;
    const uint64_t before = __ballot(lane * step < left && number <= unit);
    if (!before) return none;
    const int f = 63 - __builtin_clzll(before);
    first = __builtin_amdgcn_readlane(number, f);
    at += f * step;
    left = min(step, left - f * step);
    if (step == 1) break;
  }
  Place p = sequence(at);
  p.tile = unit - first;
  p.found = p.tile < tiles_of(KEYS ? p.nk : p.nq);
  return p;
}

// The same in scalar registers, which the compiler does not see through the loop.
template <bool KEYS, int OWN, class... Args>
__device__ __forceinline__ Place locate(Args... args) {
  const Place p = place_of<KEYS, OWN>(args...);
  auto one = [](int v) { return static_cast<int>(uniform(static_cast<uint32_t>(v))); };
  return {one(p.q0), one(p.nq), one(p.k0), one(p.nk), one(p.tile), one(p.found) != 0, one(p.rest) != 0};
}

// ------------------------------------------------------------- forward pass ----
// The running maximum and sum are fp32, one row a lane.  Rescaling is put off while no
// row's maximum has grown by more than 2^kSlack since the last one: P then reaches 2^kSlack
// at most, which costs no precision, and the sums are multiplied in few of the tiles
// instead of all.  The first load of the loop has to find nothing of the compiler's in
// flight (`arrived`): with Q's loads pending it waited for the next tile in each step (659
// us instead of 594 for the case above, when it was found).
constexpr float kSlack = 8.f;

//
// PACKED: a tile's rows are the queries of all heads that share a key and value head, one
// query after the other (row i: query i / group), so that few queries a sequence read their
// keys and values once, and a tile spans fewer queries, which a causal mask cuts closer (us
// with and without: 32 single queries over 4096 keys each, 32 heads of 128 over 8, 104, at
// 5.2 TB/s, and 217; 23 sequences of 8 to 1843 with 16 heads of 80 over 4, causal, 48 and
// 61; 8192 with 16 heads of 64 over 2 175 and 193; 4 x 4096 as above 566 and 575).
template <int DB, bool ALIGNED, bool PACKED>
__global__ __launch_bounds__(kThreads, DB == 3 ? 3 : 2) void k_attn(muon_attention_t op, uint32_t units, float* part_o, float* part_lse) {
  using G = Geo<DB>;
  __shared__ __attribute__((aligned(256))) char smem[4 * G::TILE];      // K, V; K, V of the next tile
  const int tid = threadIdx.x, lane = tid & 63, w = uniform(tid >> 6), h = lane >> 5;
  const Blocks g = grid(units);
  const auto [dealt, unit] = g.deal();
  const int group = uniform(static_cast<uint32_t>(op.heads / op.kv_heads)), each = PACKED ? group : 1;
  const Place pl = locate<false, BM>(op.starts, op.k_starts, op.sequences, op.tokens, op.k_tokens, op.zero_rest != 0, op.causal != 0, unit, lane, each);
  if (!pl.found) return;
  const int kv = PACKED ? dealt : static_cast<int>(uniform(static_cast<uint32_t>(dealt) / static_cast<uint32_t>(group))), dim = op.dim;
  auto query = [&](int row) { return PACKED ? static_cast<uint32_t>(row) / static_cast<uint32_t>(each) : static_cast<uint32_t>(row); };
  auto query_of_all = [&](int row) { return static_cast<int>(uniform(query(row))); };
  const int first = pl.tile * BM + 32 * w, row = first + (lane & 31);                  // the wave's first row, the lane's
  const int lowest = query_of_all(first), highest = query_of_all(first + 31), mine = query(row);   // their queries
  const int head = PACKED ? kv * each + row - mine * each : dealt, token = query_of_all(pl.q0) + mine;
  const int offset = pl.nk - query_of_all(pl.nq);                                      // key i + offset is query i's last (causal)
  const int block_last = query_of_all(min(pl.tile * BM + BM, pl.nq) - 1) + offset;
  const int keys = op.causal ? max(0, min(pl.nk, block_last + 1)) : pl.nk;             // that any query of the block sees

  bf16x8_t qf[G::KS];
  own_rows<DB>(op.q, token - row, row, pl.nq, head, dim, h, qf);
  const Feed<DB, ALIGNED> fk(op.k, pl.k0, keys, kv, dim, tid), fv(op.v, pl.k0, keys, kv, dim, tid);
  const Frags<DB> fr(lane);
  f32x16_t o[DB];
#pragma unroll
  for (int db = 0; db < DB; ++db) o[db] = f32x16_t{};
  float top = -kInf, sum = 0.f;                // top: the maximum that P is taken against; sum: of this half's keys
  const float c = op.scale * kLog2e;
  // kSlack in units of the scores; finite, as top is -inf at first and no NaN may arise (the
  // file is compiled as if there were none)
  const float slack = __uint_as_float(uniform(__float_as_uint(fminf(kSlack / c, 1e38f))));

  const auto [j0, j1] = g.range((keys + BN - 1) / BN);
  fk.load(j0 * BN, smem);
  fv.load(j0 * BN, smem + G::TILE);
  arrived(qf);
  block_barrier();
  auto step = [&](int j, const char* now, char* next) __attribute__((always_inline)) {
    fk.load((j + 1) * BN, next);
    fv.load((j + 1) * BN, next + G::TILE);
    const int k0 = j * BN;
    // no query of the wave sees the tile
    if (!(op.causal && k0 > highest + offset) && first < pl.nq) {
      // fragments of K are read AHEAD of their use, the first of V before the softmax
      constexpr int KS = G::KS, AHEAD = 3, EARLY = DB;
      f32x16_t s[2] = {};
      bf16x8_t f[2 * KS], vf[4 * DB];
      static_for<AHEAD>([&](auto i) __attribute__((always_inline)) { f[decltype(i)::value] = fr.rows(now, 32 * (decltype(i)::value % 2), decltype(i)::value / 2); });
      static_for<2 * KS>([&](auto ic) __attribute__((always_inline)) {
        constexpr int i = decltype(ic)::value, n = i + AHEAD;
        if constexpr (n < 2 * KS) f[n] = fr.rows(now, 32 * (n % 2), n / 2);
        else if constexpr (n - 2 * KS < EARLY) vf[n - 2 * KS] = fr.cols(now + G::TILE, (n - 2 * KS) / DB, (n - 2 * KS) % DB);
        s[i % 2] = mfma(f[i], qf[i / 2], s[i % 2]);
        __builtin_amdgcn_sched_barrier(0);
      });
      static_for<EARLY - (AHEAD < EARLY ? AHEAD : EARLY)>([&](auto ic) __attribute__((always_inline)) {
        constexpr int n = AHEAD + decltype(ic)::value;
        vf[n] = fr.cols(now + G::TILE, n / DB, n % DB);
      });
      if (k0 + BN > pl.nk || (op.causal && k0 + BN - 1 > lowest + offset)) {
        const int last = op.causal ? min(pl.nk - 1, mine + offset) : pl.nk - 1;
#pragma unroll
        for (int kb = 0; kb < 2; ++kb)
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (k0 + 32 * kb + 8 * (i / 4) + 4 * h + i % 4 > last) s[kb][i] = -kInf;
      }
      float m = fmaxf(s[0][0], s[1][0]);
#pragma unroll
      for (int i = 1; i < 16; ++i) m = fmaxf(m, fmaxf(s[0][i], s[1][i]));
      m = halves_max(m);
      if (__any(m > top + slack)) {
        const float grown = fmaxf(m, top);
        const float f = grown == -kInf ? 0.f : exp2_fast((top - grown) * c);
        top = grown;
        sum *= f;
#pragma unroll
        for (int db = 0; db < DB; ++db) o[db] *= f;
      }
      const float base = top == -kInf ? 0.f : top * c;
      float part[4] = {};
#pragma unroll
      for (int kb = 0; kb < 2; ++kb)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          s[kb][i] = exp2_fast(s[kb][i] * c - base);
          part[i & 3] += s[kb][i];
        }
      sum += (part[0] + part[1]) + (part[2] + part[3]);
      bf16x8_t pf[4];
#pragma unroll
      for (int st = 0; st < 4; ++st) pf[st] = pack8(s[st / 2], 8 * (st % 2));
      __builtin_amdgcn_sched_barrier(0);
      static_for<4 * DB>([&](auto ic) __attribute__((always_inline)) {
        constexpr int i = decltype(ic)::value, n = i + EARLY;
        if constexpr (n < 4 * DB) vf[n] = fr.cols(now + G::TILE, n / DB, n % DB);
        o[i % DB] = mfma(vf[i], pf[i / DB], o[i % DB]);
        __builtin_amdgcn_sched_barrier(0);
      });
    }
    block_barrier();
  };
  for (int j = j0; j < j1; j += 2) {
    step(j, smem, smem + 2 * G::TILE);
    if (j + 1 < j1) step(j + 1, smem + 2 * G::TILE, smem);
  }
  sum = halves_sum(sum);
  const bool live = row < pl.nq;
  const auto* end = late<muon_attention_t>();
  const int rest = pl.rest ? end->zero_rest : ~0;
  if (g.parts > 1) {
    const int64_t at = (static_cast<int64_t>(g.part) * end->tokens + token) * end->heads + head;
    store_part<DB>(part_o + at * dim, dim, h, live, o, sum == 0.f ? 0.f : 1.f / sum);
    if (live && h == 0) gst<float>(part_lse + at, sum == 0.f ? -kInf : (top * c + __builtin_amdgcn_logf(sum)) * kLn2);
    return;
  }
  store_row<DB>(copy(end->o), token, head, dim, h, live && (rest & MUON_ATTN_ZERO_O), o, sum == 0.f ? 0.f : 1.f / sum);
  if (end->lse && live && h == 0 && (rest & MUON_ATTN_ZERO_LSE))
    gst<float>(end->lse + head * end->ld_lse + token, sum == 0.f ? -kInf : (top * c + __builtin_amdgcn_logf(sum)) * kLn2);
}

// ------------------------------------------------------------ backward: dQ ----
// As the forward pass, with both S^T = K Q^T and dP^T = V dO^T; the row's lse and
// rowsum(dO O) are one value a lane, left for the other kernel (lse in powers of two, +inf
// where the row sees nothing, so that its P is 0; the sum negated, as dP begins with it).
template <int DB, bool ALIGNED>
__device__ __forceinline__ void dq_tile(const muon_attention_grad_t& op, Blocks g, float* stats, float* part_dq, char* smem) {
  using G = Geo<DB>;
  const int tid = threadIdx.x, lane = tid & 63, w = uniform(tid >> 6), h = lane >> 5;
  const auto [head, unit] = g.deal();
  const Place pl = locate<false, BM>(op.starts, op.k_starts, op.sequences, op.tokens, op.k_tokens, (op.zero_rest & MUON_ATTN_ZERO_DQ) != 0,
                                   op.causal != 0, unit, lane);
  if (!pl.found) return;
  const int kv = uniform(static_cast<uint32_t>(head) / static_cast<uint32_t>(op.heads / op.kv_heads)), dim = op.dim;
  const int first = pl.tile * BM + 32 * w, mine = first + (lane & 31), offset = pl.nk - pl.nq;
  const int block_last = min(pl.tile * BM + BM, pl.nq) - 1 + offset;
  const int keys = op.causal ? max(0, min(pl.nk, block_last + 1)) : pl.nk;

  const Feed<DB, ALIGNED> fk(op.k, pl.k0, keys, kv, dim, tid), fv(op.v, pl.k0, keys, kv, dim, tid);
  const auto [j0, j1] = g.range((keys + BN - 1) / BN);
  fk.load(j0 * BN, smem);
  fv.load(j0 * BN, smem + G::TILE);
  bf16x8_t qf[G::KS], gf[G::KS];
  float delta = 0.f, base = 0.f;
  {
    own_rows<DB>(op.o, pl.q0, mine, pl.nq, head, dim, h, qf);
    own_rows<DB>(op.dout, pl.q0, mine, pl.nq, head, dim, h, gf);
#pragma unroll
    for (int ks = 0; ks < G::KS; ++ks)
#pragma unroll
      for (int e = 0; e < 8; ++e) delta += static_cast<float>(qf[ks][e]) * static_cast<float>(gf[ks][e]);
    delta = halves_sum(delta);
    if (mine < pl.nq) {
      const int64_t row = pl.q0 + mine;
      const float l = gld<float>(op.lse + head * op.ld_lse + row);
      base = l == -kInf ? kInf : l * kLog2e;
      if (h == 0 && g.part == 0 && stats) {
        gst<float>(stats + head * op.tokens + row, base);
        gst<float>(stats + (op.heads + head) * op.tokens + row, -delta);
      }
    }
    own_rows<DB>(op.q, pl.q0, mine, pl.nq, head, dim, h, qf);
  }
  const Frags<DB> fr(lane);
  // dP's sums begin with -delta, where registers hold that many copies of it
  constexpr bool LESS = DB < 4;
  f32x16_t less{};
  if constexpr (LESS)
#pragma unroll
    for (int i = 0; i < 16; ++i) less[i] = -delta;
  f32x16_t dq[DB];
#pragma unroll
  for (int db = 0; db < DB; ++db) dq[db] = f32x16_t{};
  const float c = op.scale * kLog2e;

  arrived(qf);
  arrived(gf);
  block_barrier();
  auto step = [&](int j, const char* now, char* next) __attribute__((always_inline)) {
    fk.load((j + 1) * BN, next);
    fv.load((j + 1) * BN, next + G::TILE);
    const int k0 = j * BN;
    if (!(op.causal && k0 > first + 31 + offset) && first < pl.nq) {
      const bool partial = k0 + BN > pl.nk || (op.causal && k0 + BN - 1 > first + offset);
      const int last = op.causal ? min(pl.nk - 1, mine + offset) : pl.nk - 1;
      // six phases of KS matrix instructions, a fragment of K or V each, read AHEAD of its
      // use: S, dP of the first 32 keys, S, dP of the others, dQ from both; beside dP the
      // exponentials, beside the next phase the rest of dS
      constexpr int KS = G::KS, AHEAD = 3;
      f32x16_t s[2] = {}, dp[2] = {less, less};
      bf16x8_t f[6 * KS], sf[4];
      auto fetch = [&](auto i) __attribute__((always_inline)) {
        constexpr int phase = decltype(i)::value / KS, n = decltype(i)::value % KS;
        if constexpr (phase < 4) f[decltype(i)::value] = fr.rows(now + phase % 2 * G::TILE, 32 * (phase / 2), n);
        else f[decltype(i)::value] = fr.cols(now, 2 * (phase - 4) + n / DB, n % DB);
      };
      auto phase = [&](auto ph) __attribute__((always_inline)) {
        constexpr int P = decltype(ph)::value, kb = P < 4 ? P / 2 : P - 4;
        static_for<KS>([&](auto nc) __attribute__((always_inline)) {
          constexpr int n = decltype(nc)::value, at_f = P * KS + n;
          if constexpr (at_f + AHEAD < 6 * KS) fetch(std::integral_constant<int, at_f + AHEAD>{});
          if constexpr (P == 0 || P == 2) s[kb] = mfma(f[at_f], qf[n], s[kb]);
          if constexpr (P == 1 || P == 3) dp[kb] = mfma(f[at_f], gf[n], dp[kb]);
          if constexpr (P >= 4) dq[n % DB] = mfma(f[at_f], sf[2 * kb + n / DB], dq[n % DB]);
          if constexpr (P >= 1 && P <= 4) {
            constexpr int of = P <= 2 ? 0 : 1;
            static_for<16 * (n + 1) / KS - 16 * n / KS>([&](auto u) __attribute__((always_inline)) {
              constexpr int i = 16 * n / KS + decltype(u)::value;
              if constexpr (P % 2) s[of][i] = exp2_fast(s[of][i] * c - base);
              else if constexpr (LESS) s[of][i] *= dp[of][i];
              else s[of][i] *= dp[of][i] - delta;
              if constexpr (P % 2 == 0 && i % 8 == 7) sf[2 * of + i / 8] = pack8(s[of], i - 7);
            });
          }
          __builtin_amdgcn_sched_barrier(0);
        });
      };
      auto mask = [&](int kb) __attribute__((always_inline)) {
        if (!partial) return;
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (k0 + 32 * kb + 8 * (i / 4) + 4 * h + i % 4 > last) s[kb][i] = -kInf;
      };
      static_for<AHEAD>([&](auto i) __attribute__((always_inline)) { fetch(i); });
      phase(std::integral_constant<int, 0>{});
      mask(0);
      phase(std::integral_constant<int, 1>{});
      phase(std::integral_constant<int, 2>{});
      mask(1);
      phase(std::integral_constant<int, 3>{});
      phase(std::integral_constant<int, 4>{});
      phase(std::integral_constant<int, 5>{});
    }
    block_barrier();
  };
  for (int j = j0; j < j1; j += 2) {
    step(j, smem, smem + 2 * G::TILE);
    if (j + 1 < j1) step(j + 1, smem + 2 * G::TILE, smem);
  }
  const auto* end = late<muon_attention_grad_t>();
  if (g.parts > 1) {
    const int64_t row = (static_cast<int64_t>(g.part) * end->tokens + pl.q0 + mine) * end->heads + head;
    store_part<DB>(part_dq + row * dim, dim, h, mine < pl.nq, dq, 1.f);
    return;
  }
  store_row<DB>(copy(end->dq), pl.q0 + mine, head, dim, h, mine < pl.nq, dq, end->scale);
}

template <int DB, bool ALIGNED>
__global__ __launch_bounds__(kThreads, 2) void k_attn_dq(muon_attention_grad_t op, uint32_t units, float* stats, float* part_dq) {
  __shared__ __attribute__((aligned(256))) char smem[4 * Geo<DB>::TILE];
  dq_tile<DB, ALIGNED>(op, grid(units), stats, part_dq, smem);
}

// ------------------------------------------------------- backward: dK and dV ----
// A wave owns KB blocks of 32 keys, one per lane and half, and walks the queries of every
// head that shares them, 32 at a time: S = Q K^T and dP = dO V^T leave a lane with 16 of 32
// queries of its keys, in whose order dV^T = dO^T P and dK^T = Q^T dS then take them.  lse
// and rowsum(dO O) come with the tile.  A query past the sequence's end has zeros
// everywhere and adds nothing.
//
// The four products of a step are four phases of KS fragments of Q or dO, in a fixed
// order: a fragment is read AHEAD of its use, the exponentials of P are spread over the
// instructions of dP, the products of dS over the ones of dV (1791 -> 1075 us for the case
// above; left to the compiler, each matrix instruction waited for its own read).  Sums, K
// and V of 128 columns are more than a wave's 256 registers hold beside that: V then waits
// in LDS, 8 waves to a block, so that two of them still share a SIMD.  (64 keys a wave, one
// wave to a SIMD, spilled: the compiler moves accumulators between the register files.)
template <int DB>
constexpr int kKeyWaves = DB == 4 ? 8 : 4;

template <int DB>
struct KeyLds {
  using G = Geo<DB>;
  static constexpr int STAGE = 2 * G::TILE + 2 * BN * 4;       // Q, dO, lse, -rowsum(dO O)
  static constexpr bool V = DB == 4;                           // the registers hold K alone
  static constexpr int bytes = 2 * STAGE + (V ? 32 * kKeyWaves<DB> * G::ROWB : 0);
};

// STATS: lse and rowsum(dO O) are in `stats`; else they are formed with each tile.
template <int DB, bool ALIGNED, bool STATS>
__device__ __forceinline__ void dkv_tile(const muon_attention_grad_t& op, Blocks g_, const float* stats, float* part_dkv, char* smem) {
  using G = Geo<DB>;
  constexpr int KB = 1, KS = G::KS, AHEAD = 2, WAVES = kKeyWaves<DB>, OWN = 32 * WAVES;
  constexpr int STAGE = KeyLds<DB>::STAGE;
  constexpr bool V_LDS = KeyLds<DB>::V;
  const int tid = threadIdx.x, lane = tid & 63, w = uniform(tid >> 6), h = lane >> 5;
  const auto [kv, unit] = g_.deal();
  const Place pl = locate<true, OWN>(op.starts, op.k_starts, op.sequences, op.tokens, op.k_tokens,
                                     (op.zero_rest & (MUON_ATTN_ZERO_DK | MUON_ATTN_ZERO_DV)) != 0, op.causal != 0, unit, lane);
  if (!pl.found) return;
  const int share = uniform(static_cast<uint32_t>(op.heads) / static_cast<uint32_t>(op.kv_heads)), dim = op.dim;
  const int first = pl.tile * OWN + 32 * KB * w, mine = first + (lane & 31), offset = pl.nk - pl.nq;
  // the first query that sees a key of the block
  const int from = op.causal ? max(0, pl.tile * OWN - offset) : 0;
  const int first_tile = from / BN, tiles = max((pl.nq + BN - 1) / BN - first_tile, 0);
  const auto [s0, s1] = g_.range(share * tiles);          // steps: the heads' tiles, one head after the other

  bf16x8_t kf[KB][KS], vf[V_LDS ? 1 : KB][KS];
  char* const own_v = smem + 2 * STAGE + w * (32 * KB) * G::ROWB;       // the wave's own rows of V, for itself
#pragma unroll
  for (int kb = 0; kb < KB; ++kb) {
    own_rows<DB>(op.k, pl.k0, mine + 32 * kb, pl.nk, kv, dim, h, kf[kb]);
    bf16x8_t (&v)[KS] = vf[V_LDS ? 0 : kb];
    own_rows<DB>(op.v, pl.k0, mine + 32 * kb, pl.nk, kv, dim, h, v);
    if constexpr (V_LDS) {
      const int row = 32 * kb + (lane & 31);
#pragma unroll
      for (int ks = 0; ks < KS; ++ks)
        *reinterpret_cast<bf16x8_t*>(own_v + row * G::ROWB + (((2 * ks + h) ^ swz<G::COLS>(row)) << 4)) = v[ks];
    }
  }
  const Frags<DB, (DB > 2)> fr(lane);
  f32x16_t dk[KB][DB], dv[KB][DB];
#pragma unroll
  for (int kb = 0; kb < KB; ++kb)
#pragma unroll
    for (int db = 0; db < DB; ++db) dk[kb][db] = dv[kb][db] = f32x16_t{};
  const float c = op.scale * kLog2e;
#pragma unroll
  for (int kb = 0; kb < KB; ++kb) {
    arrived(kf[kb]);
    if constexpr (!V_LDS) arrived(vf[kb]);
  }

  for (int turn = 0; turn < share; ++turn) {
    const int head = kv * share + turn, j0 = uniform(first_tile + max(s0 - turn * tiles, 0)),
              j1 = uniform(first_tile + min(s1 - turn * tiles, tiles));
    if (j0 >= j1) continue;
    const auto* in = late<muon_attention_grad_t>();
    const Feed<DB, ALIGNED, WAVES> fq(copy(in->q), pl.q0, pl.nq, head, dim, tid), fg(copy(in->dout), pl.q0, pl.nq, head, dim, tid);
    // wave 0: lse, 1: delta
    const float* rows = STATS ? stats + head * in->tokens + pl.q0 + (w == 1 ? in->heads * in->tokens : 0) : nullptr;
    auto load = [&](int j, char* to) __attribute__((always_inline)) {
      fq.load(j * BN, to);
      fg.load(j * BN, to + G::TILE);
      const int left = min(pl.nq - j * BN, BN);
      if constexpr (!STATS) {
        if (left > 0 && tid < 4 * BN) {          // four threads to a row
          const auto* more = late<muon_attention_grad_t>();
          const int r = tid >> 2;
          const int64_t row = pl.q0 + j * BN + r;
          float sum = 0.f, l = 0.f;
          if (r < left) {
            const uint16_t* po = static_cast<const uint16_t*>(more->o.data) + row * more->o.ld_token + head * more->o.ld_head;
            const uint16_t* pg = static_cast<const uint16_t*>(more->dout.data) + row * more->dout.ld_token + head * more->dout.ld_head;
            for (int c = (tid & 3) * 8; c < dim; c += 32) {
              Vec8<uint16_t> a, b;
              a.load(po + c);
              b.load(pg + c);
#pragma unroll
              for (int e = 0; e < 8; ++e) sum += a.get(e) * b.get(e);
            }
            l = gld<float>(more->lse + head * more->ld_lse + row);
            l = l == -kInf ? kInf : l * kLog2e;
          }
          sum += __uint_as_float(quad_perm<0xB1>(__float_as_uint(sum)));
          sum += __uint_as_float(quad_perm<0x4E>(__float_as_uint(sum)));
          if ((tid & 3) == 0) {
            float* stat = reinterpret_cast<float*>(to + 2 * G::TILE);
            stat[r] = l;
            stat[BN + r] = -sum;
          }
        }
      } else if (w < 2 && left > 0)
        dma<4>(buffer(rows + j * BN, left * 4), lane * 4, 0, lds_at(to + 2 * G::TILE + w * BN * 4));
    };
    auto step = [&](int j, const char* now, char* next) __attribute__((always_inline)) {
      load(j + 1, next);
#pragma unroll
      for (int qb = 0; qb < 2; ++qb) {
        const int q0 = j * BN + 32 * qb;
        // none of the queries sees a key of the wave, or there are none
        if ((op.causal && q0 + 31 + offset < first) || q0 >= pl.nq || first >= pl.nk) continue;
        f32x16_t s[KB] = {}, dp[KB];
        bf16x8_t f[4 * KS], vl[V_LDS ? KB : 1][KS], pf[KB][2], xf[KB][2];
        f32x4_t l[4];
        auto fetch = [&](auto i) __attribute__((always_inline)) {
          constexpr int phase = decltype(i)::value / KS, n = decltype(i)::value % KS;
          if constexpr (phase == 1 && V_LDS)
            static_for<KB>([&](auto kb) __attribute__((always_inline)) { vl[decltype(kb)::value][n] = fr.rows(own_v, 32 * decltype(kb)::value, n); });
          if constexpr (phase < 2) f[decltype(i)::value] = fr.rows(now + phase * G::TILE, 32 * qb, n);
          else f[decltype(i)::value] = fr.cols(now + (3 - phase) * G::TILE, 2 * qb + n / DB, n % DB);
        };
        // four rows' lse or -delta, before their first use; dP's sums begin with the latter
        auto stat = [&](int which, int g) __attribute__((always_inline)) {
          return *reinterpret_cast<const f32x4_t*>(now + 2 * G::TILE + which * BN * 4 + (32 * qb + 8 * g + 4 * h) * 4);
        };
        // the j-th value of P (then of dS): four queries of each key block in turn
        auto element = [&](auto second, auto jc) __attribute__((always_inline)) {
          constexpr int jj = decltype(jc)::value, g = jj / (4 * KB), kb = jj / 4 % KB, e = jj % 4, i = 4 * g + e;
          if constexpr (!decltype(second)::value) s[kb][i] = exp2_fast(s[kb][i] * c - l[g][e]);
          else dp[kb][i] *= s[kb][i];
          if constexpr (e == 3 && (g & 1)) (decltype(second)::value ? xf : pf)[kb][g / 2] = pack8(decltype(second)::value ? dp[kb] : s[kb], 8 * (g / 2));
          if constexpr (!decltype(second)::value && e == 3 && kb == KB - 1 && g < 3) l[g + 1] = stat(0, g + 1);
        };
        auto phase = [&](auto ph) __attribute__((always_inline)) {
          constexpr int P = decltype(ph)::value;
          static_for<KS>([&](auto nc) __attribute__((always_inline)) {
            constexpr int n = decltype(nc)::value, at_f = P * KS + n;
            if constexpr (at_f + AHEAD < 4 * KS) fetch(std::integral_constant<int, at_f + AHEAD>{});
            if constexpr (P == 0 && n == KS - 2) l[0] = stat(0, 0);
            if constexpr (P == 0 && n >= KS - 4) {
              const f32x4_t d = stat(1, n - KS + 4);
#pragma unroll
              for (int kb = 0; kb < KB; ++kb)
#pragma unroll
                for (int e = 0; e < 4; ++e) dp[kb][4 * (n - KS + 4) + e] = d[e];
            }
            static_for<KB>([&](auto kc) __attribute__((always_inline)) {
              constexpr int kb = decltype(kc)::value, slot = n * KB + kb;
              if constexpr (P == 0) s[kb] = mfma(f[at_f], kf[kb][n], s[kb]);
              if constexpr (P == 1) dp[kb] = mfma(f[at_f], V_LDS ? vl[V_LDS ? kb : 0][n] : vf[V_LDS ? 0 : kb][n], dp[kb]);
              if constexpr (P == 2) dv[kb][n % DB] = mfma(f[at_f], pf[kb][n / DB], dv[kb][n % DB]);
              if constexpr (P == 3) dk[kb][n % DB] = mfma(f[at_f], xf[kb][n / DB], dk[kb][n % DB]);
              if constexpr (P == 1 || P == 2) {
                constexpr int j0_ = 16 * slot / KS, j1_ = 16 * (slot + 1) / KS;
                static_for<j1_ - j0_>([&](auto u) __attribute__((always_inline)) {
                  element(std::integral_constant<bool, P == 2>{}, std::integral_constant<int, j0_ + decltype(u)::value>{});
                });
              }
              __builtin_amdgcn_sched_barrier(0);
            });
          });
        };
        static_for<AHEAD>([&](auto i) __attribute__((always_inline)) { fetch(i); });
        phase(std::integral_constant<int, 0>{});
        if (op.causal && q0 + offset < first + 32 * KB - 1) {
#pragma unroll
          for (int kb = 0; kb < KB; ++kb)
#pragma unroll
            for (int i = 0; i < 16; ++i)
              if (mine + 32 * kb > q0 + 8 * (i / 4) + 4 * h + i % 4 + offset) s[kb][i] = -kInf;
        }
        phase(std::integral_constant<int, 1>{});
        phase(std::integral_constant<int, 2>{});
        phase(std::integral_constant<int, 3>{});
      }
      block_barrier();
    };
    load(j0, smem);
    block_barrier();
    for (int j = j0; j < j1; j += 2) {
      step(j, smem, smem + STAGE);
      if (j + 1 < j1) step(j + 1, smem + STAGE, smem);
    }
  }
  const auto* end = late<muon_attention_grad_t>();
  const int rest = pl.rest ? end->zero_rest : ~0;
#pragma unroll
  for (int kb = 0; kb < KB; ++kb) {
    const int key = mine + 32 * kb;
    const bool live = key < pl.nk;
    if (g_.parts > 1) {
      const int64_t rows = end->k_tokens * end->kv_heads, row = (pl.k0 + key) * end->kv_heads + kv;
      store_part<DB>(part_dkv + (2 * g_.part * rows + row) * dim, dim, h, live, dk[kb], 1.f);
      store_part<DB>(part_dkv + ((2 * g_.part + 1) * rows + row) * dim, dim, h, live, dv[kb], 1.f);
      continue;
    }
    store_row<DB>(copy(end->dk), pl.k0 + key, kv, dim, h, live && (rest & MUON_ATTN_ZERO_DK), dk[kb], end->scale);
    store_row<DB>(copy(end->dv), pl.k0 + key, kv, dim, h, live && (rest & MUON_ATTN_ZERO_DV), dv[kb], 1.f);
  }
}

template <int DB, bool ALIGNED>
__global__ __launch_bounds__(64 * kKeyWaves<DB>, 2) void k_attn_dkv(muon_attention_grad_t op, uint32_t units, const float* stats, float* part_dkv) {
  __shared__ __attribute__((aligned(256))) char smem[KeyLds<DB>::bytes];
  dkv_tile<DB, ALIGNED, true>(op, grid(units), stats, part_dkv, smem);
}

// Both in one launch, for few blocks: the first q_blocks make dQ, the others dK and dV, with
// rowsum(dO O) for themselves.  Past 96 columns a block has a CU's LDS to itself, so that there
// 257 and more take two rounds.
template <int DB, bool ALIGNED>
__global__ __launch_bounds__(64 * kKeyWaves<DB>, 2) void k_attn_grad(muon_attention_grad_t op, uint32_t units, uint32_t q_blocks, uint32_t k_units) {
  constexpr int bytes = KeyLds<DB>::bytes > 4 * Geo<DB>::TILE ? KeyLds<DB>::bytes : 4 * Geo<DB>::TILE;
  __shared__ __attribute__((aligned(256))) char smem[bytes];
  if (blockIdx.x >= q_blocks)
    dkv_tile<DB, ALIGNED, false>(op, Blocks{blockIdx.x - q_blocks, gridDim.x - q_blocks, k_units, 0, 1}, nullptr, nullptr, smem);
  else if (threadIdx.x < kThreads)
    dq_tile<DB, ALIGNED>(op, Blocks{blockIdx.x, q_blocks, units, 0, 1}, nullptr, nullptr, smem);
}

// ------------------------------------------------------------------- parts ----
// Joins the parts of a few long rows, in their order: 8 columns a thread of `rows` x `heads`
// x `dim` (gridDim.y: 2 tensors, one behind the other in each part).  With lse, parts of
// attention are weighted by exp(lse of the part - lse).
struct Join {
  muon_heads_t  out[2];
  const float*  part;
  const float*  part_lse;      // NULL: sums
  float*        lse;           // may be NULL
  const int32_t* starts;
  int64_t       sequences, rows, heads, dim, ld_lse;
  int           parts;
  float         factor[2];
  bool          all[2], all_lse;   // also rows behind the last sequence
};

__global__ __launch_bounds__(256) void k_attn_join(Join j) {
  const int which = blockIdx.y;
  const int64_t chunks = j.dim / 8, i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x, at = i / chunks, row = at / j.heads;
  if (row >= j.rows) return;
  const int64_t head = at - row * j.heads, d = (i - at * chunks) * 8, end = j.starts ? gld<int32_t>(j.starts + j.sequences) : j.rows;
  const bool inside = row < end;
  float v[8] = {}, top = -kInf, total = 0.f;
  if (j.part_lse)
#pragma unroll 4
    for (int p = 0; p < j.parts; ++p) top = fmaxf(top, gld<float>(j.part_lse + (p * j.rows + row) * j.heads + head));
  const float base = top == -kInf ? 0.f : top;
#pragma unroll 4
  for (int p = 0; p < j.parts; ++p) {
    const float* from = j.part + ((static_cast<int64_t>(p) * gridDim.y + which) * j.rows * j.heads + at) * j.dim + d;
    const f32x4_t a = gld<f32x4_t>(from), b = gld<f32x4_t>(from + 4);
    float f = 1.f;
    if (j.part_lse) {
      f = exp2_fast((gld<float>(j.part_lse + (p * j.rows + row) * j.heads + head) - base) * kLog2e);
      total += f;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[e] += f * a[e];
      v[4 + e] += f * b[e];
    }
  }
  const float f = j.part_lse ? (total == 0.f ? 0.f : 1.f / total) : j.factor[which];
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] *= f;
  if (inside || j.all[which])
    Vec8<uint16_t>::store(static_cast<uint16_t*>(j.out[which].data) + row * j.out[which].ld_token + head * j.out[which].ld_head + d, 8, v);
  if (j.lse && d == 0 && (inside || j.all_lse))
    gst<float>(j.lse + head * j.ld_lse + row, total == 0.f ? -kInf : base + __builtin_amdgcn_logf(total) * kLn2);
}

// ---------------------------------------------------------------- dispatch ----
uint32_t units_of(int64_t tokens, int64_t sequences, bool ragged, int own = BM) {
  return static_cast<uint32_t>((tokens + own - 1) / own + (ragged ? sequences + 1 : 0));
}

bool aligned16(const muon_heads_t& t) {
  return reinterpret_cast<uintptr_t>(t.data) % 16 == 0 && t.ld_token % 8 == 0 && t.ld_head % 8 == 0 && t.ld_token < (1 << 24);
}

// f(blocks of 32 columns, whether rows can be loaded straight into LDS)
template <class F>
int by_shape(int64_t dim, bool aligned, F&& f) {
  auto with = [&](auto db) { return aligned ? f(db, std::true_type{}) : f(db, std::false_type{}); };
  if (dim <= 64) return with(std::integral_constant<int, 2>{});
  if (dim <= 96) return with(std::integral_constant<int, 3>{});
  return with(std::integral_constant<int, 4>{});
}

int key_rows(int64_t dim) { return dim > 96 ? 32 * kKeyWaves<4> : 32 * kKeyWaves<2>; }   // that a block of k_attn_dkv owns

// Parts that the steps of `blocks` blocks are cut into, `steps` each on average: up to 512
// blocks, of 8 steps at least: the join costs a launch.  Forward and backward, us, with parts
// of 8 steps, of 4, and whole: 32 queries over 8192 keys, 8 heads of 128, 25 and 40, 28 and
// 40, 137 and 156; causal, 1024 tokens of 32 heads of 64, 20 and 45, 27 and 63, 20 and 45;
// 2048 of 8 heads of 64 27 and 64, -, 31 and 65.  (512 is two blocks a CU.  k_attn_dkv<4>, whose
// LDS allows one, would do with half: 4096 causal tokens of 8 heads of 128 over 2 take 244 us
// backward, with 256 215.  And two parts cost more than they give where the whole would be one
// launch: 1024 tokens of 8 heads of 64 without a mask 42 us backward, whole 35.  The average is
// all that the host knows of the sequences: one long one among many short is not cut.)
int parts_of(int64_t blocks, int64_t steps, int64_t most = kMaxParts) {
  return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>({most, 512 / std::max<int64_t>(blocks, 1), steps / 8})));
}

template <class Op>
int64_t sequences_of(const Op& op) {
  return std::max<int64_t>(1, op.starts ? op.sequences : 1);
}

// Steps over the queries or keys that one of `rows` keys or queries meets, in the mean.
template <class Op>
int64_t average_steps(const Op& op, int64_t rows) {
  const int64_t q = op.tokens, k = op.k_tokens, pairs = !op.causal ? q * k : k < q ? k * k / 2 : q * (k - q / 2);
  return pairs / std::max<int64_t>(rows, 1) / sequences_of(op) / BN;
}

size_t rounded(size_t bytes) { return (bytes + 255) / 256 * 256; }

// Blocks that own queries, `each` rows a query, in `heads` heads.
template <class Op>
int64_t query_blocks(const Op& op, int64_t each, int64_t heads) {
  return std::max((op.tokens * each + BM - 1) / BM, sequences_of(op)) * heads;
}

}  // namespace

AttnPlan attention_plan(const muon_attention_t& op) {
  AttnPlan p{};
  p.packed = op.heads > op.kv_heads;      // (tokens x heads fit 32 bits)
  const int64_t each = p.packed ? op.heads / op.kv_heads : 1;
  p.parts = parts_of(query_blocks(op, each, op.heads / each), average_steps(op, op.tokens), kMaxForwardParts);
  if (p.parts > 1) {
    const size_t rows = static_cast<size_t>(p.parts) * op.tokens * op.heads;
    p.lse_off = rounded(rows * op.dim * sizeof(float));
    p.bytes = p.lse_off + rounded(rows * sizeof(float));
  }
  return p;
}

AttnGradPlan attention_grad_plan(const muon_attention_grad_t& op) {
  AttnGradPlan p{};
  const size_t q = static_cast<size_t>(op.tokens) * op.heads, k = static_cast<size_t>(op.k_tokens) * op.kv_heads;
  p.parts_q = parts_of(query_blocks(op, 1, op.heads), average_steps(op, op.tokens));
  const int own = key_rows(op.dim);
  p.parts_k = parts_of((op.k_tokens + own - 1) / own * op.kv_heads, op.heads / op.kv_heads * average_steps(op, op.k_tokens));
  const bool ragged = op.starts != nullptr;
  // (us, and in two launches: 2 x 37 tokens, 4 heads of 64, 13, 18; 512, 8 of 64, 21, 29; 1024, 16
  // of 64, 36, 45; 1024, 28 of 128, 76, 87; 32 of 128 88, 87; but 4 x 256, 32 of 128 over 8, 89, 75)
  p.one_launch = p.parts_q == 1 && p.parts_k == 1 &&
                 units_of(op.tokens, op.sequences, ragged) * op.heads + units_of(op.k_tokens, op.sequences, ragged, own) * op.kv_heads <= 512;
  if (p.one_launch) return p;
  p.dq_off = rounded(2 * q * sizeof(float));
  p.dkv_off = p.dq_off + (p.parts_q > 1 ? rounded(p.parts_q * q * op.dim * sizeof(float)) : 0);
  p.bytes = p.dkv_off + (p.parts_k > 1 ? rounded(2 * p.parts_k * k * op.dim * sizeof(float)) : 0);
  return p;
}

int launch_attention(const muon_attention_t& op, const AttnPlan& p, char* ws, void* stream) {
  const int64_t each = p.packed ? op.heads / op.kv_heads : 1;
  const uint32_t units = units_of(op.tokens * each, op.sequences, op.starts != nullptr);
  const dim3 grid(units * static_cast<uint32_t>(op.heads / each), p.parts);
  return by_shape(op.dim, aligned16(op.k) && aligned16(op.v), [&](auto db, auto al) {
    auto launch = [&](auto kernel) {
      hipLaunchKernelGGL(kernel, grid, dim3(kThreads), 0, static_cast<hipStream_t>(stream), op, units, reinterpret_cast<float*>(ws),
                         reinterpret_cast<float*>(ws + p.lse_off));
      return static_cast<int>(hipGetLastError());
    };
    return p.packed ? launch(k_attn<decltype(db)::value, decltype(al)::value, true>)
                    : launch(k_attn<decltype(db)::value, decltype(al)::value, false>);
  });
}

int launch_attention_dq(const muon_attention_grad_t& op, const AttnGradPlan& p, char* ws, void* stream) {
  const uint32_t units = units_of(op.tokens, op.sequences, op.starts != nullptr);
  return by_shape(op.dim, aligned16(op.k) && aligned16(op.v), [&](auto db, auto al) {
    hipLaunchKernelGGL((k_attn_dq<decltype(db)::value, decltype(al)::value>), dim3(units * static_cast<uint32_t>(op.heads), p.parts_q),
                       dim3(kThreads), 0, static_cast<hipStream_t>(stream), op, units, reinterpret_cast<float*>(ws),
                       reinterpret_cast<float*>(ws + p.dq_off));
    return static_cast<int>(hipGetLastError());
  });
}

int launch_attention_grad(const muon_attention_grad_t& op, void* stream) {
  const bool ragged = op.starts != nullptr, aligned = aligned16(op.k) && aligned16(op.v) && aligned16(op.q) && aligned16(op.dout);
  return by_shape(op.dim, aligned, [&](auto db, auto al) {
    constexpr int waves = kKeyWaves<decltype(db)::value>;
    const uint32_t units = units_of(op.tokens, op.sequences, ragged), k_units = units_of(op.k_tokens, op.sequences, ragged, 32 * waves);
    const uint32_t q_blocks = op.tokens ? units * static_cast<uint32_t>(op.heads) : 0, k_blocks = op.k_tokens ? k_units * static_cast<uint32_t>(op.kv_heads) : 0;
    hipLaunchKernelGGL((k_attn_grad<decltype(db)::value, decltype(al)::value>), dim3(q_blocks + k_blocks), dim3(64 * waves), 0,
                       static_cast<hipStream_t>(stream), op, units, q_blocks, k_units);
    return static_cast<int>(hipGetLastError());
  });
}

int launch_attention_dkv(const muon_attention_grad_t& op, const AttnGradPlan& p, char* ws, void* stream) {
  return by_shape(op.dim, aligned16(op.q) && aligned16(op.dout), [&](auto db, auto al) {
    constexpr int waves = kKeyWaves<decltype(db)::value>;
    const uint32_t units = units_of(op.k_tokens, op.sequences, op.starts != nullptr, 32 * waves);
    hipLaunchKernelGGL((k_attn_dkv<decltype(db)::value, decltype(al)::value>), dim3(units * static_cast<uint32_t>(op.kv_heads), p.parts_k),
                       dim3(64 * waves), 0, static_cast<hipStream_t>(stream), op, units, reinterpret_cast<const float*>(ws),
                       reinterpret_cast<float*>(ws + p.dkv_off));
    return static_cast<int>(hipGetLastError());
  });
}

namespace {
int launch_join(const Join& j, int tensors, void* stream) {
  const int64_t threads = j.rows * j.heads * (j.dim / 8);
  hipLaunchKernelGGL(k_attn_join, dim3(static_cast<unsigned>((threads + 255) / 256), tensors), dim3(256), 0, static_cast<hipStream_t>(stream), j);
  return static_cast<int>(hipGetLastError());
}
}  // namespace

int launch_attention_join(const muon_attention_t& op, const AttnPlan& p, const char* ws, void* stream) {
  Join j{};
  j.out[0] = op.o;
  j.part = reinterpret_cast<const float*>(ws);
  j.part_lse = reinterpret_cast<const float*>(ws + p.lse_off);
  j.lse = op.lse;
  j.ld_lse = op.ld_lse;
  j.starts = op.starts;
  j.sequences = op.sequences;
  j.rows = op.tokens;
  j.heads = op.heads;
  j.dim = op.dim;
  j.parts = p.parts;
  j.all[0] = op.zero_rest & MUON_ATTN_ZERO_O;
  j.all_lse = op.zero_rest & MUON_ATTN_ZERO_LSE;
  return launch_join(j, 1, stream);
}

int launch_attention_dq_join(const muon_attention_grad_t& op, const AttnGradPlan& p, const char* ws, void* stream) {
  Join j{};
  j.out[0] = op.dq;
  j.part = reinterpret_cast<const float*>(ws + p.dq_off);
  j.starts = op.starts;
  j.sequences = op.sequences;
  j.rows = op.tokens;
  j.heads = op.heads;
  j.dim = op.dim;
  j.parts = p.parts_q;
  j.factor[0] = op.scale;
  j.all[0] = op.zero_rest & MUON_ATTN_ZERO_DQ;
  return launch_join(j, 1, stream);
}

int launch_attention_dkv_join(const muon_attention_grad_t& op, const AttnGradPlan& p, const char* ws, void* stream) {
  Join j{};
  j.out[0] = op.dk;
  j.out[1] = op.dv;
  j.part = reinterpret_cast<const float*>(ws + p.dkv_off);
  j.starts = op.k_starts ? op.k_starts : op.starts;
  j.sequences = op.sequences;
  j.rows = op.k_tokens;
  j.heads = op.kv_heads;
  j.dim = op.dim;
  j.parts = p.parts_k;
  j.factor[0] = op.scale;
  j.factor[1] = 1.f;
  j.all[0] = op.zero_rest & MUON_ATTN_ZERO_DK;
  j.all[1] = op.zero_rest & MUON_ATTN_ZERO_DV;
  return launch_join(j, 2, stream);
}

}  // namespace muon
