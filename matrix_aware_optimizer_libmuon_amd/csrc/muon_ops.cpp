// Host side of the training operators (include/muon.h): argument checks,
// workspace sizes and the launch sequences.  Their arguments travel with the
// launches, so there is no descriptor table, and a stream may be capturing.
#include <hip/hip_runtime.h>

#include <cmath>
#include <initializer_list>
#include <string>
#include <utility>

#include "muon.h"
#include "muon_internal.h"
#include "muon_ops.h"

using namespace muon;

namespace {

constexpr int64_t kMaxRows = (int64_t(1) << 31) - 1;
constexpr int64_t kMaxSpan = int64_t(1) << 46;   // elements from a matrix's first to its last

bool is_aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
size_t type_size(int32_t dtype) { return dtype == MUON_BF16 ? 2 : 4; }
bool type_ok(int32_t dtype) { return dtype == MUON_F32 || dtype == MUON_BF16; }
bool size_ok(int64_t rows, int64_t cols) { return rows >= 0 && rows <= kMaxRows && cols >= 1 && cols <= MUON_MAX_DIM; }

// The bytes of a strided tensor: `rows` rows, `stride` apart, of `n` pieces of `width`
// bytes, `step` apart.  A row's pieces span a stride at most (n is 1 for a matrix).
struct Span {
  uintptr_t begin = 0;
  uint64_t rows = 0, width = 0, stride = 0, n = 1, step = 0;
  uint64_t extent() const { return (n - 1) * step + width; }
  uintptr_t end() const { return begin + (rows - 1) * stride + extent(); }
  // the same bytes with each piece a row, where rows follow each other in steps of one length
  bool even() const { return n > 1 && stride == n * step; }
  Span flat() const { return {begin, rows * n, width, step, 1, 0}; }
};

// Whether a piece of a row of b, which begins `at` bytes behind one of a, meets one of a:
// some j has -b.width < at + j step < a.width.
bool rows_meet(const Span& a, const Span& b, int64_t at) {
  const int64_t wa = static_cast<int64_t>(a.width), wb = static_cast<int64_t>(b.width), step = static_cast<int64_t>(a.n > 1 ? a.step : b.step);
  if (a.n == 1 && b.n == 1) return at < wa && at + wb > 0;
  if (a.n > 1 && b.n > 1 && a.step != b.step)   // (as if they had no gaps)
    return at < static_cast<int64_t>(a.extent()) && at + static_cast<int64_t>(b.extent()) > 0;
  const int64_t over = -wb - at, first = (over >= 0 ? over / step : -((-over + step - 1) / step)) + 1;   // the least j past the left bound
  const int64_t j = first > 1 - static_cast<int64_t>(a.n) ? first : 1 - static_cast<int64_t>(a.n);
  return j < static_cast<int64_t>(b.n) && at + j * step < wa;
}

// Slices of one buffer, rows of the same stride: the rows of b begin d + r stride bytes
// behind those of a, 0 <= d < stride, and only r = 0 and r = -1 can meet.
bool slices_meet(const Span& a, const Span& b) {
  const int64_t s = static_cast<int64_t>(a.stride), by = static_cast<int64_t>(b.begin - a.begin);
  const int64_t m = by >= 0 ? by / s : -((-by + s - 1) / s), d = by - m * s;
  // the row of b that lies r strides behind some row of a: its number less that row's is r - m
  auto there = [&](int64_t r) { return r - m > -static_cast<int64_t>(a.rows) && r - m < static_cast<int64_t>(b.rows); };
  return (there(0) && rows_meet(a, b, d)) || (there(-1) && rows_meet(a, b, d - s));
}

bool overlap(const Span& a, const Span& b) {
  if (!a.rows || !b.rows || a.end() <= b.begin || b.end() <= a.begin) return false;
  auto alike = [](const Span& x, const Span& y) { return x.rows > 1 && y.rows > 1 && x.stride == y.stride; };
  if (alike(a, b)) return slices_meet(a, b);
  if (a.even() && alike(a.flat(), b)) return slices_meet(a.flat(), b);
  if (b.even() && alike(a, b.flat())) return slices_meet(a, b.flat());
  if (a.even() && b.even() && alike(a.flat(), b.flat())) return slices_meet(a.flat(), b.flat());
  return true;
}

// Checks of one call: matrices noted as read or written, then the overlaps.
class Args {
 public:
  // A matrix; `need`: it must be there (else a null pointer means it is not).
  bool mat(const void* p, int64_t rows, int64_t cols, int64_t ld, size_t esize, bool written, bool need = true) {
    if (rows == 0) return true;
    if (!p) return !need;
    if (!is_aligned(p, esize) || (rows > 1 && (ld < cols || ld > kMaxSpan / rows))) return false;
    Span s;
    s.begin = reinterpret_cast<uintptr_t>(p);
    s.rows = static_cast<uint64_t>(rows);
    s.width = static_cast<uint64_t>(cols) * esize;
    s.stride = rows > 1 ? static_cast<uint64_t>(ld) * esize : s.width;
    note(s, written);
    return true;
  }
  bool act8(const muon_act8_t& a, int64_t rows, int64_t cols, bool written, bool need = true) {
    if (rows > 0 && !a.codes) return !need;
    if (rows > 0 && !a.scales) return false;
    return mat(a.codes, rows, cols, a.ld_codes, 1, written) &&
           mat(a.scales, rows, (cols + MUON_ACT8_GROUP - 1) / MUON_ACT8_GROUP, a.ld_scales, 1, written);
  }
  // A tokens x heads x dim tensor of bf16: each token's heads lie within a token's stride,
  // or each head's tokens within a head's.
  bool heads(const muon_heads_t& t, int64_t tokens, int64_t heads, int64_t dim, bool written) {
    const int64_t lt = t.ld_token, lh = t.ld_head;
    if (tokens == 0 || heads == 1) return mat(t.data, tokens, dim, lt, 2, written);
    if (tokens == 1) return mat(t.data, heads, dim, lh, 2, written);
    if (!t.data || !is_aligned(t.data, 2) || lt < dim || lh < dim || lt > kMaxSpan / tokens || lh > kMaxSpan / heads) return false;
    const bool by_token = lt >= (heads - 1) * lh + dim;
    if (!by_token && lh < (tokens - 1) * lt + dim) return false;
    if (lh == dim) return mat(t.data, tokens, heads * dim, lt, 2, written);
    Span s{reinterpret_cast<uintptr_t>(t.data), static_cast<uint64_t>(tokens), static_cast<uint64_t>(dim) * 2, static_cast<uint64_t>(lt) * 2,
           static_cast<uint64_t>(heads), static_cast<uint64_t>(lh) * 2};
    if (!by_token) {
      std::swap(s.rows, s.n);
      std::swap(s.stride, s.step);
    }
    note(s, written);
    return true;
  }
  bool vec(const void* p, int64_t n, size_t esize, bool written, bool need) { return n == 0 || mat(p, 1, n, n, esize, written, need); }
  bool clash() const {
    for (int i = 0; i < n_out_; ++i) {
      for (int j = 0; j < i; ++j)
        if (overlap(out_[i], out_[j])) return true;
      for (int j = 0; j < n_in_; ++j)
        if (overlap(out_[i], in_[j])) return true;
    }
    return false;
  }

 private:
  void note(const Span& s, bool written) { (written ? out_ : in_)[written ? n_out_++ : n_in_++] = s; }
  Span in_[12], out_[10];   // more than any call notes
  int n_in_ = 0, n_out_ = 0;
};

// A call's stream: on the current device; under MUON_DEBUG (and not capturing)
// each launch is waited for and checked.
class Launcher {
 public:
  explicit Launcher(hipStream_t stream) : stream_(stream) {}
  int open() {
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return host_hip_fail(e, "hipGetDevice");
    // (the null stream is the current device's)
    if (stream_ && !host_stream_on_device(stream_, dev)) return MUON_EINVAL;
    if (host_debug()) {
      hipStreamCaptureStatus cap = hipStreamCaptureStatusNone;
      e = hipStreamIsCapturing(stream_, &cap);
      if (e != hipSuccess) return host_hip_fail(e, "hipStreamIsCapturing");
      debug_ = cap == hipStreamCaptureStatusNone;
    }
    return MUON_OK;
  }
  template <class F>
  int run(const char* what, F&& launch) {
    int e = launch(static_cast<void*>(stream_));
    if (e == hipSuccess && debug_) e = hipStreamSynchronize(stream_);
    return e == hipSuccess ? MUON_OK : host_hip_fail(e, what);
  }
  // MUON_DEBUG: a value that no kernel of the call wrote shows up as NaN
  int poison(void* workspace, size_t bytes) {
    if (!debug_ || bytes < 4) return MUON_OK;
    return run("workspace fill", [&](void* st) {
      return launch_fill_u32(static_cast<uint32_t*>(workspace), static_cast<int64_t>(bytes / 4), 0x7FC07FC0u, st);
    });
  }

 private:
  hipStream_t stream_;
  bool debug_ = false;
};

bool workspace_ok(const void* ws, size_t have, size_t need) {
  return need == 0 || (ws && have >= need && is_aligned(ws, 256));
}

// Sizes and options that both directions of attention have.
template <class Op>
bool attention_ok(const Op* op, int32_t zero_bits) {
  constexpr int64_t max_tokens = int64_t(1) << 30, max_blocks = int64_t(1) << 22;
  if (!op || op->reserved || op->tokens < 0 || op->tokens > max_tokens || op->k_tokens < 0 || op->k_tokens > max_tokens ||
      op->heads < 1 || op->heads > max_blocks || op->kv_heads < 1 || op->heads % op->kv_heads || op->dim < 8 ||
      op->dim > MUON_ATTN_MAX_DIM || op->dim % 8 || !(op->scale > 0.f) || !(op->scale <= 1e30f) ||
      (op->causal != 0 && op->causal != 1) || (op->zero_rest & ~zero_bits))
    return false;
  if (!op->starts ? op->k_starts != nullptr
                  : op->sequences < 0 || op->sequences > max_blocks || (!op->k_starts && op->tokens != op->k_tokens))
    return false;
  const int64_t rows = op->tokens > op->k_tokens ? op->tokens : op->k_tokens;
  return (rows / 128 + (op->starts ? op->sequences : 0) + 2) * op->heads <= max_blocks;
}

// Strides of axes of length one are not read: the kernels get ones that fit.
muon_heads_t heads_strides(muon_heads_t t, int64_t tokens, int64_t heads) {
  if (tokens <= 1) t.ld_token = MUON_ATTN_MAX_DIM;
  if (heads <= 1) t.ld_head = 0;
  return t;
}

template <class Op>
bool note_starts(Args& a, const Op* op) {
  return a.vec(op->starts, op->starts ? op->sequences + 1 : 0, 4, false, false) &&
         a.vec(op->k_starts, op->k_starts ? op->sequences + 1 : 0, 4, false, false);
}

}  // namespace

extern "C" {

int muon_act8_pack(const void* x, int64_t ld_x, int32_t dtype, int64_t rows, int64_t cols,
                   const muon_act8_t* out, hipStream_t stream) {
  Args a;
  if (!out || !type_ok(dtype) || !size_ok(rows, cols) || !a.mat(x, rows, cols, ld_x, type_size(dtype), false) ||
      !a.act8(*out, rows, cols, true))
    return MUON_EINVAL;
  if (a.clash()) return MUON_EALIAS;
  if (rows == 0) return MUON_OK;
  Launcher l(stream);
  if (int rc = l.open()) return rc;
  return l.run("8-bit pack", [&](void* st) { return launch_act8_pack(x, ld_x, dtype, rows, cols, *out, st); });
}

int muon_act8_unpack(const muon_act8_t* in, int64_t rows, int64_t cols, void* out, int64_t ld_out,
                     int32_t dtype, hipStream_t stream) {
  Args a;
  if (!in || !type_ok(dtype) || !size_ok(rows, cols) || !a.act8(*in, rows, cols, false) ||
      !a.mat(out, rows, cols, ld_out, type_size(dtype), true))
    return MUON_EINVAL;
  if (a.clash()) return MUON_EALIAS;
  if (rows == 0) return MUON_OK;
  Launcher l(stream);
  if (int rc = l.open()) return rc;
  return l.run("8-bit unpack", [&](void* st) { return launch_act8_unpack(*in, rows, cols, out, ld_out, dtype, st); });
}

int muon_rmsnorm_act8(const muon_rmsnorm_t* op, hipStream_t stream) {
  Args a;
  if (!op || !type_ok(op->dtype) || !size_ok(op->rows, op->cols) || op->cols > MUON_NORM_MAX_COLS) return MUON_EINVAL;
  if (!(op->eps >= 0.f) || !std::isfinite(op->eps)) return MUON_EINVAL;
  const size_t es = type_size(op->dtype);
  const int64_t rows = op->rows, cols = op->cols;
  if (!a.mat(op->x, rows, cols, op->ld_x, es, false) || !a.mat(op->residual, rows, cols, op->ld_residual, es, false, false) ||
      !a.vec(op->gain, cols, 4, false, false) || !a.mat(op->h, rows, cols, op->ld_h, es, true, false) ||
      !a.mat(op->y, rows, cols, op->ld_y, es, true, false) || !a.act8(op->n, rows, cols, true, false) ||
      !a.vec(op->rstd, rows, 4, true, false))
    return MUON_EINVAL;
  if (a.clash()) return MUON_EALIAS;
  if (rows == 0) return MUON_OK;
  Launcher l(stream);
  if (int rc = l.open()) return rc;
  return l.run("RMS norm", [&](void* st) { return launch_rmsnorm(*op, st); });
}

size_t muon_rmsnorm_act8_grad_workspace_bytes(int64_t rows, int64_t cols) {
  if (!size_ok(rows, cols) || cols > MUON_NORM_MAX_COLS) return 0;
  const int64_t blocks = rmsnorm_grad_blocks(rows, cols);
  return blocks > 1 ? static_cast<size_t>(blocks) * static_cast<size_t>(cols) * sizeof(float) : 0;
}

int muon_rmsnorm_act8_grad(const muon_rmsnorm_grad_t* op, void* workspace, size_t workspace_bytes,
                           hipStream_t stream) {
  Args a;
  if (!op || op->reserved || !type_ok(op->dtype) || !size_ok(op->rows, op->cols) || op->cols > MUON_NORM_MAX_COLS)
    return MUON_EINVAL;
  const size_t es = type_size(op->dtype);
  const int64_t rows = op->rows, cols = op->cols;
  if (!a.mat(op->dy, rows, cols, op->ld_dy, es, false) || !a.mat(op->dres, rows, cols, op->ld_dres, es, false, false) ||
      !a.vec(op->gain, cols, 4, false, false) || !a.vec(op->rstd, rows, 4, false, true) ||
      !a.act8(op->n, rows, cols, false) || !a.mat(op->dx, rows, cols, op->ld_dx, es, true) ||
      !a.vec(op->dgain, cols, 4, true, false))
    return MUON_EINVAL;
  const size_t need = op->dgain ? muon_rmsnorm_act8_grad_workspace_bytes(rows, cols) : 0;
  if (!workspace_ok(workspace, workspace_bytes, need)) return MUON_EWORKSPACE;
  if (need && !a.mat(workspace, 1, static_cast<int64_t>(need), 0, 1, true)) return MUON_EWORKSPACE;
  if (a.clash()) return MUON_EALIAS;
  if (rows == 0 && !op->dgain) return MUON_OK;
  Launcher l(stream);
  if (int rc = l.open()) return rc;
  if (int rc = l.poison(workspace, need)) return rc;
  float* partial = static_cast<float*>(workspace);
  const int64_t blocks = rmsnorm_grad_blocks(rows, cols);
  if (rows > 0)
    if (int rc = l.run("RMS norm gradient", [&](void* st) { return launch_rmsnorm_grad(*op, partial, st); })) return rc;
  if (op->dgain && blocks != 1)
    return l.run("RMS norm gain gradient", [&](void* st) { return launch_rmsnorm_dgain(partial, blocks, cols, op->dgain, st); });
  return MUON_OK;
}

int muon_swiglu_act8(const muon_swiglu_t* op, hipStream_t stream) {
  Args a;
  if (!op || op->reserved || !type_ok(op->dtype) || !size_ok(op->rows, op->cols)) return MUON_EINVAL;
  if (!op->gate8.codes != !op->up8.codes) return MUON_EINVAL;
  const size_t es = type_size(op->dtype);
  const int64_t rows = op->rows, cols = op->cols;
  if (!a.mat(op->gate, rows, cols, op->ld_gate, es, false) || !a.mat(op->up, rows, cols, op->ld_up, es, false) ||
      !a.mat(op->a, rows, cols, op->ld_a, es, true, false) || !a.act8(op->gate8, rows, cols, true, false) ||
      !a.act8(op->up8, rows, cols, true, false))
    return MUON_EINVAL;
  if (a.clash()) return MUON_EALIAS;
  if (rows == 0) return MUON_OK;
  Launcher l(stream);
  if (int rc = l.open()) return rc;
  return l.run("gated unit", [&](void* st) { return launch_swiglu(*op, st); });
}

int muon_swiglu_act8_grad(const muon_swiglu_grad_t* op, hipStream_t stream) {
  Args a;
  if (!op || op->reserved || !type_ok(op->dtype) || !size_ok(op->rows, op->cols)) return MUON_EINVAL;
  const size_t es = type_size(op->dtype);
  const int64_t rows = op->rows, cols = op->cols;
  if (!a.mat(op->da, rows, cols, op->ld_da, es, false) || !a.act8(op->gate8, rows, cols, false) ||
      !a.act8(op->up8, rows, cols, false) || !a.mat(op->dgate, rows, cols, op->ld_dgate, es, true) ||
      !a.mat(op->dup, rows, cols, op->ld_dup, es, true) || !a.act8(op->a8, rows, cols, true, false))
    return MUON_EINVAL;
  if (a.clash()) return MUON_EALIAS;
  if (rows == 0) return MUON_OK;
  Launcher l(stream);
  if (int rc = l.open()) return rc;
  return l.run("gated unit gradient", [&](void* st) { return launch_swiglu_grad(*op, st); });
}

static bool wgrad_sizes_ok(const muon_act8_wgrad_t* op) {
  return op && type_ok(op->dw_dtype) && op->tokens >= 0 && op->tokens <= kMaxRows && op->n >= 1 &&
         op->n <= MUON_MAX_DIM && op->k >= 1 && op->k <= MUON_MAX_DIM;
}

// The row strides of a single row are not read: the kernel gets ones that fit.
static muon_act8_wgrad_t wgrad_strides(const muon_act8_wgrad_t* op) {
  muon_act8_wgrad_t r = *op;
  if (r.tokens <= 1) {
    r.ld_dy = (r.n + 7) / 8 * 8;
    r.x8.ld_codes = (r.k + 15) / 16 * 16;
    r.x8.ld_scales = (r.k + 31) / 32;
  }
  return r;
}

size_t muon_act8_wgrad_workspace_bytes(const muon_act8_wgrad_t* op) {
  if (!wgrad_sizes_ok(op)) return 0;
  const muon_act8_wgrad_t in = wgrad_strides(op);
  if (in.ld_dy < in.n || in.x8.ld_codes < in.k || in.x8.ld_scales < (in.k + 31) / 32) return 0;
  return wgrad_plan(in).bytes;
}

int muon_act8_wgrad(const muon_act8_wgrad_t* op, void* workspace, size_t workspace_bytes,
                    hipStream_t stream) {
  Args a;
  if (!wgrad_sizes_ok(op) || (op->accumulate != 0 && op->accumulate != 1)) return MUON_EINVAL;
  if (!a.mat(op->dy, op->tokens, op->n, op->ld_dy, 2, false) || !a.act8(op->x8, op->tokens, op->k, false) ||
      !a.vec(op->col_gain, op->k, 4, false, false) ||
      !a.mat(op->dw, op->n, op->k, op->ld_dw, type_size(op->dw_dtype), true))
    return MUON_EINVAL;
  muon_act8_wgrad_t in = wgrad_strides(op);
  const WgradPlan p = wgrad_plan(in);
  if (!workspace_ok(workspace, workspace_bytes, p.bytes)) return MUON_EWORKSPACE;
  if (p.bytes && !a.mat(workspace, 1, static_cast<int64_t>(p.bytes), 0, 1, true)) return MUON_EWORKSPACE;
  if (a.clash()) return MUON_EALIAS;
  if (op->tokens == 0 && op->accumulate) return MUON_OK;
  Launcher l(stream);
  if (int rc = l.open()) return rc;
  if (int rc = l.poison(workspace, p.bytes)) return rc;
  char* ws = static_cast<char*>(workspace);
  if (p.copy_dy || p.copy_x)
    if (int rc = l.run("weight gradient, aligned copies", [&](void* st) { return launch_wgrad_copy(in, p, ws, st); })) return rc;
  if (op->tokens > 0)
    if (int rc = l.run("weight gradient", [&](void* st) { return launch_wgrad(in, p, ws, st); })) return rc;
  if (p.splits != 1)     // several ranges, or no tokens
    return l.run("weight gradient, join", [&](void* st) { return launch_wgrad_join(in, p, ws, st); });
  return MUON_OK;
}

int muon_embed(const muon_embed_t* op, hipStream_t stream) {
  Args a;
  if (!op || !type_ok(op->table_dtype) || !type_ok(op->out_dtype) || !size_ok(op->tokens, op->cols) ||
      op->vocab < 1 || op->vocab > kMaxRows - 1 || !std::isfinite(op->scale) || (op->id_bytes != 4 && op->id_bytes != 8))
    return MUON_EINVAL;
  if (!a.mat(op->table, op->vocab, op->cols, op->ld_table, type_size(op->table_dtype), false) ||
      !a.vec(op->ids, op->tokens, op->id_bytes, false, true) ||
      !a.mat(op->out, op->tokens, op->cols, op->ld_out, type_size(op->out_dtype), true))
    return MUON_EINVAL;
  if (a.clash()) return MUON_EALIAS;
  if (op->tokens == 0) return MUON_OK;
  Launcher l(stream);
  if (int rc = l.open()) return rc;
  return l.run("embedding lookup", [&](void* st) { return launch_embed(*op, st); });
}

size_t muon_embed_grad_workspace_bytes(int64_t tokens, int64_t vocab, int64_t cols) {
  if (!size_ok(tokens, cols) || vocab < 1 || vocab > kMaxRows - 1) return 0;
  return embed_sort_plan(tokens, vocab, cols).bytes;
}

int muon_embed_grad(const muon_embed_grad_t* op, void* workspace, size_t workspace_bytes,
                    hipStream_t stream) {
  Args a;
  if (!op || op->reserved || !type_ok(op->dy_dtype) || !type_ok(op->table_dtype) || !size_ok(op->tokens, op->cols) ||
      op->vocab < 1 || op->vocab > kMaxRows - 1 || !std::isfinite(op->scale) || (op->id_bytes != 4 && op->id_bytes != 8) ||
      (op->accumulate != 0 && op->accumulate != 1))
    return MUON_EINVAL;
  if (!a.mat(op->dy, op->tokens, op->cols, op->ld_dy, type_size(op->dy_dtype), false) ||
      !a.vec(op->ids, op->tokens, op->id_bytes, false, true) ||
      !a.mat(op->dtable, op->vocab, op->cols, op->ld_dtable, type_size(op->table_dtype), true))
    return MUON_EINVAL;
  const EmbedSortPlan p = embed_sort_plan(op->tokens, op->vocab, op->cols);
  if (!workspace_ok(workspace, workspace_bytes, p.bytes)) return MUON_EWORKSPACE;
  if (p.bytes && !a.mat(workspace, 1, static_cast<int64_t>(p.bytes), 0, 1, true)) return MUON_EWORKSPACE;
  if (a.clash()) return MUON_EALIAS;
  if (op->tokens == 0 && op->accumulate) return MUON_OK;
  Launcher l(stream);
  if (int rc = l.open()) return rc;
  if (int rc = l.poison(workspace, p.bytes)) return rc;
  char* ws = static_cast<char*>(workspace);
  if (p.passes == 0)
    return l.run("embedding gradient", [&](void* st) { return launch_embed_sums(*op, p, ws, st); });
  if (p.log_buckets) {
    if (int rc = l.run("token sort", [&](void* st) { return launch_embed_buckets(*op, p, ws, st); })) return rc;
  } else {
    for (int pass = 0; pass < p.passes; ++pass) {
      if (int rc = l.run("token sort, count", [&](void* st) { return launch_embed_count(*op, p, pass, ws, st); })) return rc;
      if (int rc = l.run("token sort, scatter", [&](void* st) { return launch_embed_scatter(*op, p, pass, ws, st); })) return rc;
    }
    if (int rc = l.run("embedding gradient, starts", [&](void* st) { return launch_embed_starts(*op, p, ws, st); })) return rc;
  }
  if (int rc = l.run("embedding gradient, sums", [&](void* st) { return launch_embed_sums(*op, p, ws, st); })) return rc;
  return l.run("embedding gradient, join", [&](void* st) { return launch_embed_join(*op, p, ws, st); });
}

size_t muon_attention_workspace_bytes(const muon_attention_t* op) {
  return attention_ok(op, MUON_ATTN_ZERO_O | MUON_ATTN_ZERO_LSE) ? attention_plan(*op).bytes : 0;
}

int muon_attention(const muon_attention_t* op, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  Args a;
  if (!attention_ok(op, MUON_ATTN_ZERO_O | MUON_ATTN_ZERO_LSE)) return MUON_EINVAL;
  const int64_t n = op->tokens, nk = op->k_tokens;
  if (!a.heads(op->q, n, op->heads, op->dim, false) || !a.heads(op->k, nk, op->kv_heads, op->dim, false) ||
      !a.heads(op->v, nk, op->kv_heads, op->dim, false) || !a.heads(op->o, n, op->heads, op->dim, true) ||
      (n > 0 && !a.mat(op->lse, op->heads, n, op->ld_lse, 4, true, false)) || !note_starts(a, op))
    return MUON_EINVAL;
  const AttnPlan p = attention_plan(*op);
  if (!workspace_ok(workspace, workspace_bytes, p.bytes)) return MUON_EWORKSPACE;
  if (p.bytes && !a.mat(workspace, 1, static_cast<int64_t>(p.bytes), 0, 1, true)) return MUON_EWORKSPACE;
  if (a.clash()) return MUON_EALIAS;
  if (n == 0) return MUON_OK;
  muon_attention_t in = *op;
  in.q = heads_strides(op->q, n, op->heads);
  in.o = heads_strides(op->o, n, op->heads);
  in.k = heads_strides(op->k, nk, op->kv_heads);
  in.v = heads_strides(op->v, nk, op->kv_heads);
  Launcher l(stream);
  if (int rc = l.open()) return rc;
  if (int rc = l.poison(workspace, p.bytes)) return rc;
  char* ws = static_cast<char*>(workspace);
  if (int rc = l.run("attention", [&](void* st) { return launch_attention(in, p, ws, st); })) return rc;
  if (p.parts == 1) return MUON_OK;
  return l.run("attention, join", [&](void* st) { return launch_attention_join(in, p, ws, st); });
}

static constexpr int32_t kGradZeros = MUON_ATTN_ZERO_DQ | MUON_ATTN_ZERO_DK | MUON_ATTN_ZERO_DV;

size_t muon_attention_grad_workspace_bytes(const muon_attention_grad_t* op) {
  return attention_ok(op, kGradZeros) ? attention_grad_plan(*op).bytes : 0;
}

int muon_attention_grad(const muon_attention_grad_t* op, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  Args a;
  if (!attention_ok(op, kGradZeros)) return MUON_EINVAL;
  const int64_t n = op->tokens, nk = op->k_tokens, h = op->heads, kv = op->kv_heads, d = op->dim;
  if (!a.heads(op->dout, n, h, d, false) || !a.heads(op->q, n, h, d, false) || !a.heads(op->o, n, h, d, false) ||
      !a.heads(op->k, nk, kv, d, false) || !a.heads(op->v, nk, kv, d, false) || !a.heads(op->dq, n, h, d, true) ||
      !a.heads(op->dk, nk, kv, d, true) || !a.heads(op->dv, nk, kv, d, true) ||
      (n > 0 && !a.mat(op->lse, h, n, op->ld_lse, 4, false)) || !note_starts(a, op))
    return MUON_EINVAL;
  const AttnGradPlan p = attention_grad_plan(*op);
  if (!workspace_ok(workspace, workspace_bytes, p.bytes)) return MUON_EWORKSPACE;
  if (p.bytes && !a.mat(workspace, 1, static_cast<int64_t>(p.bytes), 0, 1, true)) return MUON_EWORKSPACE;
  if (a.clash()) return MUON_EALIAS;
  if (n == 0 && nk == 0) return MUON_OK;
  muon_attention_grad_t in = *op;
  for (muon_heads_t* t : {&in.dout, &in.q, &in.o, &in.dq}) *t = heads_strides(*t, n, h);
  for (muon_heads_t* t : {&in.k, &in.v, &in.dk, &in.dv}) *t = heads_strides(*t, nk, kv);
  Launcher l(stream);
  if (int rc = l.open()) return rc;
  if (int rc = l.poison(workspace, p.bytes)) return rc;
  char* ws = static_cast<char*>(workspace);
  if (p.one_launch) return l.run("attention gradient", [&](void* st) { return launch_attention_grad(in, st); });
  if (n > 0) {
    if (int rc = l.run("attention gradient, queries", [&](void* st) { return launch_attention_dq(in, p, ws, st); })) return rc;
    if (p.parts_q > 1)
      if (int rc = l.run("attention gradient, queries' join", [&](void* st) { return launch_attention_dq_join(in, p, ws, st); })) return rc;
  }
  if (nk == 0) return MUON_OK;
  if (int rc = l.run("attention gradient, keys", [&](void* st) { return launch_attention_dkv(in, p, ws, st); })) return rc;
  if (p.parts_k == 1) return MUON_OK;
  return l.run("attention gradient, keys' join", [&](void* st) { return launch_attention_dkv_join(in, p, ws, st); });
}

static bool temperature_ok(float t) { return t >= 1e-6f && t <= 1e6f; }

int muon_distill(const muon_distill_t* op, hipStream_t stream) {
  Args a;
  if (!op || !type_ok(op->dtype) || !type_ok(op->teacher_dtype) || !size_ok(op->tokens, op->vocab) || op->top < 1 ||
      op->top > MUON_DISTILL_MAX_TOP || (op->id_bytes != 4 && op->id_bytes != 8) || !temperature_ok(op->temperature))
    return MUON_EINVAL;
  const int64_t n = op->tokens;
  const size_t es = type_size(op->dtype);
  if (!a.mat(op->logits, n, op->vocab, op->ld_logits, es, false) || !a.mat(op->ids, n, op->top, op->ld_ids, op->id_bytes, false) ||
      !a.mat(op->teacher, n, op->top, op->ld_teacher, type_size(op->teacher_dtype), false) ||
      !a.vec(op->weights, n, 4, false, false) || !a.vec(op->loss, n, 4, true, true) ||
      !a.mat(op->dlogits, n, op->vocab, op->ld_dlogits, es, true, false))
    return MUON_EINVAL;
  if (a.clash()) return MUON_EALIAS;
  if (n == 0) return MUON_OK;
  Launcher l(stream);
  if (int rc = l.open()) return rc;
  return l.run("distillation loss", [&](void* st) { return launch_distill(*op, st); });
}

int muon_policy(const muon_policy_t* op, hipStream_t stream) {
  Args a;
  if (!op || !type_ok(op->dtype) || !size_ok(op->tokens, op->vocab) || (op->id_bytes != 4 && op->id_bytes != 8) ||
      !temperature_ok(op->temperature) || !(op->clip_low >= 0.f && op->clip_low <= 1.f) || !(op->clip_high >= 0.f) ||
      !std::isfinite(op->clip_high) || !std::isfinite(op->kl_coef))
    return MUON_EINVAL;
  const int64_t n = op->tokens;
  const size_t es = type_size(op->dtype);
  if (!a.mat(op->logits, n, op->vocab, op->ld_logits, es, false) || !a.vec(op->actions, n, op->id_bytes, false, true) ||
      !a.vec(op->old_logp, n, 4, false, true) || !a.vec(op->advantages, n, 4, false, true) ||
      !a.vec(op->ref_logp, n, 4, false, false) || !a.vec(op->weights, n, 4, false, false) || !a.vec(op->loss, n, 4, true, true) ||
      !a.vec(op->logp, n, 4, true, false) || !a.mat(op->dlogits, n, op->vocab, op->ld_dlogits, es, true, false))
    return MUON_EINVAL;
  if (a.clash()) return MUON_EALIAS;
  if (n == 0) return MUON_OK;
  Launcher l(stream);
  if (int rc = l.open()) return rc;
  return l.run("policy loss", [&](void* st) { return launch_policy(*op, st); });
}

}  // extern "C"
