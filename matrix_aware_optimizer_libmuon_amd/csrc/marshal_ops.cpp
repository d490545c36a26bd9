// Argument marshalling of the training operators (ops.py): checks the tensors,
// allocates what the caller did not give, fills the C structs of include/muon.h
// and makes the call through the library's own entry, whose address bind_ops()
// was given.  Everything runs on the tensors' device and its current stream
// (ops.py makes another stream current first), so that memory allocated here
// belongs to the stream that uses it.  In C++ because the smallest calls take
// the GPU a few microseconds, less than Python needs to read as many tensor
// attributes.
//
// Errors raise ValueError (structure) or TypeError (element type) naming the
// argument; a call's status is returned with its outputs.
#include <torch/extension.h>

#include <ATen/hip/EmptyTensor.h>
#include <ATen/hip/impl/HIPStreamMasqueradingAsCUDA.h>
#include <c10/core/DeviceGuard.h>

#include <cstdint>
#include <map>
#include <string>
#include <tuple>

#include "muon.h"

namespace {

namespace py = pybind11;
using OptTensor = c10::optional<at::Tensor>;

struct Entries {
  decltype(&muon_act8_pack) act8_pack = nullptr;
  decltype(&muon_act8_unpack) act8_unpack = nullptr;
  decltype(&muon_rmsnorm_act8) rmsnorm = nullptr;
  decltype(&muon_rmsnorm_act8_grad_workspace_bytes) rmsnorm_grad_ws = nullptr;
  decltype(&muon_rmsnorm_act8_grad) rmsnorm_grad = nullptr;
  decltype(&muon_swiglu_act8) swiglu = nullptr;
  decltype(&muon_swiglu_act8_grad) swiglu_grad = nullptr;
  decltype(&muon_act8_wgrad_workspace_bytes) wgrad_ws = nullptr;
  decltype(&muon_act8_wgrad) wgrad = nullptr;
  decltype(&muon_embed) embed = nullptr;
  decltype(&muon_embed_grad_workspace_bytes) embed_grad_ws = nullptr;
  decltype(&muon_embed_grad) embed_grad = nullptr;
} g_entry;

void bind_ops(const std::map<std::string, uintptr_t>& at) {
  auto get = [&](const char* name, auto& fn) { fn = reinterpret_cast<std::decay_t<decltype(fn)>>(at.at(name)); };
  get("muon_act8_pack", g_entry.act8_pack);
  get("muon_act8_unpack", g_entry.act8_unpack);
  get("muon_rmsnorm_act8", g_entry.rmsnorm);
  get("muon_rmsnorm_act8_grad_workspace_bytes", g_entry.rmsnorm_grad_ws);
  get("muon_rmsnorm_act8_grad", g_entry.rmsnorm_grad);
  get("muon_swiglu_act8", g_entry.swiglu);
  get("muon_swiglu_act8_grad", g_entry.swiglu_grad);
  get("muon_act8_wgrad_workspace_bytes", g_entry.wgrad_ws);
  get("muon_act8_wgrad", g_entry.wgrad);
  get("muon_embed", g_entry.embed);
  get("muon_embed_grad_workspace_bytes", g_entry.embed_grad_ws);
  get("muon_embed_grad", g_entry.embed_grad);
}

[[noreturn]] void bad_value(const char* name, const std::string& what) { throw py::value_error(std::string(name) + " " + what); }
[[noreturn]] void bad_type(const char* name, const std::string& what) { throw py::type_error(std::string(name) + " " + what); }

std::string sizes(int64_t r, int64_t c) { return "(" + std::to_string(r) + ", " + std::to_string(c) + ")"; }

// The call's device (that of its first tensor), made current for its duration.
class Call {
 public:
  explicit Call(const at::Tensor& first, const char* name) : device_(first.device()) {
    if (!first.is_cuda()) bad_value(name, "must be a GPU tensor");
    if (!g_entry.embed_grad) throw std::runtime_error("the library's entries are not bound");
    guard_.reset_device(device_);
  }
  hipStream_t stream() const { return c10::hip::getCurrentHIPStreamMasqueradingAsCUDA(device_.index()).stream(); }
  const c10::Device& device() const { return device_; }
  // (the allocation alone: about 0.2 us less than at::empty with its dispatcher)
  at::Tensor empty(at::IntArrayRef size, at::ScalarType t) const {
    return at::Tensor(at::detail::empty_cuda(size, t, device_, c10::nullopt));
  }
  // a workspace of n bytes (torch aligns allocations to 256 bytes and more)
  at::Tensor workspace(size_t n) const { return n ? empty({static_cast<int64_t>(n)}, at::kByte) : at::Tensor(); }
  void on_device(const at::Tensor& t, const char* name) const {
    if (!t.is_cuda()) bad_value(name, "must be a GPU tensor");
    if (t.device() != device_) bad_value(name, "is on another device than the first tensor");
  }
  // 2-D with unit column stride; returns the row stride
  int64_t matrix(const at::Tensor& t, const char* name, int64_t rows = -1, int64_t cols = -1) const {
    if (t.dim() != 2) bad_value(name, "must be 2-D");
    on_device(t, name);
    if ((rows >= 0 && t.size(0) != rows) || (cols >= 0 && t.size(1) != cols))
      bad_value(name, "must have shape " + sizes(rows < 0 ? t.size(0) : rows, cols < 0 ? t.size(1) : cols) + ", got " + sizes(t.size(0), t.size(1)));
    if (t.size(1) < 1) bad_value(name, "must have a column");
    if (t.size(1) > 1 && t.stride(1) != 1) bad_value(name, "must have unit column stride");
    if (t.size(0) > 1 && t.stride(0) < t.size(1)) bad_value(name, "must have rows that do not overlap");
    return t.size(0) > 1 ? t.stride(0) : t.size(1);
  }
  float* fp32_vector(const at::Tensor& t, const char* name, int64_t n) const {
    on_device(t, name);
    if (t.scalar_type() != at::kFloat) bad_type(name, "must be float32");
    if (t.dim() != 1 || t.size(0) != n || !t.is_contiguous()) bad_value(name, "must be a contiguous vector of " + std::to_string(n));
    return t.data_ptr<float>();
  }

 private:
  c10::Device device_;
  c10::OptionalDeviceGuard guard_;
};

int32_t code_of(at::ScalarType t, const char* name) {
  if (t == at::kFloat) return MUON_F32;
  if (t == at::kBFloat16) return MUON_BF16;
  bad_type(name, "must be float32 or bfloat16");
}
void same_type(const at::Tensor& t, const at::Tensor& as, const char* name, const char* as_name) {
  if (t.scalar_type() != as.scalar_type()) bad_type(name, std::string("must have the type of ") + as_name);
}

int64_t groups_of(int64_t cols) { return (cols + MUON_ACT8_GROUP - 1) / MUON_ACT8_GROUP; }

// (codes, scales) of a rows x cols matrix, read from or written to.
muon_act8_t act8(const Call& c, const at::Tensor& codes, const at::Tensor& scales, const char* name, int64_t rows, int64_t cols) {
  muon_act8_t a;
  a.ld_codes = c.matrix(codes, name, rows, cols);
  a.ld_scales = c.matrix(scales, (std::string(name) + ".scales").c_str(), rows, groups_of(cols));
  if (codes.scalar_type() != at::kFloat8_e4m3fn) bad_type(name, "must have codes of float8_e4m3fn");
  if (scales.scalar_type() != at::kByte) bad_type(name, "must have scales of uint8");
  a.codes = static_cast<uint8_t*>(codes.data_ptr());
  a.scales = static_cast<uint8_t*>(scales.data_ptr());
  return a;
}

// New ones: rows of codes padded to whole groups, which keeps them 32-byte aligned.
std::pair<at::Tensor, at::Tensor> new_act8(const Call& c, int64_t rows, int64_t cols) {
  const int64_t g = groups_of(cols);
  at::Tensor codes = c.empty({rows, g * MUON_ACT8_GROUP}, at::kFloat8_e4m3fn);
  if (cols % MUON_ACT8_GROUP) codes = codes.narrow(1, 0, cols);
  return {codes, c.empty({rows, g}, at::kByte)};
}

using Codes = std::tuple<at::Tensor, at::Tensor>;

py::tuple act8_pack(const at::Tensor& x) {
  Call c(x, "x");
  const int64_t ld = c.matrix(x, "x"), rows = x.size(0), cols = x.size(1);
  const int32_t dt = code_of(x.scalar_type(), "x");
  auto [codes, scales] = new_act8(c, rows, cols);
  const muon_act8_t out = act8(c, codes, scales, "out", rows, cols);
  const int st = g_entry.act8_pack(x.data_ptr(), ld, dt, rows, cols, &out, c.stream());
  return py::make_tuple(st, codes, scales);
}

py::tuple act8_unpack(const Codes& x8, at::ScalarType dtype) {
  const auto& [codes, scales] = x8;
  Call c(codes, "x8");
  if (codes.dim() != 2) bad_value("x8", "must be 2-D");
  const int64_t rows = codes.size(0), cols = codes.size(1);
  const muon_act8_t in = act8(c, codes, scales, "x8", rows, cols);
  const int32_t dt = code_of(dtype, "dtype");
  const at::Tensor out = c.empty({rows, cols}, dtype);
  const int st = g_entry.act8_unpack(&in, rows, cols, out.data_ptr(), cols, dt, c.stream());
  return py::make_tuple(st, out);
}

py::tuple rmsnorm(const at::Tensor& x, const OptTensor& gain, const OptTensor& residual, double eps, bool save) {
  Call c(x, "x");
  muon_rmsnorm_t op{};
  op.ld_x = c.matrix(x, "x");
  op.rows = x.size(0);
  op.cols = x.size(1);
  op.dtype = code_of(x.scalar_type(), "x");
  op.eps = static_cast<float>(eps);
  op.x = x.data_ptr();
  if (gain) op.gain = c.fp32_vector(*gain, "gain", op.cols);
  at::Tensor h = x, codes, scales, rstd;
  if (residual) {
    op.ld_residual = c.matrix(*residual, "residual", op.rows, op.cols);
    same_type(*residual, x, "residual", "x");
    op.residual = residual->data_ptr();
    h = c.empty({op.rows, op.cols}, x.scalar_type());
    op.h = h.data_ptr();
    op.ld_h = op.cols;
  }
  const at::Tensor y = c.empty({op.rows, op.cols}, x.scalar_type());
  op.y = y.data_ptr();
  op.ld_y = op.cols;
  if (save) {
    std::tie(codes, scales) = new_act8(c, op.rows, op.cols);
    op.n = act8(c, codes, scales, "n", op.rows, op.cols);
    rstd = c.empty({op.rows}, at::kFloat);
    op.rstd = rstd.data_ptr<float>();
  }
  const int st = g_entry.rmsnorm(&op, c.stream());
  if (!save) return py::make_tuple(st, h, y);
  return py::make_tuple(st, h, y, codes, scales, rstd);
}

py::tuple rmsnorm_grad(const at::Tensor& dy, const Codes& n8, const at::Tensor& rstd, const OptTensor& gain,
                       const OptTensor& dres, bool want_dgain) {
  Call c(dy, "dy");
  muon_rmsnorm_grad_t op{};
  op.ld_dy = c.matrix(dy, "dy");
  op.rows = dy.size(0);
  op.cols = dy.size(1);
  op.dtype = code_of(dy.scalar_type(), "dy");
  op.dy = dy.data_ptr();
  op.n = act8(c, std::get<0>(n8), std::get<1>(n8), "n8", op.rows, op.cols);
  op.rstd = c.fp32_vector(rstd, "rstd", op.rows);
  if (gain) op.gain = c.fp32_vector(*gain, "gain", op.cols);
  if (dres) {
    op.ld_dres = c.matrix(*dres, "dres", op.rows, op.cols);
    same_type(*dres, dy, "dres", "dy");
    op.dres = dres->data_ptr();
  }
  const at::Tensor dx = c.empty({op.rows, op.cols}, dy.scalar_type());
  op.dx = dx.data_ptr();
  op.ld_dx = op.cols;
  at::Tensor dgain, ws;
  size_t bytes = 0;
  if (want_dgain) {
    dgain = c.empty({op.cols}, at::kFloat);
    op.dgain = dgain.data_ptr<float>();
    bytes = g_entry.rmsnorm_grad_ws(op.rows, op.cols);
    ws = c.workspace(bytes);
  }
  const int st = g_entry.rmsnorm_grad(&op, bytes ? ws.data_ptr() : nullptr, bytes, c.stream());
  return py::make_tuple(st, dx, want_dgain ? py::cast(dgain) : py::none());
}

py::tuple swiglu(const at::Tensor& gate, const at::Tensor& up, bool save) {
  Call c(gate, "gate");
  muon_swiglu_t op{};
  op.ld_gate = c.matrix(gate, "gate");
  op.rows = gate.size(0);
  op.cols = gate.size(1);
  op.dtype = code_of(gate.scalar_type(), "gate");
  op.ld_up = c.matrix(up, "up", op.rows, op.cols);
  same_type(up, gate, "up", "gate");
  op.gate = gate.data_ptr();
  op.up = up.data_ptr();
  const at::Tensor a = c.empty({op.rows, op.cols}, gate.scalar_type());
  op.a = a.data_ptr();
  op.ld_a = op.cols;
  at::Tensor gc, gs, uc, us;
  if (save) {
    std::tie(gc, gs) = new_act8(c, op.rows, op.cols);
    std::tie(uc, us) = new_act8(c, op.rows, op.cols);
    op.gate8 = act8(c, gc, gs, "gate8", op.rows, op.cols);
    op.up8 = act8(c, uc, us, "up8", op.rows, op.cols);
  }
  const int st = g_entry.swiglu(&op, c.stream());
  if (!save) return py::make_tuple(st, a);
  return py::make_tuple(st, a, gc, gs, uc, us);
}

py::tuple swiglu_grad(const at::Tensor& da, const Codes& gate8, const Codes& up8, const OptTensor& dgate,
                      const OptTensor& dup, bool want_a8) {
  Call c(da, "da");
  muon_swiglu_grad_t op{};
  op.ld_da = c.matrix(da, "da");
  op.rows = da.size(0);
  op.cols = da.size(1);
  op.dtype = code_of(da.scalar_type(), "da");
  op.da = da.data_ptr();
  op.gate8 = act8(c, std::get<0>(gate8), std::get<1>(gate8), "gate8", op.rows, op.cols);
  op.up8 = act8(c, std::get<0>(up8), std::get<1>(up8), "up8", op.rows, op.cols);
  const at::Tensor dg = dgate ? *dgate : c.empty({op.rows, op.cols}, da.scalar_type());
  const at::Tensor du = dup ? *dup : c.empty({op.rows, op.cols}, da.scalar_type());
  op.ld_dgate = c.matrix(dg, "dgate", op.rows, op.cols);
  op.ld_dup = c.matrix(du, "dup", op.rows, op.cols);
  same_type(dg, da, "dgate", "da");
  same_type(du, da, "dup", "da");
  op.dgate = dg.data_ptr();
  op.dup = du.data_ptr();
  at::Tensor ac, as;
  if (want_a8) {
    std::tie(ac, as) = new_act8(c, op.rows, op.cols);
    op.a8 = act8(c, ac, as, "a8", op.rows, op.cols);
  }
  const int st = g_entry.swiglu_grad(&op, c.stream());
  if (!want_a8) return py::make_tuple(st, dg, du);
  return py::make_tuple(st, dg, du, ac, as);
}

py::tuple act8_wgrad(const at::Tensor& dy, const Codes& x8, const OptTensor& col_gain, const OptTensor& out,
                     at::ScalarType dtype, bool accumulate) {
  Call c(dy, "dy");
  muon_act8_wgrad_t op{};
  op.ld_dy = c.matrix(dy, "dy");
  if (dy.scalar_type() != at::kBFloat16) bad_type("dy", "must be bfloat16");
  op.dy = dy.data_ptr();
  op.tokens = dy.size(0);
  op.n = dy.size(1);
  const auto& [codes, scales] = x8;
  if (codes.dim() != 2) bad_value("x8", "must be 2-D");
  op.k = codes.size(1);
  op.x8 = act8(c, codes, scales, "x8", op.tokens, op.k);
  if (col_gain) op.col_gain = c.fp32_vector(*col_gain, "col_gain", op.k);
  if (accumulate && !out) bad_value("out", "must be given to accumulate");
  const at::Tensor dw = out ? *out : c.empty({op.n, op.k}, dtype);
  op.ld_dw = c.matrix(dw, "out", op.n, op.k);
  op.dw_dtype = code_of(dw.scalar_type(), "out");
  op.dw = dw.data_ptr();
  op.accumulate = accumulate ? 1 : 0;
  const size_t bytes = g_entry.wgrad_ws(&op);
  const at::Tensor ws = c.workspace(bytes);
  const int st = g_entry.wgrad(&op, bytes ? ws.data_ptr() : nullptr, bytes, c.stream());
  return py::make_tuple(st, dw);
}

const void* id_vector(const Call& c, const at::Tensor& ids, int32_t& id_bytes) {
  c.on_device(ids, "ids");
  if (ids.scalar_type() != at::kLong && ids.scalar_type() != at::kInt) bad_type("ids", "must be int32 or int64");
  if (ids.dim() != 1 || !ids.is_contiguous()) bad_value("ids", "must be a contiguous vector");
  id_bytes = ids.scalar_type() == at::kLong ? 8 : 4;
  return ids.data_ptr();
}

py::tuple embed(const at::Tensor& table, const at::Tensor& ids, double scale, const OptTensor& out, at::ScalarType dtype) {
  Call c(table, "table");
  muon_embed_t op{};
  op.ld_table = c.matrix(table, "table");
  op.vocab = table.size(0);
  op.cols = table.size(1);
  op.table_dtype = code_of(table.scalar_type(), "table");
  op.table = table.data_ptr();
  op.ids = id_vector(c, ids, op.id_bytes);
  op.tokens = ids.size(0);
  const at::Tensor o = out ? *out : c.empty({op.tokens, op.cols}, dtype);
  op.ld_out = c.matrix(o, "out", op.tokens, op.cols);
  op.out_dtype = code_of(o.scalar_type(), "out");
  op.out = o.data_ptr();
  op.scale = static_cast<float>(scale);
  const int st = g_entry.embed(&op, c.stream());
  return py::make_tuple(st, o);
}

py::tuple embed_grad(const at::Tensor& dy, const at::Tensor& ids, int64_t vocab, double scale, const OptTensor& out,
                     at::ScalarType dtype, bool accumulate) {
  Call c(dy, "dy");
  muon_embed_grad_t op{};
  op.ld_dy = c.matrix(dy, "dy");
  op.tokens = dy.size(0);
  op.cols = dy.size(1);
  op.vocab = vocab;
  op.dy_dtype = code_of(dy.scalar_type(), "dy");
  op.dy = dy.data_ptr();
  op.ids = id_vector(c, ids, op.id_bytes);
  if (ids.size(0) != op.tokens) bad_value("ids", "must have one id per row of dy");
  if (vocab < 1) bad_value("vocab", "must be at least 1");
  if (accumulate && !out) bad_value("out", "must be given to accumulate");
  const at::Tensor o = out ? *out : c.empty({vocab, op.cols}, dtype);
  op.ld_dtable = c.matrix(o, "out", vocab, op.cols);
  op.table_dtype = code_of(o.scalar_type(), "out");
  op.dtable = o.data_ptr();
  op.scale = static_cast<float>(scale);
  op.accumulate = accumulate ? 1 : 0;
  const size_t bytes = g_entry.embed_grad_ws(op.tokens, op.vocab, op.cols);
  const at::Tensor ws = c.workspace(bytes);
  const int st = g_entry.embed_grad(&op, bytes ? ws.data_ptr() : nullptr, bytes, c.stream());
  return py::make_tuple(st, o);
}

}  // namespace

void register_ops(py::module_& mod) {
  mod.def("bind_ops", &bind_ops);
  mod.def("act8_pack", &act8_pack);
  mod.def("act8_unpack", &act8_unpack);
  mod.def("rmsnorm_act8", &rmsnorm);
  mod.def("rmsnorm_act8_grad", &rmsnorm_grad);
  mod.def("swiglu_act8", &swiglu);
  mod.def("swiglu_act8_grad", &swiglu_grad);
  mod.def("act8_wgrad", &act8_wgrad);
  mod.def("embed", &embed);
  mod.def("embed_grad", &embed_grad);
  mod.attr("OP_BYTES") = std::map<std::string, size_t>{
      {"muon_act8_t", sizeof(muon_act8_t)}, {"muon_rmsnorm_t", sizeof(muon_rmsnorm_t)},
      {"muon_rmsnorm_grad_t", sizeof(muon_rmsnorm_grad_t)}, {"muon_swiglu_t", sizeof(muon_swiglu_t)},
      {"muon_swiglu_grad_t", sizeof(muon_swiglu_grad_t)}, {"muon_act8_wgrad_t", sizeof(muon_act8_wgrad_t)},
      {"muon_embed_t", sizeof(muon_embed_t)}, {"muon_embed_grad_t", sizeof(muon_embed_grad_t)}};
}
