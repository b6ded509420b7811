// binding.cpp -- torch tensors in and out of the operators around the chunk
// core (include/carve.h): the gated linear scan, the norms of q and k with the
// position rotation, and the short causal convolution.
//
// The one-token calls run for 1 to 3 us on the GPU, and a call through ctypes
// with its checks in Python took the host 9 to 12 us; here it takes 3.5 to 4.3,
// most of it the launch.  Checks, allocation and marshalling only: every step
// of the operators runs in the CUDA kernels of libcarve.so.  Work
// is enqueued on torch's current stream of the tensors' device, which need not
// be the current device.
#include <ATen/EmptyTensor.h>
#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/utils/pybind.h>

#include <initializer_list>
#include <optional>
#include <string>
#include <type_traits>
#include <utility>
#include <vector>

#include "../../../include/carve.h"

namespace py = pybind11;
using at::IntArrayRef;
using at::Tensor;
using MaybeTensor = std::optional<Tensor>;

namespace {

std::string text(const std::string& v) { return v; }
std::string text(int64_t v) { return std::to_string(v); }
std::string text(IntArrayRef v) {
  std::string s = "(";
  for (size_t i = 0; i < v.size(); ++i) s += (i ? ", " : "") + std::to_string(v[i]);
  return s + (v.size() == 1 ? ",)" : ")");
}
template <typename... A>
[[noreturn]] void bad(const A&... parts) {
  throw py::value_error((text(parts) + ...));
}

// Raises carve.CarveError for a status.
void ok(carve_status rc, const char* entry) {
  if (rc == CARVE_OK) return;
  py::object error =
      py::module_::import("chunk_gated_delta_02_b200.carve").attr("CarveError");
  PyErr_SetObject(error.ptr(), error(entry, (int)rc).ptr());
  throw py::error_already_set();
}

// ------------------------------------------------------------------ checks
// The type and device that a call's tensors share, from its first one; that
// device is the current one as long as this lives.
struct Common {
  at::ScalarType type;
  at::Device dev;
  int code;  // carve_dtype
  c10::cuda::OptionalCUDAGuard guard;
  Common(const Tensor& t, const char* name) : type(t.scalar_type()), dev(t.device()) {
    if (!t.is_cuda()) bad(name, " must be a CUDA tensor (no CPU path)");
    if (type != at::kBFloat16 && type != at::kFloat) bad("dtype must be bfloat16 or float32");
    code = type == at::kBFloat16 ? CARVE_BF16 : CARVE_FP32;
    guard.set_device(dev);
  }
  // A new contiguous tensor, from torch's allocator without its dispatcher
  // (a third of the host's time of a one-token call's allocation).
  Tensor empty(IntArrayRef shape, at::ScalarType t) const {
    return Tensor(at::detail::empty_generic(shape, c10::cuda::CUDACachingAllocator::get(),
                                            c10::DispatchKeySet(c10::DispatchKey::CUDA), t,
                                            std::nullopt));
  }
  void* stream() const { return c10::cuda::getCurrentCUDAStream(dev.index()).stream(); }
};

void same(const Tensor& t, const char* name, at::ScalarType type, IntArrayRef shape,
          at::Device dev) {
  if (!t.is_cuda()) bad(name, " must be a CUDA tensor (no CPU path)");
  if (t.device() != dev) bad(name, " is on ", t.device().str(), ", expected ", dev.str());
  if (t.scalar_type() != type) bad(name, " has dtype ", std::string(c10::toString(t.scalar_type())), ", expected ", std::string(c10::toString(type)));
  if (t.sizes() != shape) bad(name, " has shape ", text(t.sizes()), ", expected ", text(shape));
}
void need(const Tensor& t, const char* name, at::ScalarType type, IntArrayRef shape,
          at::Device dev) {
  same(t, name, type, shape, dev);
  if (!t.is_contiguous()) bad(name, " must be contiguous");
}
void need(const MaybeTensor& t, const char* name, at::ScalarType type, IntArrayRef shape,
          at::Device dev) {
  if (t) need(*t, name, type, shape, dev);
}
const Tensor& given(const MaybeTensor& t, const char* name) {
  if (!t) bad(name, " is required");
  return *t;
}

// Elements from one token to the next of an input with `lead` leading
// dimensions (batch and time, or time alone): tokens are rows of contiguous
// channels, evenly spaced.  0: the tensor is contiguous.
int64_t pitch_of(const Tensor& t, const char* name, int64_t lead) {
  if (t.is_contiguous()) return 0;
  int64_t width = 1, rows = 1, pitch = -1;  // -1: one token, no step yet
  bool fine = true;
  for (int64_t d = t.dim() - 1; d >= lead; --d) {
    fine &= t.size(d) == 1 || t.stride(d) == width;
    width *= t.size(d);
  }
  for (int64_t d = lead - 1; d >= 0; --d) {
    if (t.size(d) > 1) {
      if (pitch < 0) {
        pitch = t.stride(d) / rows;
        fine &= t.stride(d) % rows == 0;
      }
      fine &= t.stride(d) == pitch * rows;
    }
    rows *= t.size(d);
  }
  if (pitch < 0) pitch = width;
  if (!fine || pitch < width || pitch % 8)
    bad(name, ": the channels of a token must be contiguous and tokens evenly spaced by a "
        "multiple of 8 elements (strides ", text(t.strides()), " of shape ", text(t.sizes()), ")");
  return pitch;
}
int64_t pitch(const Tensor& t, const char* name, const Common& k, IntArrayRef shape,
              int64_t lead) {
  same(t, name, k.type, shape, k.dev);
  return pitch_of(t, name, lead);
}

// A caller's output, checked, or a new contiguous tensor like t.
Tensor like(const Common& k, const Tensor& t, const MaybeTensor& mine, const char* name) {
  if (!mine) return k.empty(t.sizes(), t.scalar_type());
  need(*mine, name, t.scalar_type(), t.sizes(), t.device());
  return *mine;
}
// The bytes from a tensor's first element to its last.
struct Span {
  uintptr_t lo, hi;
  explicit Span(const Tensor& t) : lo((uintptr_t)t.data_ptr()), hi(lo) {
    if (!t.numel()) return;
    int64_t last = 0;
    for (int64_t d = 0; d < t.dim(); ++d) last += (t.size(d) - 1) * t.stride(d);
    hi += (last + 1) * t.element_size();
  }
};
// A caller's output must not overlap what the call reads, nor another output.
using Others = std::initializer_list<const Tensor*>;
const Tensor* the(const MaybeTensor& t) { return t ? &*t : nullptr; }
void apart(const Tensor& mine, const char* name, Others others) {
  const Span o(mine);
  for (const Tensor* t : others) {
    if (!t) continue;
    const Span s(*t);
    if (o.lo < s.hi && s.lo < o.hi) bad(name, " overlaps another tensor of the call");
  }
}
void apart(const MaybeTensor& mine, const char* name, Others others) {
  if (mine) apart(*mine, name, others);
}

Tensor workspace(const MaybeTensor& mine, size_t bytes, const char* entry, const Common& k) {
  if (!bytes) ok(CARVE_ERR_UNSUPPORTED, entry);
  if (!mine) return k.empty({(int64_t)bytes}, at::kByte);
  if (mine->scalar_type() != at::kByte || mine->device() != k.dev || !mine->is_contiguous() ||
      mine->numel() < (int64_t)bytes)
    bad("workspace must be ", (int64_t)bytes, " contiguous bytes (uint8) on ", k.dev.str());
  if ((uintptr_t)mine->data_ptr() % 16) ok(CARVE_ERR_WORKSPACE, entry);
  return *mine;
}

// Tells autograd that a call has written into a caller's tensors: a backward
// pass that has kept one then refuses to run instead of reading new values.
void written(Others ts) {
  for (const Tensor* t : ts)
    if (t && !t->is_inference()) t->unsafeGetTensorImpl()->bump_version();
}

// What a call returns: tensors or None, in a tuple or under names.
PyObject* wrapped(const Tensor* t) {
  if (t) return THPVariable_Wrap(*t);
  Py_RETURN_NONE;
}
py::tuple tuple_of(std::initializer_list<const Tensor*> ts) {
  py::tuple r(ts.size());
  Py_ssize_t i = 0;
  for (const Tensor* t : ts) PyTuple_SET_ITEM(r.ptr(), i++, wrapped(t));
  return r;
}
py::dict dict_of(std::initializer_list<std::pair<const char*, const Tensor*>> ts) {
  py::dict r;
  for (const auto& [name, t] : ts) {
    const py::object o = py::reinterpret_steal<py::object>(wrapped(t));
    if (PyDict_SetItemString(r.ptr(), name, o.ptr())) throw py::error_already_set();
  }
  return r;
}

const void* in(const MaybeTensor& t) { return t ? t->data_ptr() : nullptr; }
const float* fin(const MaybeTensor& t) { return static_cast<const float*>(in(t)); }
void* out(const MaybeTensor& t) { return t ? t->data_ptr() : nullptr; }
float* fout(const MaybeTensor& t) { return static_cast<float*>(out(t)); }
const int32_t* iin(const MaybeTensor& t) { return static_cast<const int32_t*>(in(t)); }

int32_t i32(int64_t v, const char* what) {
  if (v > INT32_MAX) bad(what, " is too large");
  return (int32_t)v;
}

// Sequences, tokens and channels of a token tensor, dense [B, T, ...] or
// packed [T, ...] with offsets.
struct Batch {
  int64_t lead;
  int32_t B, T, C;
  at::DimVector state;  // shape of a state of `per` rows a sequence (0: none)
  Batch(const Tensor& x, const char* name, const MaybeTensor& cu, const Common& k, int64_t per) {
    lead = cu ? 1 : 2;
    if (x.dim() <= lead) bad(name, " needs ", lead, " leading dimensions and channels");
    if (cu) {
      if (cu->numel() < 2) bad("cu_seqlens needs at least two entries");
      need(*cu, "cu_seqlens", at::kInt, {cu->numel()}, k.dev);
    }
    B = i32(cu ? cu->numel() - 1 : x.size(0), "the batch");
    T = i32(x.size(lead - 1), "the number of tokens");
    state.push_back(B);
    if (per) state.push_back(per);
    int64_t c = 1;
    for (int64_t d = lead; d < x.dim(); ++d) {
      c *= x.size(d);
      state.push_back(x.size(d));
    }
    C = i32(c, "the number of channels");
  }
};

at::ScalarType kState = at::kFloat;

// -------------------------------------------------------------------- scan
carve_scan_shape scan_shape(const Batch& b, const Common& k, double scale, bool comp, bool fill,
                            int64_t xp, int64_t gp) {
  return {b.B, b.T, b.C, k.code, (float)scale, comp, fill, 0, xp, gp};
}

py::tuple scan_fwd(const Tensor& x, const Tensor& g, const MaybeTensor& h0,
                   const MaybeTensor& cu, bool training, const MaybeTensor& mine_ws,
                   const MaybeTensor& mine, bool want_state, double scale, bool comp) {
  const Common k(x, "x");
  const Batch b(x, "x", cu, k, 0);
  const carve_scan_shape s = scan_shape(b, k, scale, comp, !mine, pitch_of(x, "x", b.lead),
                                        pitch(g, "g", k, x.sizes(), b.lead));
  need(h0, "h0", kState, b.state, k.dev);
  MaybeTensor ws;
  if (training || cu || mine_ws)
    ws = workspace(mine_ws, carve_scan_workspace_bytes(&s, cu.has_value(), training),
                   "carve_scan_workspace_bytes", k);
  apart(mine_ws, "workspace", {&x, &g, the(h0), the(cu)});
  const Tensor h = like(k, x, mine, "h");
  apart(mine, "h", {&x, &g, the(h0), the(cu), the(ws)});
  MaybeTensor h_T;
  if (want_state) h_T = k.empty(b.state, kState);
  ok(carve_scan_fwd(&s, iin(cu), x.data_ptr(), g.data_ptr(), fin(h0), h.data_ptr(), fout(h_T),
                    out(ws), ws ? ws->numel() : 0, training, k.stream()),
     "carve_scan_fwd");
  written({the(mine), the(ws)});
  return tuple_of({&h, the(h_T), the(ws)});
}

// Outputs that the caller may bring in a dict.
MaybeTensor item(const std::optional<py::dict>& d, const char* name) {
  if (!d || !d->contains(name)) return std::nullopt;
  return (*d)[name].cast<MaybeTensor>();
}

py::dict scan_bwd(const Tensor& x, const Tensor& g, const Tensor& d_h, const MaybeTensor& ws,
                  const MaybeTensor& dh_T, const MaybeTensor& cu, bool want_dh0,
                  const std::optional<py::dict>& mine, double scale, bool comp) {
  const Common k(x, "x");
  const Batch b(x, "x", cu, k, 0);
  const carve_scan_shape s = scan_shape(b, k, scale, comp, !mine, pitch_of(x, "x", b.lead),
                                        pitch(g, "g", k, x.sizes(), b.lead));
  need(d_h, "d_h", k.type, x.sizes(), k.dev);
  need(dh_T, "dh_T", kState, b.state, k.dev);
  if (!ws) bad("scan_bwd needs the workspace of a training forward");
  workspace(ws, carve_scan_workspace_bytes(&s, cu.has_value(), 1), "carve_scan_workspace_bytes", k);
  apart(ws, "workspace", {&x, &g, &d_h, the(dh_T), the(cu)});
  const Tensor dx = like(k, x, mine ? given(item(mine, "dx"), "dx") : MaybeTensor(), "dx");
  const Tensor dg = like(k, x, mine ? given(item(mine, "dg"), "dg") : MaybeTensor(), "dg");
  MaybeTensor dh0 = item(mine, "dh0");
  if (dh0) need(*dh0, "dh0", kState, b.state, k.dev);
  else if (!mine && want_dh0) dh0 = k.empty(b.state, kState);
  if (mine) {
    apart(dx, "dx", {&x, &g, &d_h, the(dh_T), the(cu), the(ws), &dg, the(dh0)});
    apart(dg, "dg", {&x, &g, &d_h, the(dh_T), the(cu), the(ws), the(dh0)});
    apart(dh0, "dh0", {&x, &g, &d_h, the(dh_T), the(cu), the(ws)});
  }
  ok(carve_scan_bwd(&s, iin(cu), x.data_ptr(), g.data_ptr(), d_h.data_ptr(), fin(dh_T),
                    ws->data_ptr(), ws->numel(), dx.data_ptr(), dg.data_ptr(), fout(dh0),
                    k.stream()),
     "carve_scan_bwd");
  if (mine) written({&dx, &dg, the(dh0)});
  return dict_of({{"dx", &dx}, {"dg", &dg}, {"dh0", the(dh0)}});
}

Tensor scan_step(const Tensor& x, const Tensor& g, const Tensor& h, const MaybeTensor& mine,
                 double scale, bool comp) {
  const Common k(x, "x");
  if (x.dim() < 2) bad("x needs a batch dimension and channels");
  const int64_t B = x.size(0), C = B ? x.numel() / B : 0;
  const carve_scan_shape s{i32(B, "the batch"), 1, i32(C, "the number of channels"), k.code,
                           (float)scale, comp, 0, 0, pitch_of(x, "x", 1),
                           pitch(g, "g", k, x.sizes(), 1)};
  need(h, "h", kState, x.sizes(), k.dev);
  const Tensor o = like(k, x, mine, "o");
  apart(h, "h", {&x, &g});
  apart(mine, "o", {&x, &g, &h});
  ok(carve_scan_step(&s, x.data_ptr(), g.data_ptr(), h.data_ptr<float>(), o.data_ptr(),
                     k.stream()),
     "carve_scan_step");
  written({&h, the(mine)});
  return o;
}

// ---------------------------------------------------------------- rotation
struct Rope {
  Common k;
  carve_rope_shape s;
  Rope(const Tensor& q, const MaybeTensor& key, const MaybeTensor& pos, const MaybeTensor& freqs,
       const MaybeTensor& w_q, const MaybeTensor& w_k, double eps, bool l2norm, bool inter)
      : k(q, "q") {
    if (q.dim() < 3) bad("q needs token dimensions, heads and elements");
    const int64_t lead = q.dim() - 2, D = q.size(-1);
    const IntArrayRef tokens = q.sizes().slice(0, lead);
    int64_t N = 1, HK = 0, kp = 0;
    for (int64_t n : tokens) N *= n;
    if (key) {
      if (key->dim() != q.dim()) bad("k must have as many dimensions as q");
      at::DimVector shape(q.sizes());
      shape[lead] = HK = key->size(lead);
      kp = pitch(*key, "k", k, shape, lead);
    }
    const int64_t RD = freqs ? 2 * freqs->numel() : 0;
    if (RD) {
      need(*freqs, "freqs", at::kDouble, {RD / 2}, k.dev);
      need(given(pos, "pos"), "pos", at::kInt, tokens, k.dev);
    }
    need(w_q, "w_q", k.type, {D}, k.dev);
    need(w_k, "w_k", k.type, {D}, k.dev);
    s = {N, i32(q.size(lead), "the number of heads"), i32(HK, "the number of heads"),
         i32(D, "the head width"), i32(RD, "the rotated width"), k.code, (float)eps, l2norm,
         inter, pitch_of(q, "q", lead), kp};
  }
};

py::tuple qk_rope_fwd(const Tensor& q, const MaybeTensor& key, const MaybeTensor& pos,
                      const MaybeTensor& freqs, const MaybeTensor& w_q, const MaybeTensor& w_k,
                      double eps, bool l2norm, bool inter, const MaybeTensor& q_mine,
                      const MaybeTensor& k_mine) {
  const Rope r(q, key, pos, freqs, w_q, w_k, eps, l2norm, inter);
  const Tensor q_out = like(r.k, q, q_mine, "q_out");
  MaybeTensor k_out;
  if (key) k_out = like(r.k, *key, k_mine, "k_out");
  apart(q_mine, "q_out", {&q, the(key), the(pos), the(freqs), the(w_q), the(w_k), the(k_mine)});
  apart(k_mine, "k_out", {&q, the(key), the(pos), the(freqs), the(w_q), the(w_k)});
  ok(carve_qk_rope_fwd(&r.s, q.data_ptr(), in(key), iin(pos),
                       static_cast<const double*>(in(freqs)), in(w_q), in(w_k), q_out.data_ptr(),
                       out(k_out), r.k.stream()),
     "carve_qk_rope_fwd");
  written({the(q_mine), the(k_mine)});
  return tuple_of({&q_out, the(k_out)});
}

py::dict qk_rope_bwd(const Tensor& q, const MaybeTensor& key, const MaybeTensor& pos,
                     const MaybeTensor& freqs, const Tensor& dq_out, const MaybeTensor& dk_out,
                     const MaybeTensor& w_q, const MaybeTensor& w_k, double eps, bool l2norm,
                     bool inter, const std::optional<py::dict>& mine) {
  const Rope r(q, key, pos, freqs, w_q, w_k, eps, l2norm, inter);
  const Common& k = r.k;
  need(dq_out, "dq_out", k.type, q.sizes(), k.dev);
  if (key) need(given(dk_out, "dk_out"), "dk_out", k.type, key->sizes(), k.dev);
  const Tensor dq = like(k, q, mine ? given(item(mine, "dq"), "dq") : MaybeTensor(), "dq");
  MaybeTensor dk, dw_q, dw_k, ws;
  if (key) dk = like(k, *key, mine ? given(item(mine, "dk"), "dk") : MaybeTensor(), "dk");
  auto sum = [&](const MaybeTensor& w, const char* name) -> MaybeTensor {
    if (!w) return std::nullopt;
    if (!mine) return k.empty({r.s.D}, kState);
    const MaybeTensor t = item(mine, name);
    need(given(t, name), name, kState, {r.s.D}, k.dev);
    return t;
  };
  dw_q = sum(w_q, "dw_q");
  dw_k = sum(w_k, "dw_k");
  if (mine) {
    const Tensor *kt = the(key), *dkt = the(dk_out), *p = the(pos), *f = the(freqs);
    apart(dq, "dq", {&q, kt, p, f, the(w_q), the(w_k), &dq_out, dkt, the(dk), the(dw_q), the(dw_k)});
    apart(dk, "dk", {&q, kt, p, f, the(w_q), the(w_k), &dq_out, dkt, the(dw_q), the(dw_k)});
    apart(dw_q, "dw_q", {&q, kt, p, f, the(w_q), the(w_k), &dq_out, dkt, the(dw_k)});
    apart(dw_k, "dw_k", {&q, kt, p, f, the(w_q), the(w_k), &dq_out, dkt});
  }
  if (w_q || w_k)
    ws = workspace(std::nullopt, carve_qk_rope_workspace_bytes(&r.s),
                   "carve_qk_rope_workspace_bytes", k);
  ok(carve_qk_rope_bwd(&r.s, q.data_ptr(), in(key), iin(pos),
                       static_cast<const double*>(in(freqs)), in(w_q), in(w_k),
                       dq_out.data_ptr(), in(key ? dk_out : MaybeTensor()), out(ws),
                       ws ? ws->numel() : 0, dq.data_ptr(), out(dk), fout(dw_q), fout(dw_k),
                       k.stream()),
     "carve_qk_rope_bwd");
  if (mine) written({&dq, the(dk), the(dw_q), the(dw_k)});
  return dict_of({{"dq", &dq}, {"dk", the(dk)}, {"dw_q", the(dw_q)}, {"dw_k", the(dw_k)}});
}

// ------------------------------------------------------------- convolution
int32_t taps(const Tensor& w, const MaybeTensor& bias, const Common& k, int64_t C) {
  if (w.dim() != 2) bad("w must be a [channels, taps] tensor");
  need(w, "w", k.type, {C, w.size(1)}, k.dev);
  need(bias, "bias", k.type, {C}, k.dev);
  return i32(w.size(1), "the number of taps");
}
struct Conv {
  Common k;
  Batch b;
  carve_conv_shape s;
  Conv(const Tensor& x, const Tensor& w, const MaybeTensor& bias, const MaybeTensor& state,
       const MaybeTensor& cu, bool silu, bool fill)
      : k(x, "x"), b(x, "x", cu, k, w.dim() == 2 ? w.size(1) - 1 : 1) {
    const int32_t W = taps(w, bias, k, b.C);
    if (W < 2) ok(CARVE_ERR_UNSUPPORTED, "carve_conv_workspace_bytes");
    need(state, "state", k.type, b.state, k.dev);
    s = {b.B, b.T, b.C, W, k.code, silu, fill, 0, pitch_of(x, "x", b.lead)};
  }
};

py::tuple conv_fwd(const Tensor& x, const Tensor& w, const MaybeTensor& bias,
                   const MaybeTensor& state, const MaybeTensor& cu, bool silu,
                   const MaybeTensor& mine, bool want_state, const MaybeTensor& mine_ws) {
  const Conv c(x, w, bias, state, cu, silu, !mine);
  MaybeTensor ws;
  if (cu || mine_ws)
    ws = workspace(mine_ws, carve_conv_workspace_bytes(&c.s, cu.has_value(), 0), "carve_conv_workspace_bytes", c.k);
  apart(mine_ws, "workspace", {&x, &w, the(bias), the(state), the(cu)});
  const Tensor y = like(c.k, x, mine, "y");
  apart(mine, "y", {&x, &w, the(bias), the(state), the(cu), the(ws)});
  MaybeTensor state_T;
  if (want_state) state_T = c.k.empty(c.b.state, c.k.type);
  ok(carve_conv_fwd(&c.s, iin(cu), x.data_ptr(), w.data_ptr(), in(bias), in(state), y.data_ptr(),
                    out(state_T), out(ws), ws ? ws->numel() : 0, c.k.stream()),
     "carve_conv_fwd");
  written({the(mine), the(ws)});
  return tuple_of({&y, the(state_T)});
}

py::dict conv_bwd(const Tensor& x, const Tensor& w, const Tensor& dy, const MaybeTensor& bias,
                  const MaybeTensor& state, const MaybeTensor& dstate_T, const MaybeTensor& cu,
                  bool silu, const std::optional<py::dict>& mine, const MaybeTensor& mine_ws) {
  const Conv c(x, w, bias, state, cu, silu, !mine);
  const Common& k = c.k;
  need(dy, "dy", k.type, x.sizes(), k.dev);
  need(dstate_T, "dstate_T", k.type, c.b.state, k.dev);
  const MaybeTensor ws = workspace(
      mine_ws, carve_conv_workspace_bytes(&c.s, cu.has_value(), 1), "carve_conv_workspace_bytes", k);
  apart(mine_ws, "workspace", {&x, &w, &dy, the(bias), the(state), the(dstate_T), the(cu)});
  const Tensor dx = like(k, x, mine ? given(item(mine, "dx"), "dx") : MaybeTensor(), "dx");
  MaybeTensor dw = item(mine, "dw"), dbias = item(mine, "dbias"), dstate = item(mine, "dstate");
  if (mine) {
    need(given(dw, "dw"), "dw", kState, w.sizes(), k.dev);
    need(dbias, "dbias", kState, {c.s.C}, k.dev);
    need(dstate, "dstate", k.type, c.b.state, k.dev);
    const Tensor *bt = the(bias), *st = the(state), *dt = the(dstate_T), *ct = the(cu);
    apart(dx, "dx", {&x, &w, bt, st, &dy, dt, ct, the(ws), the(dw), the(dbias), the(dstate)});
    apart(dw, "dw", {&x, &w, bt, st, &dy, dt, ct, the(ws), the(dbias), the(dstate)});
    apart(dbias, "dbias", {&x, &w, bt, st, &dy, dt, ct, the(ws), the(dstate)});
    apart(dstate, "dstate", {&x, &w, bt, st, &dy, dt, ct, the(ws)});
  } else {
    dw = k.empty(w.sizes(), kState);
    if (bias) dbias = k.empty({c.s.C}, kState);
    dstate = k.empty(c.b.state, k.type);
  }
  ok(carve_conv_bwd(&c.s, iin(cu), x.data_ptr(), w.data_ptr(), in(bias), in(state),
                    dy.data_ptr(), in(dstate_T), ws->data_ptr(), ws->numel(), dx.data_ptr(),
                    fout(dw), fout(dbias), out(dstate), k.stream()),
     "carve_conv_bwd");
  if (mine) written({&dx, the(dw), the(dbias), the(dstate)});
  written({the(ws)});
  return dict_of({{"dx", &dx}, {"dw", the(dw)}, {"dbias", the(dbias)}, {"dstate", the(dstate)}});
}

Tensor conv_step(const Tensor& x, const Tensor& w, const Tensor& state, const MaybeTensor& bias,
                 bool silu, const MaybeTensor& mine) {
  const Common k(x, "x");
  if (x.dim() < 2) bad("x needs a batch dimension and channels");
  const int64_t B = x.size(0), C = B ? x.numel() / B : 0;
  const int32_t W = taps(w, bias, k, C);
  at::DimVector kept(x.sizes());
  kept.insert(kept.begin() + 1, W - 1);
  need(state, "state", k.type, kept, k.dev);
  const carve_conv_shape s{i32(B, "the batch"), 1, i32(C, "the number of channels"), W, k.code,
                           silu, 0, 0, pitch_of(x, "x", 1)};
  const Tensor y = like(k, x, mine, "y");
  apart(state, "state", {&x, &w, the(bias)});
  apart(mine, "y", {&x, &w, the(bias), &state});
  ok(carve_conv_step(&s, x.data_ptr(), w.data_ptr(), in(bias), state.data_ptr(), y.data_ptr(),
                     k.stream()),
     "carve_conv_step");
  written({&state, the(mine)});
  return y;
}

// ---------------------------------------------------------------- calling
// Arguments by position or keyword, straight from the interpreter's arrays:
// of a one-token call's host time that leaves out about 1 us that building
// and matching a keyword dict takes.
template <typename T>
struct Arg;
template <>
struct Arg<Tensor> {
  static const Tensor& from(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) throw py::type_error(std::string(name) + " must be a tensor");
    return THPVariable_Unpack(o);
  }
};
template <>
struct Arg<MaybeTensor> {
  static MaybeTensor from(PyObject* o, const char* name) {
    if (o == Py_None) return std::nullopt;
    return Arg<Tensor>::from(o, name);
  }
};
template <>
struct Arg<bool> {
  static bool from(PyObject* o, const char*) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw py::error_already_set();
    return v != 0;
  }
};
template <>
struct Arg<double> {
  static double from(PyObject* o, const char*) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw py::error_already_set();
    return v;
  }
};
template <>
struct Arg<std::optional<py::dict>> {
  static std::optional<py::dict> from(PyObject* o, const char* name) {
    if (o == Py_None) return std::nullopt;
    if (!PyDict_Check(o)) throw py::type_error(std::string(name) + " must be a dict");
    return py::reinterpret_borrow<py::dict>(o);
  }
};
PyObject* give(const Tensor& t) { return THPVariable_Wrap(t); }
PyObject* give(py::object&& o) { return o.release().ptr(); }

// A parameter: its name (interned) and, unless it is required, its default.
struct Param {
  const char* name;
  PyObject *key, *value;
};
Param arg(const char* name) { return {name, PyUnicode_InternFromString(name), nullptr}; }
Param arg(const char* name, PyObject* value) {
  Py_INCREF(value);
  return {name, PyUnicode_InternFromString(name), value};
}
struct Entry {
  const char* name;
  std::vector<Param> params;
  std::string doc;
  PyMethodDef def;
};
template <auto fn>
Entry* entry = nullptr;

[[noreturn]] void no_call(const Entry& e, const char* what, PyObject* key) {
  PyErr_Format(PyExc_TypeError, key ? "%s() %s '%U'" : "%s() %s", e.name, what, key);
  throw py::error_already_set();
}
// Fills slots[] from a call's arrays.
void match(const Entry& e, PyObject* const* args, Py_ssize_t n, PyObject* names,
           PyObject** slots) {
  const Py_ssize_t count = (Py_ssize_t)e.params.size();
  if (n > count) no_call(e, "takes fewer positional arguments", nullptr);
  for (Py_ssize_t i = 0; i < count; ++i) slots[i] = i < n ? args[i] : nullptr;
  const Py_ssize_t keys = names ? PyTuple_GET_SIZE(names) : 0;
  for (Py_ssize_t k = 0; k < keys; ++k) {
    PyObject* const key = PyTuple_GET_ITEM(names, k);
    Py_ssize_t i = 0;
    while (i < count && e.params[i].key != key) ++i;
    if (i == count)  // not the interned object
      for (i = 0; i < count && PyUnicode_Compare(e.params[i].key, key) != 0;) ++i;
    if (i == count) no_call(e, "got an unexpected keyword argument", key);
    if (slots[i]) no_call(e, "got multiple values for argument", key);
    slots[i] = args[n + k];
  }
  for (Py_ssize_t i = 0; i < count; ++i) {
    if (!slots[i]) slots[i] = e.params[i].value;
    if (!slots[i]) no_call(e, "misses the required argument", e.params[i].key);
  }
}
template <auto fn, typename R, typename... A, size_t... I>
PyObject* invoke(R (*)(A...), PyObject* const* s, const Entry& e, std::index_sequence<I...>) {
  return give(fn(Arg<std::decay_t<A>>::from(s[I], e.params[I].name)...));
}
template <typename R, typename... A>
constexpr size_t arity(R (*)(A...)) {
  return sizeof...(A);
}
template <auto fn>
PyObject* call(PyObject*, PyObject* const* args, Py_ssize_t n, PyObject* names) {
  HANDLE_TH_ERRORS
  constexpr size_t count = arity(fn);
  PyObject* slots[count];
  try {
    match(*entry<fn>, args, n, names, slots);
    return invoke<fn>(fn, slots, *entry<fn>, std::make_index_sequence<count>());
  } catch (py::error_already_set& e) {
    e.restore();
  } catch (py::builtin_exception& e) {
    e.set_error();
  }
  return nullptr;
  END_HANDLE_TH_ERRORS
}
// Makes fn an entry point of the module.
template <auto fn>
void def(py::module_& m, const char* name, std::vector<Param> params, const char* doc) {
  std::string text = std::string(name) + "(";
  for (size_t i = 0; i < params.size(); ++i) {
    text += (i ? ", " : "") + std::string(params[i].name);
    if (params[i].value)
      text += "=" + py::cast<std::string>(py::repr(py::handle(params[i].value)));
  }
  text += std::string(")\n--\n\n") + doc;
  if (params.size() != arity(fn)) throw py::type_error(name);
  Entry* const e = entry<fn> = new Entry{name, std::move(params), std::move(text), {}};
  e->def = {e->name, (PyCFunction)(void (*)())call<fn>, METH_FASTCALL | METH_KEYWORDS,
            e->doc.c_str()};
  const py::object owner = m.attr("__name__");
  m.attr(name) = py::reinterpret_steal<py::object>(
      PyCFunction_NewEx(&e->def, m.ptr(), owner.ptr()));
}

}  // namespace

PYBIND11_MODULE(_mixer, m) {
  m.doc() = "Bindings of the operators around the chunk core (see mixer.py).";
  PyObject *const none = Py_None, *const yes = Py_True, *const no = Py_False;
  const py::float_ zero(0.0), small(1e-6);
  def<scan_fwd>(m, "scan_fwd",
            {arg("x"), arg("g"), arg("h0", none), arg("cu_seqlens", none),
             arg("training", no), arg("workspace", none), arg("h", none), arg("want_state", yes),
             arg("decay_scale", zero.ptr()), arg("complement", no)},
        R"(Gated linear scan h_t = exp(g_t) h_{t-1} + x_t over the tokens of each
sequence, one state per channel.  Returns (h, h_T, workspace).

x, g [B, T, ...] (bf16 or fp32; a multiple of 8 channels in the trailing
dimensions), or packed [T, ...] with cu_seqlens [N + 1] int32 on the device;
h0 [B, ...] fp32 or None; h like x; h_T [B, ...] fp32 (None with
want_state=False).  decay_scale > 0: g holds raw decay logits a, the log-decay
is -decay_scale * softplus(a).  complement: the input enters as
(1 - exp(g_t)) x_t.  With training=True the returned workspace holds what
scan_bwd needs; it is None where nothing needs one and none is given (256 bytes,
uint8, without training).  Its status word (get_status(workspace)) tells whether
cu_seqlens was valid and whether a wait gave up.)");
  def<scan_bwd>(m, "scan_bwd",
            {arg("x"), arg("g"), arg("d_h"), arg("workspace"), arg("dh_T", none),
             arg("cu_seqlens", none), arg("want_dh0", yes), arg("out", none),
             arg("decay_scale", zero.ptr()), arg("complement", no)},
        R"(Backward of scan_fwd(training=True) with the same x, g, cu_seqlens and
options, from the workspace it returned.  d_h like x (contiguous); dh_T
[B, ...] fp32 or None.  Returns a dict: dx, dg like x (dg is dL/da of the raw
logits with decay_scale > 0), dh0 [B, ...] fp32.  out: a dict of preallocated
dx, dg and (or None) dh0.)");
  def<scan_step>(m, "scan_step",
            {arg("x"), arg("g"), arg("h"), arg("o", none), arg("decay_scale", zero.ptr()),
             arg("complement", no)},
        R"(One token for each sequence: x, g [B, ...] (bf16 or fp32), h [B, ...] fp32
updated in place.  Returns o [B, ...], the new state in x's dtype.)");
  def<qk_rope_fwd>(m, "qk_rope_fwd",
            {arg("q"), arg("k"), arg("pos"), arg("freqs"), arg("w_q", none),
             arg("w_k", none), arg("eps", small.ptr()), arg("l2norm", no), arg("interleaved", no),
             arg("q_out", none), arg("k_out", none)},
        R"(Norms of the queries and keys of each head, times the weights, and the
rotation by position, in one pass.  Returns (q_out, k_out).

q [..., HQ, D], k [..., HK, D] (or None), bf16 or fp32, any number of token
dimensions (one token per sequence: [B, H, D]); pos [...] int32; freqs [RD / 2]
float64 radians per position (rope_freqs; None: no rotation) for the first RD
elements; w_q, w_k [D] or None.  Rows are divided by sqrt(mean(x^2) + eps), or
with l2norm=True by sqrt(sum(x^2) + eps), which gives the unit rows that
chunk_fwd takes.)");
  def<qk_rope_bwd>(m, "qk_rope_bwd",
            {arg("q"), arg("k"), arg("pos"), arg("freqs"), arg("dq_out"), arg("dk_out"),
             arg("w_q", none), arg("w_k", none), arg("eps", small.ptr()), arg("l2norm", no),
             arg("interleaved", no), arg("out", none)},
        R"(Backward of qk_rope_fwd from its inputs and the gradients of its outputs
(contiguous).  Returns a dict: dq, dk like q, k; dw_q, dw_k [D] fp32, summed
over tokens and heads (None where there is no weight).  out: preallocated dq,
dk, and dw_q, dw_k where there are weights.)");
  def<conv_fwd>(m, "conv_fwd",
            {arg("x"), arg("w"), arg("bias", none), arg("state", none),
             arg("cu_seqlens", none), arg("silu", no), arg("y", none), arg("want_state", yes),
             arg("workspace", none)},
        R"(Short causal convolution of each channel, y_t = act(bias + sum_j w[:, j]
x_{t - W + 1 + j}).  Returns (y, state_T).

x [B, T, ...] (bf16 or fp32; a multiple of 8 channels in the trailing
dimensions), or packed [T, ...] with cu_seqlens [N + 1] int32; w [C, W] with
W = 2, 3 or 4 taps; bias [C] or None; state [B, W - 1, ...] the inputs before
each sequence (None: zeros), state_T the same after it (None with
want_state=False).  silu=True: act(z) = z sigmoid(z).  A call that is given a
workspace (256 bytes, uint8) leaves its status word there for get_status.)");
  def<conv_bwd>(m, "conv_bwd",
            {arg("x"), arg("w"), arg("dy"), arg("bias", none), arg("state", none),
             arg("dstate_T", none), arg("cu_seqlens", none), arg("silu", no),
             arg("out", none), arg("workspace", none)},
        R"(Backward of conv_fwd from its inputs; dy like x (contiguous), dstate_T
[B, W - 1, ...] or None.  Returns a dict: dx like x, dw [C, W] and dbias [C]
fp32 (dbias None without a bias), dstate [B, W - 1, ...].  out: preallocated
dx, dw and (or None) dbias, dstate.)");
  def<conv_step>(m, "conv_step",
            {arg("x"), arg("w"), arg("state"), arg("bias", none), arg("silu", no),
             arg("y", none)},
        R"(One token for each sequence: x [B, ...], state [B, W - 1, ...] updated in
place.  Returns y [B, ...].)");
}
