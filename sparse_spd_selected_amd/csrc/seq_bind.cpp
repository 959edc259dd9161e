// seq_bind.cpp -- Python binding of the sequence-mixer entry points.
//
// A token's call is over in four microseconds, so its arguments are checked and
// its struct is filled here and not in Python.  The functions take and return
// tensors; they call the entry points of the library that the package loaded
// (bind() hands over their addresses), on the current stream of the inputs'
// device.
#include <pybind11/functional.h>
#include <torch/extension.h>

#include <array>
#include <string>

#include "selinv_seq.h"

namespace {

using at::Tensor;
using Maybe = std::optional<Tensor>;
using Shape = at::IntArrayRef;

enum Op { kConv, kConvStep, kConvVjp, kQkrot, kQkrotVjp, kScan, kScanStep, kScanVjp, kOps };
const char *const kNames[kOps] = {"conv", "conv_step", "conv_vjp", "qkrot",
                                  "qkrot_vjp", "scan", "scan_step", "scan_vjp"};
const char *const kTypes[3] = {"f32", "f16", "bf16"};
std::array<std::array<void *, 3>, kOps> g_entry = {};
// the library's workspace queries
decltype(&selinv_conv_vjp_workspace_bytes) g_conv_vjp_bytes = nullptr;
decltype(&selinv_qkrot_vjp_workspace_bytes) g_qkrot_vjp_bytes = nullptr;
decltype(&selinv_scan_workspace_bytes) g_scan_bytes = nullptr;
decltype(&selinv_scan_vjp_workspace_bytes) g_scan_vjp_bytes = nullptr;
decltype(&selinv_scan_vjp_bf16_workspace_bytes) g_scan_vjp_bf16_bytes = nullptr;
PyObject *g_stream = nullptr;  // device index -> handle of its current stream
PyObject *g_failed = nullptr;  // (status, name): raises

int type_of(at::ScalarType t) {
  switch (t) {
    case at::kFloat: return 0;
    case at::kHalf: return 1;
    case at::kBFloat16: return 2;
    default: return -1;
  }
}

std::string text(Shape s) {
  std::string o = "(";
  for (size_t i = 0; i < s.size(); ++i) o += (i ? ", " : "") + std::to_string(s[i]);
  return o + ")";
}

// the first token array: its device and type go for all
Tensor leading(const Tensor &t, const char *name, int64_t dims, const char *shape) {
  TORCH_CHECK_VALUE(t.is_cuda(), name, " must be on a GPU device (got ", t.device(), ")");
  TORCH_CHECK_TYPE(type_of(t.scalar_type()) >= 0, name,
                   " must be float32, float16 or bfloat16, got ", t.scalar_type());
  TORCH_CHECK_VALUE(t.dim() == dims, name, " must be ", shape);
  return t.size(-1) > 1 && t.stride(-1) != 1 ? t.contiguous() : t;
}
Tensor tokens(const Tensor &t, const char *name, const Tensor &like) {
  TORCH_CHECK_VALUE(t.device() == like.device() && t.scalar_type() == like.scalar_type(), name,
                    ": device/dtype mismatch");
  return t.dim() && t.size(-1) > 1 && t.stride(-1) != 1 ? t.contiguous() : t;
}
Tensor tokens(const Tensor &t, const char *name, const Tensor &like, Shape shape) {
  TORCH_CHECK_VALUE(t.sizes() == shape, name, " must be ", text(shape), ", got ", text(t.sizes()));
  return tokens(t, name, like);
}
// a contiguous array of a given type
Tensor plain(const Tensor &t, const char *name, Shape shape, at::ScalarType type,
             const Tensor &like) {
  TORCH_CHECK_VALUE(t.device() == like.device() && t.scalar_type() == type, name, " must be ", type,
                    " on ", like.device());
  TORCH_CHECK_VALUE(t.sizes() == shape, name, " must be ", text(shape), ", got ", text(t.sizes()));
  return t.contiguous();
}
Maybe plain(const Maybe &t, const char *name, Shape shape, at::ScalarType type, const Tensor &like) {
  if (!t) return std::nullopt;
  return plain(*t, name, shape, type, like);
}
// the states of a _step call, updated in place: no copy may be made
void check_pool(const Tensor &t, Shape tail, at::ScalarType type, const Tensor &like) {
  TORCH_CHECK_VALUE(t.device() == like.device() && t.scalar_type() == type, "state must be ", type,
                    " on ", like.device());
  TORCH_CHECK_VALUE(t.dim() == static_cast<int64_t>(tail.size()) + 1 && t.sizes().slice(1) == tail,
                    "state must be (n_slots,) + ", text(tail));
  TORCH_CHECK_VALUE(t.is_contiguous(), "state is updated in place and must be contiguous");
}
Maybe check_slots(const Maybe &slots, int64_t B, int64_t n_slots, const Tensor &like) {
  TORCH_CHECK_VALUE(slots || n_slots >= B, "without slots the pool needs a state for every row");
  return plain(slots, "slots", {B}, at::kInt, like);
}

// a size that the structs hold in 32 bits
int32_t small(int64_t n, const char *name) {
  TORCH_CHECK_VALUE(n <= INT32_MAX, name, " must be below 2^31, got ", n);
  return static_cast<int32_t>(n);
}

void *ptr(const Tensor &t) { return t.data_ptr(); }
void *ptr(const Maybe &t) { return t ? t->data_ptr() : nullptr; }
template <typename T>
T *as(const Tensor &t) {
  return static_cast<T *>(t.data_ptr());
}
template <typename T>
T *as(const Maybe &t) {
  return t ? static_cast<T *>(t->data_ptr()) : nullptr;
}

// Enqueues an entry point on the current stream of x's device; with `bytes` of
// workspace where it takes one.
template <typename A>
void call(Op op, const A &a, const Tensor &x, int64_t bytes = -1) {
  const int type = type_of(x.scalar_type());
  void *f = g_entry[op][type];
  const c10::DeviceGuard guard(x.device());
  py::object handle =
      py::reinterpret_steal<py::object>(PyObject_CallFunction(g_stream, "i", x.get_device()));
  if (!handle) throw py::error_already_set();
  void *stream = PyLong_AsVoidPtr(handle.ptr());
  int rc;
  if (bytes < 0) {
    rc = reinterpret_cast<int (*)(const A *, void *)>(f)(&a, stream);
  } else {
    Tensor ws = at::empty({bytes ? bytes : 1}, x.options().dtype(at::kByte));
    rc = reinterpret_cast<int (*)(const A *, void *, size_t, void *)>(f)(
        &a, ws.data_ptr(), static_cast<size_t>(bytes), stream);
  }
  if (rc) {
    const std::string name = std::string("selinv_") + kNames[op] + "_" + kTypes[type];
    py::object r = py::reinterpret_steal<py::object>(
        PyObject_CallFunction(g_failed, "is", rc, name.c_str()));
    if (!r) throw py::error_already_set();
  }
}

Tensor like(const Tensor &t) { return at::empty(t.sizes(), t.options()); }
Maybe like(const Maybe &t) {
  if (!t) return std::nullopt;
  return like(*t);
}

// ------------------------------------------------------- short convolution
struct Conv {
  Tensor x, weight;
  Maybe bias;
  int64_t B, T, C, W;
  selinv_conv_args a = {};
  Conv(const Tensor &x_, const Tensor &weight_, const Maybe &bias_, bool silu, bool token)
      : x(leading(x_, "x", token ? 2 : 3, token ? "[B, C]" : "[B, T, C]")) {
    TORCH_CHECK_VALUE(weight_.dim() == 2 && weight_.size(1) >= 1 &&
                          weight_.size(1) <= SELINV_CONV_MAX_W,
                      "weight must be [C, W] with 1 <= W <= ", SELINV_CONV_MAX_W);
    B = x.size(0), T = token ? 1 : x.size(1), C = x.size(-1), W = weight_.size(1);
    TORCH_CHECK_VALUE(C >= 1, "x needs at least one channel");
    a.C = small(C, "the channels");
    weight = plain(weight_, "weight", {C, W}, at::kFloat, x);
    bias = plain(bias_, "bias", {C}, at::kFloat, x);
    a.B = B, a.T = T, a.W = static_cast<int32_t>(W), a.silu = silu;
    a.x_sb = x.stride(0), a.x_st = token ? 0 : x.stride(1);
    a.x = ptr(x), a.weight = as<float>(weight), a.bias = as<float>(bias);
  }
};

py::tuple short_conv(const Tensor &x, const Tensor &weight, const Maybe &bias, bool silu,
                     const Maybe &state_, const Maybe &lengths_) {
  Conv c(x, weight, bias, silu, false);
  const Maybe state = plain(state_, "state", {c.B, c.W - 1, c.C}, c.x.scalar_type(), c.x);
  const Maybe lengths = plain(lengths_, "lengths", {c.B}, at::kInt, c.x);
  Tensor y = like(c.x), out = at::empty({c.B, c.W - 1, c.C}, c.x.options());
  c.a.state = ptr(state), c.a.lengths = as<int32_t>(lengths);
  c.a.y = ptr(y), c.a.state_out = ptr(out);
  call(kConv, c.a, c.x);
  return py::make_tuple(y, out);
}

Tensor short_conv_step(const Tensor &x, const Tensor &state, const Tensor &weight, const Maybe &bias,
                       bool silu, const Maybe &slots_) {
  Conv c(x, weight, bias, silu, true);
  check_pool(state, {c.W - 1, c.C}, c.x.scalar_type(), c.x);
  const Maybe slots = check_slots(slots_, c.B, state.size(0), c.x);
  Tensor y = like(c.x);
  c.a.n_slots = state.size(0), c.a.state = ptr(state), c.a.slots = as<int32_t>(slots);
  c.a.y = ptr(y);
  call(kConvStep, c.a, c.x);
  return y;
}

py::tuple short_conv_vjp(const Tensor &x, const Tensor &weight, const Maybe &bias,
                         const Tensor &y_bar_, const Maybe &state_out_bar, bool silu,
                         const Maybe &state_, const Maybe &lengths_) {
  Conv c(x, weight, bias, silu, false);
  const Tensor y_bar = tokens(y_bar_, "y_bar", c.x, c.x.sizes());
  const Maybe state = plain(state_, "state", {c.B, c.W - 1, c.C}, c.x.scalar_type(), c.x);
  const Maybe sob =
      plain(state_out_bar, "state_out_bar", {c.B, c.W - 1, c.C}, c.x.scalar_type(), c.x);
  const Maybe lengths = plain(lengths_, "lengths", {c.B}, at::kInt, c.x);
  Tensor xb = like(c.x), wb = like(c.weight);
  const Maybe bb = like(c.bias), sb = like(state);
  c.a.yb_sb = y_bar.stride(0), c.a.yb_st = y_bar.stride(1), c.a.y_bar = ptr(y_bar);
  c.a.state = ptr(state), c.a.state_out_bar = ptr(sob), c.a.lengths = as<int32_t>(lengths);
  c.a.x_bar = ptr(xb), c.a.weight_bar = as<float>(wb), c.a.bias_bar = as<float>(bb);
  c.a.state_bar = ptr(sb);
  call(kConvVjp, c.a, c.x, g_conv_vjp_bytes(c.B, c.T, c.a.C, c.a.W));
  return py::make_tuple(xb, wb, bb, sb);
}

// ------------------------------------------------- head norm and rotation
struct Qk {
  Tensor q, q_weight;
  Maybe k, k_weight, cos, sin, positions;
  selinv_qkrot_args a = {};
  Qk(const Tensor &q_, const Maybe &k_, const Tensor &qw, const Maybe &kw, const Maybe &cos_,
     const Maybe &sin_, const Maybe &positions_, double eps, bool interleaved)
      : q(leading(q_, "q", 4, "[B, T, Hq, D]")) {
    const int64_t B = q.size(0), T = q.size(1), D = q.size(3);
    TORCH_CHECK_VALUE(q.size(2) >= 1 && D >= 1 && D <= SELINV_QKROT_MAX_D,
                      "need at least one query head and 1 <= D <= ", SELINV_QKROT_MAX_D);
    a.Hq = small(q.size(2), "the query heads");
    q_weight = plain(qw, "q_weight", {D}, at::kFloat, q);
    if (k_) {
      k = tokens(*k_, "k", q);
      TORCH_CHECK_VALUE(k->dim() == 4 && k->size(0) == B && k->size(1) == T && k->size(3) == D,
                        "k must be [B, T, Hk, D] matching q");
      TORCH_CHECK_TYPE(kw.has_value(), "k_weight must be a torch.Tensor");
      k_weight = plain(kw, "k_weight", {D}, at::kFloat, q);
    }
    int64_t rows = 0, R = 0;
    if (cos_) {
      TORCH_CHECK_VALUE(cos_->dim() == 2 && 2 * cos_->size(1) <= D,
                        "cos must be [rows, R/2] with R <= D");
      rows = cos_->size(0), R = 2 * cos_->size(1);
      cos = plain(cos_, "cos", {rows, R / 2}, at::kFloat, q);
      TORCH_CHECK_TYPE(sin_.has_value(), "sin must be a torch.Tensor");
      sin = plain(sin_, "sin", {rows, R / 2}, at::kFloat, q);
      TORCH_CHECK_TYPE(positions_ && (positions_->scalar_type() == at::kInt ||
                                      positions_->scalar_type() == at::kLong),
                       "positions must be an int32 or int64 tensor");
      TORCH_CHECK_VALUE(positions_->device() == q.device(), "positions must be on ", q.device());
      const int64_t want[2] = {B, T};
      if (positions_->sizes() == Shape(want)) {
        positions = positions_;
      } else {
        TORCH_CHECK_VALUE(positions_->dim() <= 2 && at::is_expandable_to(positions_->sizes(), want),
                          "positions must be [B, T] or broadcast to it, got ",
                          text(positions_->sizes()));
        positions = positions_->expand(want);
      }
    }
    a.B = B, a.T = T, a.table_rows = rows;
    a.q_sb = q.stride(0), a.q_st = q.stride(1), a.q_sh = q.stride(2);
    a.D = static_cast<int32_t>(D);
    a.R = static_cast<int32_t>(R), a.interleaved = interleaved, a.eps = static_cast<float>(eps);
    a.q = ptr(q), a.q_weight = as<float>(q_weight);
    if (k && k->size(2)) {
      a.Hk = small(k->size(2), "the key heads");
      a.k_sb = k->stride(0), a.k_st = k->stride(1), a.k_sh = k->stride(2);
      a.k = ptr(k), a.k_weight = as<float>(k_weight);
    }
    if (R) {
      a.cos_table = as<float>(cos), a.sin_table = as<float>(sin), a.positions = ptr(positions);
      a.pos_sb = positions->stride(0), a.pos_st = positions->stride(1);
      a.positions_64 = positions->scalar_type() == at::kLong;
    }
  }
};

py::tuple qk_norm_rotate(const Tensor &q, const Maybe &k, const Tensor &qw, const Maybe &kw,
                         const Maybe &cos, const Maybe &sin, const Maybe &positions, double eps,
                         bool interleaved) {
  Qk c(q, k, qw, kw, cos, sin, positions, eps, interleaved);
  Tensor qo = like(c.q);
  const Maybe ko = like(c.k);
  c.a.q_out = ptr(qo), c.a.k_out = ptr(ko);
  call(kQkrot, c.a, c.q);
  return py::make_tuple(qo, ko);
}

py::tuple qk_norm_rotate_vjp(const Tensor &q, const Maybe &k, const Tensor &qw, const Maybe &kw,
                             const Maybe &cos, const Maybe &sin, const Maybe &positions,
                             const Tensor &q_bar, const Maybe &k_bar, double eps,
                             bool interleaved) {
  Qk c(q, k, qw, kw, cos, sin, positions, eps, interleaved);
  const Tensor qb = tokens(q_bar, "q_out_bar", c.q, c.q.sizes());
  Tensor qg = like(c.q), wq = at::empty({c.a.D}, c.q.options().dtype(at::kFloat));
  Maybe kb, kg, wk;
  c.a.qb_sb = qb.stride(0), c.a.qb_st = qb.stride(1), c.a.qb_sh = qb.stride(2);
  c.a.q_bar = ptr(qb), c.a.q_grad = ptr(qg), c.a.q_weight_grad = as<float>(wq);
  if (c.k) {
    TORCH_CHECK_TYPE(k_bar.has_value(), "k_out_bar must be a torch.Tensor");
    kb = tokens(*k_bar, "k_out_bar", c.q, c.k->sizes());
    kg = like(c.k), wk = at::empty({c.a.D}, c.q.options().dtype(at::kFloat));
    c.a.kb_sb = kb->stride(0), c.a.kb_st = kb->stride(1), c.a.kb_sh = kb->stride(2);
    c.a.k_bar = ptr(kb), c.a.k_grad = ptr(kg), c.a.k_weight_grad = as<float>(wk);
  }
  call(kQkrotVjp, c.a, c.q, g_qkrot_vjp_bytes(c.a.B, c.a.T, c.a.D));
  return py::make_tuple(qg, kg, wq, wk);
}

// --------------------------------------------------------- selective scan
struct Scan {
  Tensor x, dt, A, Bm, Cm;
  Maybe D, dt_bias;
  int64_t H, P, G, N;
  selinv_scan_args a = {};
  // on [B, T, ...] arrays, or one token's [B, ...]
  Scan(const Tensor &x_, const Tensor &dt_, const Tensor &A_, const Tensor &Bm_, const Tensor &Cm_,
       const Maybe &D_, const Maybe &bias_, bool softplus, bool token)
      : x(leading(x_, "x", token ? 3 : 4, token ? "[B, H, P]" : "[B, T, H, P]")) {
    const int64_t lead = token ? 1 : 2;
    H = x.size(lead), P = x.size(lead + 1);
    Bm = tokens(Bm_, "Bm", x);
    TORCH_CHECK_VALUE(Bm.dim() == lead + 2 && Bm.sizes().slice(0, lead) == x.sizes().slice(0, lead),
                      "Bm must be ", token ? "[B, G, N]" : "[B, T, G, N]", " matching x");
    G = Bm.size(lead), N = Bm.size(lead + 1);
    TORCH_CHECK_VALUE(P >= 1 && P <= SELINV_SCAN_MAX_P && N >= 1 && N <= SELINV_SCAN_MAX_N,
                      "need 1 <= P <= ", SELINV_SCAN_MAX_P, " and 1 <= N <= ", SELINV_SCAN_MAX_N);
    TORCH_CHECK_VALUE(G >= 1 && H >= 1 && H % G == 0,
                      "the heads must be a multiple of the groups (H=", H, ", G=", G, ")");
    a.H = small(H, "the heads"), a.G = static_cast<int32_t>(G);
    Cm = tokens(Cm_, "Cm", x, Bm.sizes());
    dt = tokens(dt_, "dt", x, x.sizes().slice(0, lead + 1));
    A = plain(A_, "A", {H}, at::kFloat, x);
    D = plain(D_, "D", {H}, at::kFloat, x);
    dt_bias = plain(bias_, "dt_bias", {H}, at::kFloat, x);
    a.B = x.size(0), a.T = token ? 1 : x.size(1);
    a.x_sb = x.stride(0), a.x_sh = x.stride(lead), a.dt_sb = dt.stride(0);
    a.b_sb = Bm.stride(0), a.b_sg = Bm.stride(lead);
    a.c_sb = Cm.stride(0), a.c_sg = Cm.stride(lead);
    if (!token)
      a.x_st = x.stride(1), a.dt_st = dt.stride(1), a.b_st = Bm.stride(1), a.c_st = Cm.stride(1);
    a.P = static_cast<int32_t>(P);
    a.N = static_cast<int32_t>(N), a.softplus = softplus;
    a.x = ptr(x), a.dt = ptr(dt), a.Bm = ptr(Bm), a.Cm = ptr(Cm), a.A = as<float>(A);
    a.D = as<float>(D), a.dt_bias = as<float>(dt_bias);
  }
  std::array<int64_t, 4> states() const { return {a.B, H, P, N}; }
};

py::tuple selective_scan(const Tensor &x, const Tensor &dt, const Tensor &A, const Tensor &Bm,
                         const Tensor &Cm, const Maybe &D, const Maybe &dt_bias, bool softplus,
                         const Maybe &state_, const Maybe &lengths_) {
  Scan c(x, dt, A, Bm, Cm, D, dt_bias, softplus, false);
  const Maybe state = plain(state_, "state", c.states(), at::kFloat, c.x);
  const Maybe lengths = plain(lengths_, "lengths", {c.a.B}, at::kInt, c.x);
  Tensor y = like(c.x), out = at::empty(c.states(), c.x.options().dtype(at::kFloat));
  c.a.state = as<float>(state), c.a.lengths = as<int32_t>(lengths);
  c.a.y = ptr(y), c.a.state_out = as<float>(out);
  call(kScan, c.a, c.x, g_scan_bytes(static_cast<int>(c.x.element_size()), c.a.B,
                                                    c.a.T, c.a.H, c.a.P, c.a.N));
  return py::make_tuple(y, out);
}

Tensor selective_scan_step(const Tensor &x, const Tensor &dt, const Tensor &A, const Tensor &Bm,
                           const Tensor &Cm, const Tensor &state, const Maybe &D,
                           const Maybe &dt_bias, bool softplus, const Maybe &slots_) {
  Scan c(x, dt, A, Bm, Cm, D, dt_bias, softplus, true);
  check_pool(state, {c.H, c.P, c.N}, at::kFloat, c.x);
  const Maybe slots = check_slots(slots_, c.a.B, state.size(0), c.x);
  Tensor y = like(c.x);
  c.a.n_slots = state.size(0), c.a.state = as<float>(state), c.a.slots = as<int32_t>(slots);
  c.a.y = ptr(y);
  call(kScanStep, c.a, c.x);
  return y;
}

py::tuple selective_scan_vjp(const Tensor &x, const Tensor &dt, const Tensor &A, const Tensor &Bm,
                             const Tensor &Cm, const Tensor &y_bar_, const Maybe &state_out_bar,
                             const Maybe &D, const Maybe &dt_bias, bool softplus,
                             const Maybe &state_, const Maybe &lengths_) {
  Scan c(x, dt, A, Bm, Cm, D, dt_bias, softplus, false);
  const Tensor y_bar = tokens(y_bar_, "y_bar", c.x, c.x.sizes());
  const Maybe sob = plain(state_out_bar, "state_out_bar", c.states(), at::kFloat, c.x);
  const Maybe state = plain(state_, "state", c.states(), at::kFloat, c.x);
  const Maybe lengths = plain(lengths_, "lengths", {c.a.B}, at::kInt, c.x);
  Tensor xb = like(c.x), dtb = like(c.dt), Ab = like(c.A), Bb = like(c.Bm), Cb = like(c.Cm);
  const Maybe Db = like(c.D), bb = like(c.dt_bias), sb = like(state);
  c.a.yb_sb = y_bar.stride(0), c.a.yb_st = y_bar.stride(1), c.a.yb_sh = y_bar.stride(2);
  c.a.y_bar = ptr(y_bar), c.a.state_out_bar = as<float>(sob);
  c.a.state = as<float>(state), c.a.lengths = as<int32_t>(lengths);
  c.a.x_bar = ptr(xb), c.a.dt_bar = ptr(dtb), c.a.B_bar = ptr(Bb), c.a.C_bar = ptr(Cb);
  c.a.A_bar = as<float>(Ab), c.a.D_bar = as<float>(Db), c.a.dt_bias_bar = as<float>(bb);
  c.a.state_bar = as<float>(sb);
  const auto &a = c.a;
  call(kScanVjp, a, c.x,
       c.x.scalar_type() == at::kBFloat16
           ? g_scan_vjp_bf16_bytes(a.B, a.T, a.H, a.P, a.G, a.N)
           : g_scan_vjp_bytes(static_cast<int>(c.x.element_size()), a.B, a.T, a.H, a.P, a.G, a.N));
  return py::make_tuple(xb, dtb, Ab, Bb, Cb, Db, bb, sb);
}

// Addresses of the loaded library's functions by name, the stream query and the
// function that raises for a status.
void bind(const std::function<uintptr_t(const std::string &)> &address, const py::object &stream,
          const py::object &failed) {
  for (int op = 0; op < kOps; ++op)
    for (int type = 0; type < 3; ++type)
      g_entry[op][type] = reinterpret_cast<void *>(
          address(std::string("selinv_") + kNames[op] + "_" + kTypes[type]));
  auto set = [&](auto &f, const char *name) {
    f = reinterpret_cast<std::decay_t<decltype(f)>>(address(name));
  };
  set(g_conv_vjp_bytes, "selinv_conv_vjp_workspace_bytes");
  set(g_qkrot_vjp_bytes, "selinv_qkrot_vjp_workspace_bytes");
  set(g_scan_bytes, "selinv_scan_workspace_bytes");
  set(g_scan_vjp_bytes, "selinv_scan_vjp_workspace_bytes");
  set(g_scan_vjp_bf16_bytes, "selinv_scan_vjp_bf16_workspace_bytes");
  Py_XDECREF(g_stream);
  Py_XDECREF(g_failed);
  g_stream = stream.inc_ref().ptr();
  g_failed = failed.inc_ref().ptr();
}

}  // namespace

PYBIND11_MODULE(TORCH_EXTENSION_NAME, m) {
  m.def("bind", &bind);
  m.def("short_conv", &short_conv);
  m.def("short_conv_step", &short_conv_step);
  m.def("short_conv_vjp", &short_conv_vjp);
  m.def("qk_norm_rotate", &qk_norm_rotate);
  m.def("qk_norm_rotate_vjp", &qk_norm_rotate_vjp);
  m.def("selective_scan", &selective_scan);
  m.def("selective_scan_step", &selective_scan_step);
  m.def("selective_scan_vjp", &selective_scan_vjp);
}
