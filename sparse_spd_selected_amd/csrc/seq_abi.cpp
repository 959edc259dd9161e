// seq_abi.cpp -- the extern "C" entry points declared in include/selinv_seq.h:
// argument validation, workspace checks and dispatch to the kernels.  No
// device memory is allocated here.
#include <hip/hip_runtime.h>

#include "seq.h"

namespace {

// Bounds that keep every product of sizes below 2^63 and every launch below
// 2^32 threads (the scan's gradient has one of its own, by the chunks).
constexpr int64_t kTokens = int64_t(1) << 30;
constexpr int32_t kChannels = 1 << 27;
inline bool bad_batch(int64_t B, int64_t T, int64_t most = kTokens) {
  return B < 0 || T < 0 || B >= most || T >= most || (B > 0 && T + 128 > kTokens / B) ||
         (T > 0 && B >= (most + T - 1) / T);
}
inline bool bad_workspace(const void *ws, size_t have, size_t need) {
  return have < need || (need && !ws) || (reinterpret_cast<uintptr_t>(ws) & 255);
}
// arrays of E that the kernels index by element
template <typename E>
inline bool skewed(const void *p) {
  return reinterpret_cast<uintptr_t>(p) % sizeof(E) != 0;
}
inline int status(hipError_t e) { return e == hipSuccess ? SELINV_OK : SELINV_ERR_HIP; }

// ------------------------------------------------------ short convolution
inline bool bad_conv(const selinv_conv_args &a) {
  return bad_batch(a.B, a.T) || a.C < 1 || a.C > kChannels || a.W < 1 || a.W > SELINV_CONV_MAX_W ||
         // a thread per four tokens and channel at worst
         (a.B > 0 && a.T + 128 > kTokens * 16 / a.B / a.C);
}

template <typename E>
int conv_entry(const selinv_conv_args *p, void *stream) {
  if (!p || bad_conv(*p)) return SELINV_ERR_INVALID_ARG;
  const selinv_conv_args &a = *p;
  if (a.B > 0 && (!a.weight || (a.T > 0 && (!a.x || !a.y)))) return SELINV_ERR_INVALID_ARG;
  if (skewed<E>(a.x) || skewed<E>(a.state) || skewed<E>(a.y) || skewed<E>(a.state_out) ||
      skewed<float>(a.weight) || skewed<float>(a.bias))
    return SELINV_ERR_INVALID_ARG;
  return status(selinv::conv_launch<E>(a, static_cast<hipStream_t>(stream)));
}

template <typename E>
int conv_step_entry(const selinv_conv_args *p, void *stream) {
  if (!p || bad_conv(*p) || p->n_slots < 0) return SELINV_ERR_INVALID_ARG;
  const selinv_conv_args &a = *p;
  if (a.B > 0 && (!a.weight || !a.x || !a.y || (a.W > 1 && a.n_slots > 0 && !a.state)))
    return SELINV_ERR_INVALID_ARG;
  if (skewed<E>(a.x) || skewed<E>(a.state) || skewed<E>(a.y) || skewed<float>(a.weight) ||
      skewed<float>(a.bias))
    return SELINV_ERR_INVALID_ARG;
  return status(selinv::conv_step_launch<E>(a, static_cast<hipStream_t>(stream)));
}

template <typename E>
int conv_vjp_entry(const selinv_conv_args *p, void *ws, size_t ws_bytes, void *stream) {
  if (!p || bad_conv(*p)) return SELINV_ERR_INVALID_ARG;
  const selinv_conv_args &a = *p;
  if (!a.weight_bar || (a.B > 0 && (!a.weight || (a.T > 0 && (!a.x || !a.y_bar || !a.x_bar)))))
    return SELINV_ERR_INVALID_ARG;
  if (skewed<E>(a.x) || skewed<E>(a.state) || skewed<E>(a.y_bar) || skewed<E>(a.state_out_bar) ||
      skewed<E>(a.x_bar) || skewed<E>(a.state_bar) || skewed<float>(a.weight) ||
      skewed<float>(a.bias) || skewed<float>(a.weight_bar) || skewed<float>(a.bias_bar))
    return SELINV_ERR_INVALID_ARG;
  if (bad_workspace(ws, ws_bytes, selinv::conv_vjp_workspace_bytes(a.B, a.T, a.C, a.W)))
    return SELINV_ERR_INVALID_ARG;
  return status(selinv::conv_vjp_launch<E>(a, ws, static_cast<hipStream_t>(stream)));
}

// ------------------------------------------------- head norm and rotation
constexpr int64_t kQkTokens = (int64_t(1) << 26) - 3;  // below this: a wavefront each
constexpr int32_t kHeads = 1 << 16;
inline bool bad_qkrot(const selinv_qkrot_args &a) {
  if (bad_batch(a.B, a.T, kQkTokens) || a.Hq < 1 || a.Hk < 0 || a.Hq > kHeads || a.Hk > kHeads ||
      a.D < 1 || a.D > SELINV_QKROT_MAX_D || a.R < 0 || a.R > a.D || (a.R & 1) ||
      a.table_rows < 0)
    return true;
  if (a.B * a.T == 0) return false;
  if (!a.q || !a.q_weight || (a.Hk > 0 && (!a.k || !a.k_weight))) return true;
  return a.R > 0 && (!a.positions || (a.table_rows > 0 && (!a.cos_table || !a.sin_table)));
}
template <typename E>
inline bool skewed_qkrot(const selinv_qkrot_args &a) {
  return skewed<E>(a.q) || skewed<E>(a.k) || skewed<float>(a.q_weight) ||
         skewed<float>(a.k_weight) || skewed<float>(a.cos_table) || skewed<float>(a.sin_table) ||
         (a.positions_64 ? skewed<int64_t>(a.positions) : skewed<int32_t>(a.positions));
}

template <typename E>
int qkrot_entry(const selinv_qkrot_args *p, void *stream) {
  if (!p || bad_qkrot(*p) || skewed_qkrot<E>(*p)) return SELINV_ERR_INVALID_ARG;
  const selinv_qkrot_args &a = *p;
  if (a.B * a.T > 0 && (!a.q_out || (a.Hk > 0 && !a.k_out))) return SELINV_ERR_INVALID_ARG;
  if (skewed<E>(a.q_out) || skewed<E>(a.k_out)) return SELINV_ERR_INVALID_ARG;
  return status(selinv::qkrot_launch<E>(a, static_cast<hipStream_t>(stream)));
}

template <typename E>
int qkrot_vjp_entry(const selinv_qkrot_args *p, void *ws, size_t ws_bytes, void *stream) {
  if (!p || bad_qkrot(*p) || skewed_qkrot<E>(*p)) return SELINV_ERR_INVALID_ARG;
  const selinv_qkrot_args &a = *p;
  if (!a.q_weight_grad || (a.Hk > 0 && !a.k_weight_grad)) return SELINV_ERR_INVALID_ARG;
  if (a.B * a.T > 0 && (!a.q_bar || !a.q_grad || (a.Hk > 0 && (!a.k_bar || !a.k_grad))))
    return SELINV_ERR_INVALID_ARG;
  if (skewed<E>(a.q_bar) || skewed<E>(a.k_bar) || skewed<E>(a.q_grad) || skewed<E>(a.k_grad) ||
      skewed<float>(a.q_weight_grad) || skewed<float>(a.k_weight_grad))
    return SELINV_ERR_INVALID_ARG;
  if (bad_workspace(ws, ws_bytes, selinv::qkrot_vjp_workspace_bytes(a.B, a.T, a.D)))
    return SELINV_ERR_INVALID_ARG;
  return status(selinv::qkrot_vjp_launch<E>(a, ws, static_cast<hipStream_t>(stream)));
}

// --------------------------------------------------------- selective scan
inline bool bad_scan(const selinv_scan_args &a) {
  if (bad_batch(a.B, a.T) || a.H < 1 || a.G < 1 || a.H > kHeads || a.H % a.G || a.P < 1 ||
      a.P > SELINV_SCAN_MAX_P || a.N < 1 || a.N > SELINV_SCAN_MAX_N)
    return true;
  // workgroups of a row and head: up to four tiles of P
  if (a.B * a.H > (int64_t(1) << 20) || (a.B > 0 && a.T + 128 > kTokens * 64 / a.B / a.H)) return true;
  return a.B > 0 && (!a.A || (a.T > 0 && (!a.x || !a.dt || !a.Bm || !a.Cm)));
}
template <typename E>
inline bool skewed_scan(const selinv_scan_args &a) {
  return skewed<E>(a.x) || skewed<E>(a.dt) || skewed<E>(a.Bm) || skewed<E>(a.Cm) ||
         skewed<float>(a.A) || skewed<float>(a.D) || skewed<float>(a.dt_bias) ||
         skewed<float>(a.state) || skewed<float>(a.state_out);
}

template <typename E>
int scan_entry(const selinv_scan_args *p, void *ws, size_t ws_bytes, void *stream) {
  if (!p || bad_scan(*p) || skewed_scan<E>(*p) || skewed<E>(p->y)) return SELINV_ERR_INVALID_ARG;
  selinv_scan_args a = *p;
  a.y_bar = nullptr;  // the reverse mode's alone
  if (a.B * a.T > 0 && !a.y) return SELINV_ERR_INVALID_ARG;
  if (bad_workspace(ws, ws_bytes,
                    selinv::scan_workspace_bytes(sizeof(E), a.B, a.T, a.H, a.P, a.N)))
    return SELINV_ERR_INVALID_ARG;
  return status(selinv::scan_launch<E>(a, ws, static_cast<hipStream_t>(stream)));
}

template <typename E>
int scan_step_entry(const selinv_scan_args *p, void *stream) {
  if (!p || p->T != 1 || p->n_slots < 0 || bad_scan(*p) || skewed_scan<E>(*p) || skewed<E>(p->y))
    return SELINV_ERR_INVALID_ARG;
  if (p->B > 0 && (!p->y || (p->n_slots > 0 && !p->state))) return SELINV_ERR_INVALID_ARG;
  return status(selinv::scan_step_launch<E>(*p, static_cast<hipStream_t>(stream)));
}

template <typename E>
int scan_vjp_entry(const selinv_scan_args *p, void *ws, size_t ws_bytes, void *stream) {
  if (!p || bad_scan(*p) || skewed_scan<E>(*p)) return SELINV_ERR_INVALID_ARG;
  const selinv_scan_args &a = *p;
  if (!selinv::scan_vjp_fits<E>(a.B, a.T, a.G)) return SELINV_ERR_INVALID_ARG;
  if (!a.A_bar) return SELINV_ERR_INVALID_ARG;
  if (a.B * a.T > 0 && (!a.y_bar || !a.x_bar || !a.dt_bar || !a.B_bar || !a.C_bar))
    return SELINV_ERR_INVALID_ARG;
  if (skewed<E>(a.y_bar) || skewed<E>(a.x_bar) || skewed<E>(a.dt_bar) || skewed<E>(a.B_bar) ||
      skewed<E>(a.C_bar) || skewed<float>(a.state_out_bar) || skewed<float>(a.A_bar) ||
      skewed<float>(a.D_bar) || skewed<float>(a.dt_bias_bar) || skewed<float>(a.state_bar))
    return SELINV_ERR_INVALID_ARG;
  if (bad_workspace(ws, ws_bytes,
                    selinv::scan_vjp_workspace_bytes<E>(a.B, a.T, a.H, a.P, a.G, a.N)))
    return SELINV_ERR_INVALID_ARG;
  return status(selinv::scan_vjp_launch<E>(a, ws, static_cast<hipStream_t>(stream)));
}

// sizes alone, for the workspace queries
inline bool bad_scan_sizes(int64_t B, int64_t T, int32_t H, int32_t P, int32_t G, int32_t N) {
  selinv_scan_args a = {};
  a.B = B, a.T = T, a.H = H, a.P = P, a.G = G, a.N = N;
  a.A = reinterpret_cast<const float *>(16);
  a.x = a.dt = a.Bm = a.Cm = a.A;
  return bad_scan(a);
}

}  // namespace

extern "C" {

size_t selinv_scan_workspace_bytes(int dtype_bytes, int64_t B, int64_t T, int32_t H, int32_t P,
                                   int32_t N) {
  return bad_scan_sizes(B, T, H, P, 1, N) ? 0
                                          : selinv::scan_workspace_bytes(dtype_bytes, B, T, H, P, N);
}
size_t selinv_scan_vjp_workspace_bytes(int dtype_bytes, int64_t B, int64_t T, int32_t H, int32_t P,
                                       int32_t G, int32_t N) {
  if (bad_scan_sizes(B, T, H, P, G, N)) return 0;
  if (dtype_bytes == 4) return selinv::scan_vjp_workspace_bytes<float>(B, T, H, P, G, N);
  const size_t f16 = selinv::scan_vjp_workspace_bytes<_Float16>(B, T, H, P, G, N);
  const size_t bf16 = selinv::scan_vjp_workspace_bytes<__bf16>(B, T, H, P, G, N);
  return f16 > bf16 ? f16 : bf16;
}
size_t selinv_scan_vjp_bf16_workspace_bytes(int64_t B, int64_t T, int32_t H, int32_t P, int32_t G,
                                            int32_t N) {
  return bad_scan_sizes(B, T, H, P, G, N)
             ? 0
             : selinv::scan_vjp_workspace_bytes<__bf16>(B, T, H, P, G, N);
}

size_t selinv_conv_vjp_workspace_bytes(int64_t B, int64_t T, int32_t C, int32_t W) {
  selinv_conv_args a = {};
  a.B = B, a.T = T, a.C = C, a.W = W;
  return bad_conv(a) ? 0 : selinv::conv_vjp_workspace_bytes(B, T, C, W);
}
size_t selinv_qkrot_vjp_workspace_bytes(int64_t B, int64_t T, int32_t D) {
  if (bad_batch(B, T, kQkTokens) || D < 1 || D > SELINV_QKROT_MAX_D) return 0;
  return selinv::qkrot_vjp_workspace_bytes(B, T, D);
}

#define SELINV_SEQ_ENTRIES(SFX, E)                                                             \
  int selinv_conv_##SFX(const selinv_conv_args *a, void *stream) {                             \
    return conv_entry<E>(a, stream);                                                           \
  }                                                                                            \
  int selinv_conv_step_##SFX(const selinv_conv_args *a, void *stream) {                        \
    return conv_step_entry<E>(a, stream);                                                      \
  }                                                                                            \
  int selinv_conv_vjp_##SFX(const selinv_conv_args *a, void *ws, size_t n, void *stream) {     \
    return conv_vjp_entry<E>(a, ws, n, stream);                                                \
  }                                                                                            \
  int selinv_qkrot_##SFX(const selinv_qkrot_args *a, void *stream) {                           \
    return qkrot_entry<E>(a, stream);                                                          \
  }                                                                                            \
  int selinv_qkrot_vjp_##SFX(const selinv_qkrot_args *a, void *ws, size_t n, void *stream) {   \
    return qkrot_vjp_entry<E>(a, ws, n, stream);                                               \
  }                                                                                            \
  int selinv_scan_##SFX(const selinv_scan_args *a, void *ws, size_t n, void *stream) {         \
    return scan_entry<E>(a, ws, n, stream);                                                    \
  }                                                                                            \
  int selinv_scan_step_##SFX(const selinv_scan_args *a, void *stream) {                        \
    return scan_step_entry<E>(a, stream);                                                      \
  }                                                                                            \
  int selinv_scan_vjp_##SFX(const selinv_scan_args *a, void *ws, size_t n, void *stream) {     \
    return scan_vjp_entry<E>(a, ws, n, stream);                                                \
  }

SELINV_SEQ_ENTRIES(f32, float)
SELINV_SEQ_ENTRIES(f16, _Float16)
SELINV_SEQ_ENTRIES(bf16, __bf16)

}  // extern "C"
