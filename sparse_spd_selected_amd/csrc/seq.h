// seq.h -- shared by the sequence-mixer kernels: element types, vectors of
// them, small reductions, and the launch functions that seq_abi.cpp calls.
#pragma once

#include <hip/hip_runtime.h>

#include <cstddef>
#include <cstdint>

#include "selinv_seq.h"

namespace selinv {

// ---------------------------------------------------------------- launches
// E: element of the token arrays (float, _Float16, __bf16).  Arguments are
// validated by the caller.
template <typename E>
hipError_t conv_launch(const selinv_conv_args &a, hipStream_t s);
template <typename E>
hipError_t conv_step_launch(const selinv_conv_args &a, hipStream_t s);
size_t conv_vjp_workspace_bytes(int64_t B, int64_t T, int32_t C, int32_t W);
template <typename E>
hipError_t conv_vjp_launch(const selinv_conv_args &a, void *ws, hipStream_t s);

template <typename E>
hipError_t qkrot_launch(const selinv_qkrot_args &a, hipStream_t s);
size_t qkrot_vjp_workspace_bytes(int64_t B, int64_t T, int32_t D);
template <typename E>
hipError_t qkrot_vjp_launch(const selinv_qkrot_args &a, void *ws, hipStream_t s);

size_t scan_workspace_bytes(int dtype_bytes, int64_t B, int64_t T, int32_t H, int32_t P, int32_t N);
template <typename E>
hipError_t scan_launch(const selinv_scan_args &a, void *ws, hipStream_t s);
template <typename E>
hipError_t scan_step_launch(const selinv_scan_args &a, hipStream_t s);
template <typename E>
size_t scan_vjp_workspace_bytes(int64_t B, int64_t T, int32_t H, int32_t P, int32_t G, int32_t N);
// whether the gradient's workgroups, one a chunk and group, fit a launch
template <typename E>
bool scan_vjp_fits(int64_t B, int64_t T, int32_t G);
template <typename E>
hipError_t scan_vjp_launch(const selinv_scan_args &a, void *ws, hipStream_t s);

namespace seq {

// -------------------------------------------------------- vectors of elements
// V elements of E that move as one load or store.
template <typename E, int V>
struct Vec {
  typedef E Reg __attribute__((ext_vector_type(V)));
  Reg e;
};

template <typename E, int V>
__device__ inline Vec<E, V> vload(const E *p) {
  return *reinterpret_cast<const Vec<E, V> *>(p);
}
template <typename E, int V>
__device__ inline void vstore(E *p, const Vec<E, V> &v) {
  *reinterpret_cast<Vec<E, V> *>(p) = v;
}
template <typename E, int V>
__device__ inline Vec<E, V> vzero() {
  Vec<E, V> v;
  v.e = static_cast<E>(0.0f);
  return v;
}
// widening is exact, narrowing rounds to nearest even
template <typename E, int V>
__device__ inline void widen(const Vec<E, V> &v, float (&f)[V]) {
#pragma unroll
  for (int i = 0; i < V; ++i) f[i] = static_cast<float>(v.e[i]);
}
template <typename E, int V>
__device__ inline Vec<E, V> narrow(const float (&f)[V]) {
  Vec<E, V> v;
#pragma unroll
  for (int i = 0; i < V; ++i) v.e[i] = static_cast<E>(f[i]);
  return v;
}

// whether rows of `n` elements at p with these strides can be moved V at a time
template <typename E, int V>
inline bool whole_vectors(const void *p, int64_t n, int64_t s0 = 0, int64_t s1 = 0,
                          int64_t s2 = 0) {
  return reinterpret_cast<uintptr_t>(p) % (sizeof(E) * V) == 0 && n % V == 0 && s0 % V == 0 &&
         s1 % V == 0 && s2 % V == 0;
}

__device__ inline int row_length(const int32_t *lengths, int64_t b, int64_t T) {
  if (!lengths) return static_cast<int>(T);
  const int n = lengths[b];
  return n < 0 ? 0 : n > T ? static_cast<int>(T) : n;
}

// 1 / (1 + exp(-v)): exp2 and reciprocal of the hardware, both within an ulp
// or two of float32; exp(-v) = inf gives 0
__device__ inline float sigmoid(float v) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.442695040888963f * v));
}

// sum over W neighbouring lanes (a power of two), in every one of them: within
// a row of 16 lanes by data-parallel moves, beyond by exchange
template <int CTRL>
__device__ inline float dpp_move(float v) {
  return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), CTRL, 0xf, 0xf, true));
}
template <int W>
__device__ inline float lane_sum(float v) {
  if (W > 1) v += dpp_move<0xb1>(v);   // neighbours within pairs
  if (W > 2) v += dpp_move<0x4e>(v);   // pairs within quads
  if (W > 4) v += dpp_move<0x141>(v);  // quads within halves of a row, mirrored
  if (W > 8) v += dpp_move<0x140>(v);  // halves of a row, mirrored
  if (W > 16) v += __shfl_xor(v, 16, 64);
  if (W > 32) v += __shfl_xor(v, 32, 64);
  return v;
}

inline unsigned blocks_for(int64_t threads, int per = 256) {
  return static_cast<unsigned>((threads + per - 1) / per);
}

}  // namespace seq
}  // namespace selinv
