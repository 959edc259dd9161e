// short_conv.hip -- short causal convolution of every channel (gfx950).
//
//   v[t] = bias + sum_j w[j] whole[t + j],  whole = [state, x],  y = silu(v)
//
// One multiply-add per tap and one exponential per element against two
// elements moved: HBM bounds it.  A thread owns V neighbouring channels (one
// 16-byte vector) of a run of tokens and slides the W-tap window through
// registers, so every element is read from HBM once; the W - 1 tokens before
// a run come out of the cache.
//
// Measured in 16 bits, four taps (a large copy reaches 5.1 TB/s): forwards over
// 6 x 1531 tokens of 2304 channels 21.5 us, 3.9 TB/s; reverse mode of 8 x 2048
// tokens of 4352 channels 99 us with the parameters' sums, 4.3 TB/s; a token
// of 2304 channels 4 us, a launch.
#include <type_traits>

#include "seq.h"

namespace selinv {
namespace {

using namespace seq;

// x[t], t >= 0
template <typename E, int V>
__device__ inline Vec<E, V> token_at(const selinv_conv_args &a, int64_t b, int t, int c) {
  return vload<E, V>(static_cast<const E *>(a.x) + b * a.x_sb + t * a.x_st + c);
}

// token t of `whole` minus the state's W - 1, i.e. x[t], or the past for t < 0
template <typename E, int V>
__device__ inline Vec<E, V> whole_at(const selinv_conv_args &a, int64_t b, int t, int c) {
  if (t >= 0) return token_at<E, V>(a, b, t, c);
  if (!a.state) return vzero<E, V>();
  return vload<E, V>(static_cast<const E *>(a.state) + (b * (a.W - 1) + a.W - 1 + t) * a.C + c);
}

// Filters of 2, 3 and 4 taps have kernels of their own (K = W); any other W
// runs on K = 8, where the taps before the filter's first are skipped.
template <int K>
__device__ inline bool used(const selinv_conv_args &a, int j) {
  return K < 8 || j >= K - a.W;
}

// the taps of V channels, the last one at index K - 1
template <int K, int V>
__device__ inline void load_taps(const selinv_conv_args &a, int c, float (&w)[K][V],
                                 float (&bias)[V]) {
  const bool rows = K == 4 && reinterpret_cast<uintptr_t>(a.weight) % 16 == 0;  // W = 4
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const float *p = a.weight + static_cast<int64_t>(c + i) * a.W;
    if (rows) {
      const Vec<float, 4> v = vload<float, 4>(p);
#pragma unroll
      for (int j = 0; j < K; ++j) w[j][i] = v.e[j & 3];
    } else {
#pragma unroll
      for (int j = 0; j < K; ++j) {
        const int jj = K < 8 ? j : j - (K - a.W);
        w[j][i] = jj >= 0 ? p[jj] : 0.0f;
      }
    }
    bias[i] = a.bias ? a.bias[c + i] : 0.0f;
  }
}

// K: taps compiled for (the filter's W <= K); TT: tokens of a run
template <typename E, int V, int K, int TT>
__global__ __launch_bounds__(256) void conv_kernel(selinv_conv_args a, unsigned nc, unsigned runs) {
  const unsigned id = blockIdx.x * 256 + threadIdx.x, br = id / nc;
  const int c = static_cast<int>(id % nc) * V;
  const int64_t b = br / runs;
  if (b >= a.B) return;
  const int t0 = static_cast<int>(br % runs) * TT;
  const int len = row_length(a.lengths, b, a.T);
  const int nt = min(TT, static_cast<int>(a.T) - t0);

  Vec<E, V> raw[K - 1 + TT];
#pragma unroll
  for (int j = 0; j < K - 1 + TT; ++j) {
    const int t = t0 + j - (K - 1);
    if (j < K - 1)
      raw[j] = (t < len && t >= 1 - a.W) ? whole_at<E, V>(a, b, t, c) : vzero<E, V>();
    else
      raw[j] = t < len ? token_at<E, V>(a, b, t, c) : vzero<E, V>();
  }
  float w[K][V], bias[V];
  load_taps<K, V>(a, c, w, bias);
  E *y = static_cast<E *>(a.y) + (b * a.T + t0) * a.C + c;
  float win[K][V];
#pragma unroll
  for (int j = 0; j < K - 1; ++j) widen(raw[j], win[j]);
#pragma unroll
  for (int k = 0; k < TT; ++k) {
    widen(raw[K - 1 + k], win[K - 1]);
    float v[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      v[i] = bias[i];
#pragma unroll
      for (int j = 0; j < K; ++j)
        if (used<K>(a, j)) v[i] = fmaf(w[j][i], win[j][i], v[i]);
      if (a.silu) v[i] *= sigmoid(v[i]);
      if (t0 + k >= len) v[i] = 0.0f;
    }
    if (k < nt) vstore<E, V>(y + static_cast<int64_t>(k) * a.C, narrow<E, V>(v));
#pragma unroll
    for (int j = 0; j + 1 < K; ++j)
#pragma unroll
      for (int i = 0; i < V; ++i) win[j][i] = win[j + 1][i];
  }
  if (a.state_out && t0 == 0) {
    E *out = static_cast<E *>(a.state_out) + b * (a.W - 1) * a.C + c;
    for (int j = 0; j < a.W - 1; ++j)
      vstore<E, V>(out + static_cast<int64_t>(j) * a.C,
                   whole_at<E, V>(a, b, len + j - (a.W - 1), c));
  }
}

// One token per row.  The thread that owns a channel reads its W - 1 past
// tokens, writes them back one place on and appends x.
template <typename E, int V, int K>
__global__ __launch_bounds__(256) void conv_step_kernel(selinv_conv_args a, unsigned nc) {
  const unsigned id = blockIdx.x * 256 + threadIdx.x;
  const int c = static_cast<int>(id % nc) * V;
  const int64_t b = id / nc;
  if (b >= a.B) return;
  E *y = static_cast<E *>(a.y) + b * a.C + c;
  const int64_t slot = a.slots ? a.slots[b] : b;
  if (slot < 0 || slot >= a.n_slots) {
    vstore<E, V>(y, vzero<E, V>());
    return;
  }
  E *st = static_cast<E *>(const_cast<void *>(a.state)) + slot * (a.W - 1) * a.C + c;
  Vec<E, V> raw[K];
#pragma unroll
  for (int j = 0; j < K - 1; ++j) {
    const int jj = K < 8 ? j : j - (K - a.W);
    raw[j] = jj >= 0 ? vload<E, V>(st + static_cast<int64_t>(jj) * a.C) : vzero<E, V>();
  }
  raw[K - 1] = vload<E, V>(static_cast<const E *>(a.x) + b * a.x_sb + c);
  float w[K][V], bias[V], v[V];
  load_taps<K, V>(a, c, w, bias);
#pragma unroll
  for (int i = 0; i < V; ++i) v[i] = bias[i];
#pragma unroll
  for (int j = 0; j < K; ++j) {
    float f[V];
    widen(raw[j], f);
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (used<K>(a, j)) v[i] = fmaf(w[j][i], f[i], v[i]);
  }
#pragma unroll
  for (int j = 0; j + 1 < K; ++j) {
    const int jj = K < 8 ? j : j - (K - a.W);
    if (jj >= 0) vstore<E, V>(st + static_cast<int64_t>(jj) * a.C, raw[j + 1]);
  }
  if (a.silu)
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] *= sigmoid(v[i]);
  vstore<E, V>(y, narrow<E, V>(v));
}

// ------------------------------------------------------------ reverse mode
//   g[t] = y_bar[t] silu'(v[t]),  whole_bar[t + j] += w[j] g[t],
//   weight_bar[j] = sum g[t] whole[t + j],  bias_bar = sum g[t]
// with v recomputed from x.  A wavefront's lanes own 64 channel vectors, a
// workgroup four runs of RUN tokens; the W - 1 tokens of g past a run are
// recomputed from cached inputs.  Parameter sums of a workgroup's tokens go to
// the workspace, [tile][K + 1][C], and are added up in tile order.
//
// A run is a chain of steps, so small calls get short ones: eight tokens below
// 2^23 elements, else 32 (of 8 x 2048 tokens of 4352 channels runs of 16, 32 and 64
// take 109 us, 104 and 105, in float32 with 2304 channels 100, 102 and 115; four taps, 16 bits: 300 tokens of 2304 channels 10 us
// with eight, 19 with 32; 2000 tokens 17 and 20; 4096 23 and 24; 8192 36 and 31).
inline int run_for(int64_t B, int64_t T, int32_t C) { return B * T * C < 1 << 23 ? 8 : 32; }

template <typename E, int V, int K, int RUN>
__global__ __launch_bounds__(256) void conv_vjp_kernel(selinv_conv_args a, int ctiles, int ttiles,
                                                       float *part) {
  __shared__ float red[3][64 * V];
  constexpr int kAhead = K < 8 ? 4 : 8;  // K - 1 or more: the tail's tokens are among them
  const int lane = threadIdx.x & 63, run = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t blk = blockIdx.x;
  const int c = (static_cast<int>(blk % ctiles) * 64 + lane) * V;
  const int64_t bt = blk / ctiles;  // tile index, b-major
  const int64_t b = bt / ttiles;
  const int t0 = static_cast<int>(bt % ttiles) * (4 * RUN) + run * RUN;
  const int len = row_length(a.lengths, b, a.T);
  const bool mine = c < a.C;
  float dw[K][V] = {}, db[V] = {};
  if (mine) {
    float w[K][V], bias[V];
    load_taps<K, V>(a, c, w, bias);
    const E *yb = static_cast<const E *>(a.y_bar) + b * a.yb_sb + c;
    const E *sob = static_cast<const E *>(a.state_out_bar) + b * (a.W - 1) * a.C + c;
    // the cotangent that whole[W - 1 + t] gets from state_out
    auto from_out = [&](int t, float (&acc)[V]) {
      const int j = t + a.W - 1 - len;
      if (j < 0) return;
      float f[V];
      widen(vload<E, V>(sob + static_cast<int64_t>(j) * a.C), f);
#pragma unroll
      for (int i = 0; i < V; ++i) acc[i] += f[i];
    };
    float win[K][V], g[K][V] = {};
#pragma unroll
    for (int j = 0; j < K - 1; ++j) {
      const int t = t0 + j - (K - 1);
      widen((t < len && t >= 1 - a.W) ? whole_at<E, V>(a, b, t, c) : vzero<E, V>(), win[j]);
    }
    E *xb = static_cast<E *>(a.x_bar) + b * a.T * a.C + c;
    // kAhead tokens at a time, the next ones under way.  g[K - 1] is the newest,
    // at t; x_bar of t - (K - 1) is complete with it.
    Vec<E, V> nx[kAhead], ny[kAhead];
    auto fetch = [&](int k) {
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int t = t0 + k + u;
        nx[u] = ny[u] = vzero<E, V>();
        if (k + u < RUN + K - 1 && t < len) {
          nx[u] = token_at<E, V>(a, b, t, c);
          ny[u] = vload<E, V>(yb + t * a.yb_st);
        }
      }
    };
    // `own`: a token of this run; those past it only complete x_bar.  Past the row's
    // end nothing may come of what the window still holds, which a cotangent of zero
    // would pass on where it is not finite: chosen, not multiplied away.
    auto token = [&](int k, const Vec<E, V> &x, const Vec<E, V> &y, auto own) {
      const bool in = t0 + k < len;
      widen(x, win[K - 1]);
      float yv[V], done[V];
      widen(y, yv);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        float v = bias[i];
#pragma unroll
        for (int j = 0; j < K; ++j)
          if (used<K>(a, j)) v = fmaf(w[j][i], win[j][i], v);
        float gi = yv[i];
        if (a.silu) {
          const float sg = sigmoid(v);
          gi *= sg * fmaf(v, 1.0f - sg, 1.0f);
        }
        if (!in) gi = 0.0f;
        g[K - 1][i] = gi;
        if (own) {
          db[i] += gi;
#pragma unroll
          for (int j = 0; j < K; ++j) {
            const float sum = fmaf(gi, win[j][i], dw[j][i]);
            dw[j][i] = in ? sum : dw[j][i];
          }
        }
        done[i] = 0.0f;
#pragma unroll
        for (int j = 0; j < K; ++j)
          if (used<K>(a, j)) done[i] = fmaf(w[j][i], g[K - 1 - j][i], done[i]);
      }
      const int td = t0 + k - (K - 1);
      if (k >= K - 1 && td < a.T) {
        if (a.state_out_bar && td < len) from_out(td, done);
        vstore<E, V>(xb + static_cast<int64_t>(td) * a.C, narrow<E, V>(done));
      }
#pragma unroll
      for (int j = 0; j + 1 < K; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) {
          win[j][i] = win[j + 1][i];
          g[j][i] = g[j + 1][i];
        }
    };
    fetch(0);
#pragma unroll 1
    for (int k0 = 0; k0 < RUN; k0 += kAhead) {
      Vec<E, V> cx[kAhead], cy[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) cx[u] = nx[u], cy[u] = ny[u];
      fetch(k0 + kAhead);
#pragma unroll
      for (int u = 0; u < kAhead; ++u) token(k0 + u, cx[u], cy[u], std::true_type());
    }
#pragma unroll
    for (int u = 0; u < K - 1; ++u) token(RUN + u, nx[u], ny[u], std::false_type());
    if (a.state_bar && t0 == 0) {
      // whole[k] for k < W - 1: taps j <= k of the first tokens
      E *sb = static_cast<E *>(a.state_bar) + b * (a.W - 1) * a.C + c;
      float gs[K][V] = {};
      for (int t = 0; t < a.W - 1; ++t) {
        float out[V] = {};
        if (t < len) {
          float v[V], f[V], yv[V];
#pragma unroll
          for (int i = 0; i < V; ++i) v[i] = bias[i];
          for (int j = 0; j < a.W; ++j) {
            widen(whole_at<E, V>(a, b, t + j - (a.W - 1), c), f);
#pragma unroll
            for (int i = 0; i < V; ++i)
              v[i] = fmaf(a.weight[static_cast<int64_t>(c + i) * a.W + j], f[i], v[i]);
          }
          widen(vload<E, V>(yb + t * a.yb_st), yv);
#pragma unroll
          for (int i = 0; i < V; ++i) {
            const float sg = sigmoid(v[i]);
            out[i] = a.silu ? yv[i] * sg * (1.0f + v[i] * (1.0f - sg)) : yv[i];
          }
        }
#pragma unroll
        for (int j = 0; j < K; ++j)
          if (j == t)
#pragma unroll
            for (int i = 0; i < V; ++i) gs[j][i] = out[i];
      }
      for (int k = 0; k < a.W - 1; ++k) {
        float acc[V] = {};
#pragma unroll
        for (int t = 0; t < K; ++t)
          if (t <= k)
#pragma unroll
            for (int i = 0; i < V; ++i)
              acc[i] = fmaf(a.weight[static_cast<int64_t>(c + i) * a.W + k - t], gs[t][i], acc[i]);
        if (a.state_out_bar && k - (a.W - 1) < len) from_out(k - (a.W - 1), acc);
        vstore<E, V>(sb + static_cast<int64_t>(k) * a.C, narrow<E, V>(acc));
      }
    }
  }
  // the four runs' sums, in run order
  auto reduce = [&](float (&v)[V], int row) {
    __syncthreads();
    if (run > 0)
#pragma unroll
      for (int i = 0; i < V; ++i) red[run - 1][lane * V + i] = v[i];
    __syncthreads();
    if (run == 0 && mine) {
      float f[V];
#pragma unroll
      for (int i = 0; i < V; ++i)
        f[i] = ((v[i] + red[0][lane * V + i]) + red[1][lane * V + i]) + red[2][lane * V + i];
      float *o = part + (bt * (K + 1) + row) * a.C + c;
#pragma unroll
      for (int i = 0; i < V; ++i) o[i] = f[i];
    }
  };
#pragma unroll
  for (int j = 0; j < K; ++j) reduce(dw[j], j);
  reduce(db, K);
}

// Sums over the tiles, one workgroup per 64 channels and row; its sixteen
// wavefronts take every sixteenth tile.
template <int K>
__global__ __launch_bounds__(1024) void conv_vjp_sum(selinv_conv_args a, int64_t tiles,
                                                     const float *part) {
  __shared__ float red[16][64];
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const int c = blockIdx.x * 64 + lane, row = blockIdx.y;
  float s = 0.0f;
  if (c < a.C) {
#pragma unroll 4
    for (int64_t t = wv; t < tiles; t += 16) s += part[(t * (K + 1) + row) * a.C + c];
  }
  red[wv][lane] = s;
  __syncthreads();
  if (wv || c >= a.C) return;
#pragma unroll
  for (int k = 1; k < 16; ++k) s += red[k][lane];
  const int jj = row - (K - a.W);
  if (row == K) {
    if (a.bias_bar) a.bias_bar[c] = s;
  } else if (jj >= 0) {
    a.weight_bar[static_cast<int64_t>(c) * a.W + jj] = s;
  }
}

inline int taps_for(int W) { return W >= 2 && W <= 4 ? W : 8; }

template <typename E, int V, int K>
hipError_t conv_run(const selinv_conv_args &a, hipStream_t s) {
  const int nc = a.C / V;
  // Sixteen tokens per thread where that leaves 1024 wavefronts or more, else
  // four: the shorter run reads its three past tokens 1.75 times over, which
  // only matters once HBM is busy (1531 tokens of 2304 channels in 16 bits, four
  // or sixteen: one row 10.1 or 11.2 us, three 22 or 17.5, six 36 or 24; eight or
  // twelve lose to sixteen by 3 and 1 us at six).
  const int64_t runs16 = a.T < 1 ? 1 : (a.T + 15) / 16, runs4 = a.T < 1 ? 1 : (a.T + 3) / 4;
  if (a.B * runs16 * nc >= 1024 * 64)
    hipLaunchKernelGGL((conv_kernel<E, V, K, 16>), dim3(blocks_for(a.B * runs16 * nc)), dim3(256),
                       0, s, a, nc, static_cast<int>(runs16));
  else
    hipLaunchKernelGGL((conv_kernel<E, V, K, 4>), dim3(blocks_for(a.B * runs4 * nc)), dim3(256), 0,
                       s, a, nc, static_cast<int>(runs4));
  return hipGetLastError();
}

template <typename E, int V, int K>
hipError_t conv_step_run(const selinv_conv_args &a, hipStream_t s) {
  const int nc = a.C / V;
  hipLaunchKernelGGL((conv_step_kernel<E, V, K>), dim3(blocks_for(a.B * nc)), dim3(256), 0, s, a,
                     nc);
  return hipGetLastError();
}

// workgroups' tiles of tokens along a row
inline int64_t vjp_tiles(int64_t B, int64_t T, int32_t C) {
  const int tile = 4 * run_for(B, T, C);
  return T < 1 ? 1 : (T + tile - 1) / tile;
}

template <typename E, int V, int K>
hipError_t conv_vjp_run(const selinv_conv_args &a, void *ws, hipStream_t s) {
  const int ctiles = (a.C / V + 63) / 64;
  const int64_t ttiles = vjp_tiles(a.B, a.T, a.C), tiles = a.B * ttiles;
  const dim3 grid(static_cast<unsigned>(tiles * ctiles));
  float *part = static_cast<float *>(ws);
  if (tiles && run_for(a.B, a.T, a.C) == 8)
    hipLaunchKernelGGL((conv_vjp_kernel<E, V, K, 8>), grid, dim3(256), 0, s, a, ctiles,
                       static_cast<int>(ttiles), part);
  else if (tiles)
    hipLaunchKernelGGL((conv_vjp_kernel<E, V, K, 32>), grid, dim3(256), 0, s, a, ctiles,
                       static_cast<int>(ttiles), part);
  hipLaunchKernelGGL(conv_vjp_sum<K>, dim3((a.C + 63) / 64, K + 1), dim3(1024), 0, s, a, tiles,
                     static_cast<const float *>(ws));
  return hipGetLastError();
}

template <typename E>
constexpr int kVec = 16 / sizeof(E);

}  // namespace

template <typename E>
hipError_t conv_launch(const selinv_conv_args &a, hipStream_t s) {
  if (a.B == 0) return hipSuccess;
  constexpr int V = kVec<E>;
  const bool vec = whole_vectors<E, V>(a.x, a.C, a.x_sb, a.x_st) &&
                   whole_vectors<E, V>(a.y, a.C) && whole_vectors<E, V>(a.state, a.C) &&
                   whole_vectors<E, V>(a.state_out, a.C);
  switch (taps_for(a.W)) {
    case 2: return vec ? conv_run<E, V, 2>(a, s) : conv_run<E, 1, 2>(a, s);
    case 3: return vec ? conv_run<E, V, 3>(a, s) : conv_run<E, 1, 3>(a, s);
    case 4: return vec ? conv_run<E, V, 4>(a, s) : conv_run<E, 1, 4>(a, s);
    default: return vec ? conv_run<E, V, 8>(a, s) : conv_run<E, 1, 8>(a, s);
  }
}

template <typename E>
hipError_t conv_step_launch(const selinv_conv_args &a, hipStream_t s) {
  if (a.B == 0) return hipSuccess;
  constexpr int V = kVec<E>;
  const bool vec = whole_vectors<E, V>(a.x, a.C, a.x_sb) && whole_vectors<E, V>(a.y, a.C) &&
                   whole_vectors<E, V>(a.state, a.C);
  switch (taps_for(a.W)) {
    case 2: return vec ? conv_step_run<E, V, 2>(a, s) : conv_step_run<E, 1, 2>(a, s);
    case 3: return vec ? conv_step_run<E, V, 3>(a, s) : conv_step_run<E, 1, 3>(a, s);
    case 4: return vec ? conv_step_run<E, V, 4>(a, s) : conv_step_run<E, 1, 4>(a, s);
    default: return vec ? conv_step_run<E, V, 8>(a, s) : conv_step_run<E, 1, 8>(a, s);
  }
}

size_t conv_vjp_workspace_bytes(int64_t B, int64_t T, int32_t C, int32_t W) {
  return static_cast<size_t>(B * vjp_tiles(B, T, C)) * (taps_for(W) + 1) * C * sizeof(float);
}

template <typename E>
hipError_t conv_vjp_launch(const selinv_conv_args &a, void *ws, hipStream_t s) {
  // Window, taps, gradients and sums take 4 (K + 1) V registers: V = 8 would
  // spill, and V = 4 at K = 8 leaves too few wavefronts (7 taps, 8 x 2048 tokens
  // of 2304 channels in float32: 120 us with two, 173 with four).
  constexpr int V = 4;
  const bool vec = whole_vectors<E, V>(a.x, a.C, a.x_sb, a.x_st) &&
                   whole_vectors<E, V>(a.y_bar, a.C, a.yb_sb, a.yb_st) &&
                   whole_vectors<E, V>(a.x_bar, a.C) && whole_vectors<E, V>(a.state, a.C) &&
                   whole_vectors<E, V>(a.state_out_bar, a.C) &&
                   whole_vectors<E, V>(a.state_bar, a.C);
  switch (taps_for(a.W)) {
    case 2: return vec ? conv_vjp_run<E, V, 2>(a, ws, s) : conv_vjp_run<E, 1, 2>(a, ws, s);
    case 3: return vec ? conv_vjp_run<E, V, 3>(a, ws, s) : conv_vjp_run<E, 1, 3>(a, ws, s);
    case 4: return vec ? conv_vjp_run<E, V, 4>(a, ws, s) : conv_vjp_run<E, 1, 4>(a, ws, s);
    default: return vec ? conv_vjp_run<E, 2, 8>(a, ws, s) : conv_vjp_run<E, 1, 8>(a, ws, s);
  }
}

#define SELINV_CONV_INSTANCE(E)                                             \
  template hipError_t conv_launch<E>(const selinv_conv_args &, hipStream_t);      \
  template hipError_t conv_step_launch<E>(const selinv_conv_args &, hipStream_t); \
  template hipError_t conv_vjp_launch<E>(const selinv_conv_args &, void *, hipStream_t);
SELINV_CONV_INSTANCE(float)
SELINV_CONV_INSTANCE(_Float16)
SELINV_CONV_INSTANCE(__bf16)

}  // namespace selinv
