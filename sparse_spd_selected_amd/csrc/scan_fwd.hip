// scan_fwd.hip -- the selective scan over a prompt (gfx950): the chunked form
// of scan_tile.h.  A workgroup holds one row, segment of the row and 64 rows of
// the state of HB heads of one group, four wavefronts a head; the states stay
// in registers from chunk to chunk (16 rows a wavefront).  The heads share the
// chunk's B, C and scores, which are most of what is moved into LDS; x is read
// and y written once.
//
// A row is cut into segments where there are too few heads to fill the GPU:
// then a first pass forms what each segment adds to the state (no y), a small
// kernel chains the segments, and the main pass starts each from its state.
//
// Measured for 8192 tokens of 32 heads of 64 x 128 in bfloat16, 32 segments: first
// pass 26 us, chain 14 (64 MB, 4.6 TB/s), main pass 59, each under the profiler; 88
// us a call where calls follow each other, 121 TFLOP/s of the recurrence's count.
// In the main pass a SIMD issues vector instructions 45 % of the time and matrix
// products 21 %, LDS is busy 29 %: the steps of a chunk wait for each other, and the
// decays, the splits into bfloat16 terms and the moves into LDS cost more than the
// products.  With two terms of states and scores instead of three it is 6 % shorter;
// with main chunks of 64 tokens and one workgroup a CU 13 % longer.
#include <type_traits>

#include "scan_tile.h"

namespace selinv {
namespace scan {
namespace {

// Wavefronts per SIMD: with 128 registers a bfloat16 workgroup shares its CU
// with another, which works while it waits; float32 fragments need more.
template <typename E>
constexpr int kSides = sizeof(typename Path<E>::L) == 2 ? 4 : 2;

// The sweeps', by the columns they hold: one head with all 128 has twice the tile
// under way, in registers that a fourth wavefront would need.
template <typename E, int NC, int HB>
constexpr int kSweepSides = kSides<E> == 4 && HB == 1 && NC == 128 ? 3 : kSides<E>;

// what a workgroup works on
struct Place {
  int pt, h, seg, gr, len;
  int64_t b;
  __device__ Place(const selinv_scan_args &a, int id, int npt, int segs, int HB) {
    pt = id % npt * kPT;
    id /= npt;
    const int hn = a.H / HB;
    h = id % hn * HB;
    id /= hn;
    seg = id % segs;
    b = id / segs;
    gr = h / (a.H / a.G);
    len = row_length(a.lengths, b, a.T);
  }
};

// ---------------------------------------------------------------- main pass
template <typename E, int NP, int HB>
struct FwdShared {
  using L = typename Path<E>::L;
  static constexpr int Q = Path<E>::kMain, QS = kStride<L, Q>, NS = kStride<L, NP>;
  alignas(16) L bt[NP * QS], br[Q * NS], cr[Q * NS];
  alignas(16) L xt[HB][kPT * QS];
  alignas(16) L m[HB][Path<E>::kTerms][Q * QS];
  Decay<Q> dec[HB][2];  // of this chunk and the next
};

template <typename E, int NP, bool V4, int HB>
__global__ __launch_bounds__(256 * HB, kSides<E>) void scan_kernel(selinv_scan_args a, int nseg, int cps,
                                                        int npt, const float *init, int total) {
  using S = FwdShared<E, NP, HB>;
  using L = typename S::L;
  constexpr int Q = S::Q, QS = S::QS, NS = S::NS, NT = NP / 16, MT = Path<E>::kTerms, TQ = Q / 16;
  constexpr int NTH = 256 * HB;
  __shared__ S sh;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  int r = lane & 15, g = lane >> 4;
  const int hd = wv >> 2, w4 = wv & 3, t256 = tid & 255;  // head of the workgroup, and place in it
  const Place at(a, xcd_order(blockIdx.x, total), npt, nseg, HB);
  const int pt = at.pt, h = at.h + hd, len = at.len;
  const int64_t b = at.b;
  const int chunks = (static_cast<int>(a.T) + Q - 1) / Q;
  const int c0 = at.seg * cps, c1 = min(chunks, c0 + cps);
  const int cols = min(kPT, a.P - pt);
  const E *x = static_cast<const E *>(a.x) + b * a.x_sb + h * a.x_sh + pt;
  const E *Bm = static_cast<const E *>(a.Bm) + b * a.b_sb + at.gr * a.b_sg;
  const E *Cm = static_cast<const E *>(a.Cm) + b * a.c_sb + at.gr * a.c_sg;
  const int64_t bh = b * a.H + h, pn = static_cast<int64_t>(a.P) * a.N;
  const int p = pt + 16 * w4 + r;  // this lane's row of the state

  const int64_t row = static_cast<int64_t>(a.H) * a.P;  // of y
  const unsigned yoff = 16 * w4 + 4 * g < cols
                            ? (r * static_cast<unsigned>(row) + 16 * w4 + 4 * g) * sizeof(E)
                            : kOutside;
  f32x4 st[NT];
#pragma unroll
  for (int k = 0; k < NT; ++k) st[k] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  if (at.seg) {
    const float *src = init + ((bh * nseg + at.seg - 1) * npt + pt / kPT) * kTileSize<NP>;
#pragma unroll
    for (int k = 0; k < NT; ++k) st[k] = *reinterpret_cast<const f32x4 *>(src + in_tile(k, w4, lane));
  } else if (a.state && p < a.P) {
    const float *src = a.state + bh * pn + static_cast<int64_t>(p) * a.N;
#pragma unroll
    for (int k = 0; k < NT; ++k) st[k] = load4<V4>(src, 16 * k + 4 * g, a.N);
  }
  // score tiles above the diagonal that a K = 32 step of the diagonal tiles
  // reaches: zero, once
  for (int i = tid; i < HB * MT * Q * QS; i += NTH) sh.m[0][0][i] = static_cast<L>(0.0f);

  Tile<E, Q, kPT, 256> tx;
  Tile<E, Q, NP, NTH> tb, tc;
  const int live = min(c1, (len + Q - 1) / Q);  // chunks from here on hold no tokens
  auto load = [&](int c) {
    const int64_t t0 = static_cast<int64_t>(c) * Q;
    const int rows = c < live ? min(Q, len - static_cast<int>(t0)) : 0;
    tx.template load<V4>(x + t0 * a.x_st, a.x_st, rows, cols, t256);
    tb.template load<V4>(Bm + t0 * a.b_st, a.b_st, rows, a.N, tid);
    tc.template load<V4>(Cm + t0 * a.c_st, a.c_st, rows, a.N, tid);
  };
  // the last HB wavefronts, which have the fewest score tiles, form the next
  // chunk's decays, of one head each
  const int fw = wv - 3 * HB, fh = fw > 0 ? fw : 0;
  const E *dt = static_cast<const E *>(a.dt) + b * a.dt_sb + at.h + fh;
  const float fA = a.A[at.h + fh], fbias = a.dt_bias ? a.dt_bias[at.h + fh] : 0.0f;
  auto load_dt = [&](int c) { return raw_step<E, Q>(a, dt, c * Q, lane); };
  auto form = [&](int c, E v) {
    decays<Q>(sh.dec[fh][c & 1],
              step_of<E>(a, static_cast<float>(v) + fbias, lane < Q && c * Q + lane < len), fA, lane);
  };
  E rdt = static_cast<E>(0.0f);
  if (c0 < live) {
    load(c0);
    if (fw >= 0) {
      form(c0, load_dt(c0));
      rdt = load_dt(c0 + 1);
    }
  }
  for (int c = c0; c < live; ++c) {
    const int t0 = c * Q;
    const Decay<Q> &dec = sh.dec[hd][c & 1];
    __syncthreads();
    tx.each(fresh(t256), [&](int t, int k, const Block<E> &v) { put_cols<L>(sh.xt[hd], QS, t, k, v); });
    tb.each(fresh(tid), [&](int t, int k, const Block<E> &v) {
      put_rows<L>(sh.br, NS, t, k, v);
      put_cols<L>(sh.bt, QS, t, k, v);
    });
    tc.each(fresh(tid), [&](int t, int k, const Block<E> &v) { put_rows<L>(sh.cr, NS, t, k, v); });
    __syncthreads();
    load(c + 1);
    if (fw >= 0) {
      if (c + 1 < live) form(c + 1, rdt);
      rdt = load_dt(c + 2);
    }

    __builtin_amdgcn_sched_barrier(0);
    r = fresh(r), g = fresh(g);
    // scores: tile (rows j, columns i) of B C^T, j <= i, decayed for one head
    constexpr int kTiles = TQ * (TQ + 1) / 2;
    for (int job = wv; job < kTiles * HB; job += 4 * HB) {
      const int u = job / kTiles, k = job % kTiles;
      int it = 0;
      while ((it + 1) * (it + 2) / 2 <= k) ++it;
      const int jt = k - it * (it + 1) / 2;
      f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
      const L *pb = sh.br + (16 * jt + r) * NS + 4 * g, *pc = sh.cr + (16 * it + r) * NS + 4 * g;
#pragma unroll
      for (int n = 0; n < NP; n += 32)
        mma(acc, frag<L>(pb + n), frag<L>(pb + n + 16), frag<L>(pc + n), frag<L>(pc + n + 16));
      const int i = 16 * it + r, j = 16 * jt + 4 * g;
      const Decay<Q> &du = sh.dec[u][c & 1];
      const f32x4 x2 = (du.hi[i] - *reinterpret_cast<const f32x4 *>(du.hi + j)) +
                       (du.lo[i] - *reinterpret_cast<const f32x4 *>(du.lo + j));
      acc *= *reinterpret_cast<const f32x4 *>(du.d + j);
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[e] *= __builtin_amdgcn_exp2f(x2[e]);
      if (it == jt) {
        // chosen, not multiplied away: above the diagonal the exponential may be
        // infinite.  On it, y_i += D x_i.
        const float D = a.D ? a.D[at.h + u] : 0.0f;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          acc[e] = 4 * g + e < r ? acc[e] : 4 * g + e == r ? acc[e] + D : 0.0f;
      }
      const Terms<L, MT> mt = split<MT>(acc, L());
#pragma unroll
      for (int q = 0; q < MT; ++q) *reinterpret_cast<Frag<L> *>(&sh.m[u][q][i * QS + j]) = mt.t[q];
    }
    __syncthreads();

    // y (rows p, columns i) = e^{s_i} S C^T + x^T M^T
    __builtin_amdgcn_sched_barrier(0);
    r = fresh(r), g = fresh(g);
    f32x4 ys[TQ];
#pragma unroll
    for (int it = 0; it < TQ; ++it) ys[it] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int k = 0; k < NT; k += 2) {
      const Terms<L, MT> s0 = split<MT>(st[k], L()), s1 = split<MT>(st[k + 1], L());
#pragma unroll
      for (int it = 0; it < TQ; ++it) {
        const L *pc = sh.cr + (16 * it + r) * NS + 16 * k + 4 * g;
        const Frag<L> f0 = frag<L>(pc), f1 = frag<L>(pc + 16);
#pragma unroll
        for (int q = MT - 1; q >= 0; --q) mma(ys[it], s0.t[q], s1.t[q], f0, f1);
      }
    }
#pragma unroll
    for (int it = 0; it < TQ; ++it) {
      const int i = 16 * it + r;
      f32x4 acc = ys[it];
      acc *= dec.from[i];
#pragma unroll
      for (int j = 0; j <= 16 * it; j += 32) {
        const L *px = sh.xt[hd] + (16 * w4 + r) * QS + j + 4 * g;
        const Frag<L> x0 = frag<L>(px), x1 = frag<L>(px + 16);
#pragma unroll
        for (int q = MT - 1; q >= 0; --q) {
          const L *pm = &sh.m[hd][q][i * QS + j + 4 * g];
          mma(acc, x0, x1, frag<L>(pm), frag<L>(pm + 16));
        }
      }
      E *y = static_cast<E *>(a.y) + ((b * a.T + t0 + 16 * it) * a.H + h) * a.P + pt;
      float f[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) f[e] = t0 + i < len ? acc[e] : 0.0f;
      if (V4) {  // rows past T are dropped
        buffer_store4(buffer_rows(y, row, min(16, static_cast<int>(a.T) - t0 - 16 * it)), yoff,
                      narrow<E, 4>(f));
      } else if (t0 + i < a.T) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (16 * w4 + 4 * g + e < cols) y[r * row + 16 * w4 + 4 * g + e] = static_cast<E>(f[e]);
      }
    }
    __builtin_amdgcn_sched_barrier(0);
    r = fresh(r), g = fresh(g);
    state_update<E, NP, Q, QS>(st, sh.xt[hd] + 16 * w4 * QS, sh.bt, dec.weight, dec.total, 1.0f, r, g);
  }
  // chunks without tokens: zeros
  for (int t = max(live, c0) * Q + t256 / 16; t < min(c1 * Q, static_cast<int>(a.T)); t += 16) {
    E *y = static_cast<E *>(a.y) + ((b * a.T + t) * a.H + h) * a.P + pt;
    for (int k = t256 % 16; k < cols; k += 16) y[k] = static_cast<E>(0.0f);
  }
  if (a.state_out && at.seg == nseg - 1 && p < a.P) {
    float *dst = a.state_out + bh * pn + static_cast<int64_t>(p) * a.N;
#pragma unroll
    for (int k = 0; k < NT; ++k) store4<V4>(dst, 16 * k + 4 * g, a.N, st[k]);
  }
}

// -------------------------------------------------------- states alone
// The same walk without y: forwards over (x, B) with weights e^{s_Q - s_t} d_t,
// or backwards over (y_bar, C) with weights e^{s_t}.  The bfloat16 products are
// added up with a rounding towards minus infinity; every other wavefront (16
// rows of the state) keeps the state negated, so that sums over the rows, which
// the gradient forms, see the bias cancel.
template <typename E, int NC, int HB>
struct SweepShared {
  using L = typename Path<E>::L;
  static constexpr int Q = Path<E>::Q, QS = kStride<L, Q>;
  // Two chunks are under way where there are registers for them, as a chunk's
  // products are over before a load comes back.  They have a place each, so that
  // a wavefront may fill one while others still read the other.
  static constexpr int kAhead = NC < 128 ? 2 : 1;
  alignas(16) L bt[kAhead][NC * QS], xt[kAhead][HB][kPT * QS];
  Decay<Q> dec[HB][8];  // of four chunks and the next four
};

template <typename E, int NP, int NC, bool V4, int HB>
__global__ __launch_bounds__(256 * HB, (kSweepSides<E, NC, HB>)) void sweep_kernel(selinv_scan_args a, Sweeps sws,
                                                                    int npt, int segs, int total) {
  using S = SweepShared<E, NC, HB>;
  using L = typename S::L;
  constexpr int Q = S::Q, QS = S::QS, NT = NC / 16, NTH = 256 * HB;
  __shared__ S sh;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  int r = lane & 15, g = lane >> 4;
  const int hd = wv >> 2, w4 = wv & 3, t256 = tid & 255;
  int id = xcd_order(blockIdx.x, total);
  const int n0 = id % (NP / NC) * NC;  // first of this workgroup's columns
  id /= NP / NC;
  total /= NP / NC;
  const bool rev = id >= total / sws.ways;
  const Sweep &sw = sws.way[rev];
  const Place at(a, rev ? id - total / 2 : id, npt, segs, HB);
  const int pt = at.pt, h = at.h + hd, len = at.len, seg = at.seg;
  const int64_t b = at.b;
  const int chunks = (static_cast<int>(a.T) + Q - 1) / Q;
  const int cols = min(kPT, a.P - pt);
  const E *x = rev ? static_cast<const E *>(a.y_bar) + b * a.yb_sb + h * a.yb_sh + pt
                   : static_cast<const E *>(a.x) + b * a.x_sb + h * a.x_sh + pt;
  const int64_t xst = rev ? a.yb_st : a.x_st;
  const E *Bm = rev ? static_cast<const E *>(a.Cm) + b * a.c_sb + at.gr * a.c_sg + n0
                    : static_cast<const E *>(a.Bm) + b * a.b_sb + at.gr * a.b_sg + n0;
  const int64_t bst = rev ? a.c_st : a.b_st;
  const E *dt = static_cast<const E *>(a.dt) + b * a.dt_sb + h;
  const float A = a.A[h], bias = a.dt_bias ? a.dt_bias[h] : 0.0f;
  const int64_t bh = b * a.H + h, pn = static_cast<int64_t>(a.P) * a.N;
  const int p = pt + 16 * w4 + r;
  const float sign = sizeof(L) == 2 && (w4 & 1) ? -1.0f : 1.0f;

  f32x4 st[NT];
#pragma unroll
  for (int k = 0; k < NT; ++k) st[k] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  if (seg && !sws.local) {
    const float *src = sw.local + ((bh * sws.nseg + seg - 1) * npt + pt / kPT) * kTileSize<NP>;
#pragma unroll
    for (int k = 0; k < NT; ++k)
      st[k] = sign * *reinterpret_cast<const f32x4 *>(src + in_tile(n0 / 16 + k, w4, lane));
  } else if (!seg && sw.first && p < a.P) {
    const float *src = sw.first + bh * pn + static_cast<int64_t>(p) * a.N;
#pragma unroll
    for (int k = 0; k < NT; ++k) st[k] = sign * load4<V4>(src, n0 + 16 * k + 4 * g, a.N);
  }
  constexpr int kAhead = S::kAhead;
  Tile<E, Q, kPT, 256> tx[kAhead];
  Tile<E, Q, NC, NTH> tb[kAhead];
  // steps k of this segment, in the sweep's order
  const int k0 = seg * sws.cps, k1 = min(chunks, k0 + sws.cps);
  auto chunk_at = [&](int k) { return rev ? chunks - 1 - k : k; };
  auto load = [&](int k, auto slot) {
    const int64_t t0 = static_cast<int64_t>(chunk_at(min(k, k1 - 1))) * Q;
    const int rows = k < k1 ? min(Q, len - static_cast<int>(t0)) : 0;
    tx[slot].template load<V4>(x + t0 * xst, xst, rows, cols, t256);
    tb[slot].template load<V4>(Bm + t0 * bst, bst, rows, a.N - n0, tid);
  };
  auto load_dt = [&](int k) { return raw_step<E, Q>(a, dt, chunk_at(k) * Q, lane); };
  auto form = [&](int k, E v) {
    if (k >= k1) return;
    decays<Q>(sh.dec[hd][k - k0 & 7],
              step_of<E>(a, static_cast<float>(v) + bias, lane < Q && chunk_at(k) * Q + lane < len),
              A, lane);
  };
  constexpr std::integral_constant<int, 0> kEven{};
  constexpr std::integral_constant<int, kAhead - 1> kOdd{};
  const int keep = sw.chunk && !sws.local;
  double sum = 0.0;
  E rdt = static_cast<E>(0.0f);
  if (k0 < k1) {
    load(k0, kEven);
    if (kAhead == 2) load(k0 + 1, kOdd);
    form(k0 + w4, load_dt(k0 + w4));
    rdt = load_dt(k0 + 4 + w4);
  }
  auto step = [&](int k, auto slot) {
    const Decay<Q> &dec = sh.dec[hd][k - k0 & 7];
    {  // no branch: the pass that keeps no states stores to a buffer of no bytes
      float *dst = sw.chunk + (((b * chunks + chunk_at(k)) * a.H + h) * npt + pt / kPT) * kTileSize<NP>;
      const __amdgpu_buffer_rsrc_t tile = buffer_rows(dst, kTileSize<NP>, keep);
#pragma unroll
      for (int n = 0; n < NT; ++n)
        buffer_store4(tile, in_tile(n0 / 16 + n, w4, lane) * 4u, Vec<float, 4>{sign * st[n]});
    }
    if (kAhead == 1) __syncthreads();
    L *xt = sh.xt[slot][hd], *bt = sh.bt[slot];
    tx[slot].each(fresh(t256), [&](int t, int n, const Block<E> &v) { put_cols<L>(xt, QS, t, n, v); });
    tb[slot].each(fresh(tid), [&](int t, int n, const Block<E> &v) { put_cols<L>(bt, QS, t, n, v); });
    __syncthreads();
    load(k + kAhead, slot);
    sum += dec.sum;
    __builtin_amdgcn_sched_barrier(0);
    r = fresh(r), g = fresh(g);
    state_update<E, NC, Q, QS>(st, xt + 16 * w4 * QS, bt, rev ? dec.from : dec.weight, dec.total,
                               sign, r, g);
    // the next four chunks' decays, one a wavefront
    if ((k - k0 & 3) == 0) {
      form(k + 4 + w4, rdt);
      rdt = load_dt(k + 8 + w4);
    }
  };
  for (int k = k0; k < k1; k += 2) {
    step(k, kEven);
    if (k + 1 < k1) step(k + 1, kOdd);
  }
  if (sws.local) {
    float *dst = sw.local + ((bh * sws.nseg + seg) * npt + pt / kPT) * kTileSize<NP>;
#pragma unroll
    for (int n = 0; n < NT; ++n)
      *reinterpret_cast<f32x4 *>(dst + in_tile(n0 / 16 + n, w4, lane)) = sign * st[n];
    if (pt == 0 && n0 == 0 && t256 == 0)
      sw.decay[bh * sws.nseg + seg] = __builtin_amdgcn_exp2f(static_cast<float>(sum));
  } else if (sw.last && seg == sws.nseg - 1 && p < a.P) {
    float *dst = sw.last + bh * pn + static_cast<int64_t>(p) * a.N;
#pragma unroll
    for (int n = 0; n < NT; ++n) store4<V4>(dst, n0 + 16 * n + 4 * g, a.N, sign * st[n]);
  }
}

// One thread per element of a head's state walks over the segments, eight of
// them under way.
__global__ __launch_bounds__(256) void chain_kernel(int64_t state, int tiles, int64_t heads,
                                                    Sweeps sws) {
  int64_t head = blockIdx.x / tiles;
  const Sweep &sw = sws.way[head >= heads];
  if (head >= heads) head -= heads;
  const int64_t e = static_cast<int64_t>(blockIdx.x % tiles) * 256 + threadIdx.x;
  if (e >= state) return;
  const int n = sws.nseg - 1;  // nothing begins after the last segment
  float *p = sw.local + head * sws.nseg * state + e;
  const float *d = sw.decay + head * sws.nseg;
  float v = p[0];
  for (int i0 = 1; i0 < n; i0 += 8) {
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = i0 + i < n ? p[(i0 + i) * state] : 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i0 + i < n) {
        v = fmaf(d[i0 + i], v, x[i]);
        p[(i0 + i) * state] = v;
      }
  }
}

// Two heads a workgroup where a group's heads pair up (one: 7 % more time for a
// prompt of 8192 tokens and 32 heads).
inline int heads_together(const selinv_scan_args &a) { return a.H / a.G % 2 ? 1 : 2; }

template <typename E, bool V4, int NP>
hipError_t run_main(const selinv_scan_args &a, int nseg, int cps, const float *init, hipStream_t s) {
  const int npt = (a.P + kPT - 1) / kPT, HB = heads_together(a);
  const int total = static_cast<int>(a.B * (a.H / HB) * nseg * npt);
  if (HB == 2)
    hipLaunchKernelGGL((scan_kernel<E, NP, V4, 2>), dim3(total), dim3(512), 0, s, a, nseg, cps, npt,
                       init, total);
  else
    hipLaunchKernelGGL((scan_kernel<E, NP, V4, 1>), dim3(total), dim3(256), 0, s, a, nseg, cps, npt,
                       init, total);
  return hipGetLastError();
}

template <typename E, bool V4, int NP, int NC, int HB>
void run_sweep(const selinv_scan_args &a, const Sweeps &sw, hipStream_t s) {
  const int npt = (a.P + kPT - 1) / kPT, segs = sw.local ? sw.nseg - 1 : sw.nseg;
  const int total = static_cast<int>(sw.ways * a.B * (a.H / HB) * segs * npt * (NP / NC));
  hipLaunchKernelGGL((sweep_kernel<E, NP, NC, V4, HB>), dim3(total), dim3(256 * HB), 0, s, a, sw, npt,
                     segs, total);
}

// 128 columns in one workgroup or two
template <typename E, bool V4, int NP, int HB>
void run_cut(const selinv_scan_args &a, const Sweeps &sw, hipStream_t s) {
  if (sw.cut) run_sweep<E, V4, NP, (NP < 128 ? NP : 64), HB>(a, sw, s);
  else run_sweep<E, V4, NP, NP, HB>(a, sw, s);
}

}  // namespace

// In bfloat16 1024 workgroups of one head (512 of two) run at once.  Below half of
// that the work is cut.  Sweeps without y first share the columns of a state of 128, which
// reads x twice but has no pass to join them (the gradient's two sweeps at
// 4 x 4096 x 32 heads: 150 us, against 215 in four segments; in four parts of 32
// columns 200).  Then rows are cut, into segments of four chunks at least (one or
// two gain nothing for a prompt of 8192 tokens, eight are slower).  The first pass
// costs half of the forward's main one, but all of a sweep's, where two segments
// gain nothing (gradient of 3 x 301 tokens in float32: 55 us in two, 47 in one).
// The other types' larger fragments let half as many run where N is 128; the same
// numbers hold for them, as halves lose more at one end than they gain at the other
// (float32, 64 x 128, this rule or half: 4 x 4096 tokens of 48 heads 562 us or 671,
// 1 x 8192 of 32 204 or 187).
int segments_for(int64_t B, int32_t H, int32_t P, int32_t N, int chunks, bool *cut) {
  int64_t wgs = B * H * ((P + kPT - 1) / kPT);
  if (cut) {
    *cut = wgs < 512 && N > 64;
    if (*cut) wgs *= 2;
  }
  if (wgs == 0 || wgs >= 512) return 1;
  int64_t n = 1024 / wgs;
  if (n > chunks / 4) n = chunks / 4;
  if (n < (cut ? 3 : 2)) return 1;
  const int cps = static_cast<int>((chunks + n - 1) / n);
  return (chunks + cps - 1) / cps;
}

template <typename E>
hipError_t sweep_states(const selinv_scan_args &a, const Sweeps &sw, hipStream_t s) {
#define SELINV_RUN(V4, NP)                                       \
  if (heads_together(a) == 2) run_cut<E, V4, NP, 2>(a, sw, s);   \
  else run_cut<E, V4, NP, 1>(a, sw, s)
  SELINV_SCAN_VARIANT(rows_of_four<E>(a, sw.ways == 2), a.N, SELINV_RUN);
#undef SELINV_RUN
  return hipGetLastError();
}

hipError_t chain_segments(int64_t heads, int64_t state, const Sweeps &sw, hipStream_t s) {
  const int tiles = static_cast<int>((state + 255) / 256);
  hipLaunchKernelGGL(chain_kernel, dim3(static_cast<unsigned>(sw.ways * heads * tiles)), dim3(256),
                     0, s, state, tiles, heads, sw);
  return hipGetLastError();
}

}  // namespace scan

using namespace scan;

size_t scan_workspace_bytes(int dtype_bytes, int64_t B, int64_t T, int32_t H, int32_t P,
                            int32_t N) {
  // both chunk lengths, as float16 shares its size with bfloat16
  size_t most = 0;
  for (int Q : {32, 64}) {
    const int nseg = segments_for(B, H, P, N, chunks_of(T, Q), nullptr);
    if (nseg < 2) continue;
    const size_t n = static_cast<size_t>(B * H) * nseg;
    const size_t bytes = n * state_size(P, N) * sizeof(float) + (n * sizeof(float) + 255) / 256 * 256;
    if (bytes > most) most = bytes;
  }
  return most;
}

template <typename E>
hipError_t scan_launch(const selinv_scan_args &a, void *ws, hipStream_t s) {
  if (a.B == 0) return hipSuccess;
  const int chunks = chunks_of(a.T, Path<E>::Q);
  const int nseg = segments_for(a.B, a.H, a.P, a.N, chunks, nullptr), cps = (chunks + nseg - 1) / nseg;
  const int64_t heads = a.B * a.H, state = state_size(a.P, a.N);
  float *local = static_cast<float *>(ws);
  hipError_t e = hipSuccess;
  if (nseg > 1) {
    Sweeps sw = {};
    sw.ways = 1, sw.nseg = nseg, sw.cps = cps, sw.local = true;
    sw.way[0].first = a.state, sw.way[0].local = local;
    sw.way[0].decay = local + heads * nseg * state;
    e = sweep_states<E>(a, sw, s);
    if (e == hipSuccess && nseg > 2) e = chain_segments(heads, state, sw, s);
    if (e != hipSuccess) return e;
  }
  constexpr int kRatio = Path<E>::Q / Path<E>::kMain;
#define SELINV_RUN(V4, NP) e = run_main<E, V4, NP>(a, nseg, cps * kRatio, local, s)
  SELINV_SCAN_VARIANT(rows_of_four<E>(a, false), a.N, SELINV_RUN);
#undef SELINV_RUN
  return e;
}

#define SELINV_SCAN_INSTANCE(E)                                                      \
  template hipError_t scan_launch<E>(const selinv_scan_args &, void *, hipStream_t); \
  template hipError_t scan::sweep_states<E>(const selinv_scan_args &, const scan::Sweeps &, hipStream_t);
SELINV_SCAN_INSTANCE(float)
SELINV_SCAN_INSTANCE(_Float16)
SELINV_SCAN_INSTANCE(__bf16)

}  // namespace selinv
