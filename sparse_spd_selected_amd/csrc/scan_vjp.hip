// scan_vjp.hip -- reverse mode of the selective scan (gfx950).
//
// With g_t the cotangent of S_t (g_t = y_bar_t C_t^T + a_{t+1} g_{t+1}) and
// l_t = a_t <g_t, S_{t-1}> that of log a_t,
//   x_bar = d g B + D y_bar,  B_bar = d g^T x,  C_bar = S^T y_bar,
//   d_bar = (g B) . x + A l,  A_bar = sum d l.
// Two sweeps leave the state S that meets each chunk and the cotangent R that
// leaves it (scan_fwd.hip); then every chunk is independent.  In a chunk, with
// W = y_bar x^T, G = C B^T and L_ij = e^{s_i - s_j} (i >= j),
//   x_bar_j = d_j (sum_i (G L)_ij y_bar_i + e^{s_Q - s_j} R B_j) + D y_bar_j
//   B_bar_j = sum_i (W L d)_ij C_i + d_j e^{s_Q - s_j} R^T x_j
//   C_bar_i = sum_j (W L d)_ij B_j + e^{s_i} S^T y_bar_i
//   l_t = sum_{i >= t > j} Z_ij + sum_{i >= t} r_i + sum_{j < t} c_j + e^{s_Q} <R, S>
// where Z = W G L d, r_i = e^{s_i} (S^T y_bar_i) . C_i and c_j = d_j e^{s_Q -
// s_j} (R B_j) . x_j.  l is summed in this direct form, all of it terms that
// belong to it, because the shorter one (a running sum of C_bar . C - x_bar . x
// over the whole row) subtracts what cancels and loses its digits with length.
//
// A workgroup of eight wavefronts holds one chunk of one row and group, and
// takes the group's heads in turn: B, C and G are formed once, and B_bar and
// C_bar are summed over the heads in registers, in a fixed order.
//
// Measured for 4 x 4096 tokens of 32 heads of 64 x 128 in 2 groups, bfloat16: 478
// us a call where calls follow each other; under the profiler the sweeps take 173
// us (537 MB of states written) and this kernel 366 (the states read back, 700 MB
// with the operands); a SIMD issues vector instructions 40 % of the time and matrix
// products 17 %, LDS is busy 32 %.  LDS holds one workgroup a CU, so what waits at
// its three barriers a head waits.  (W L d) is kept by columns alone, its rows come
// by transposing reads: the copy by rows would not fit beside three terms (146 KB
// of LDS as it is), and two terms, 5 % shorter, round one 16-bit gradient in five
// hundred the other way.
#include "scan_tile.h"

namespace selinv {
namespace scan {
namespace {

constexpr int kWaves = 8, kThreads = 64 * kWaves;

template <typename E, int NP>
struct VjpShared {
  using L = typename Path<E>::L;
  static constexpr int Q = Path<E>::Q, TQ = Q / 16, MT = Path<E>::kTerms;
  static constexpr int QS = kStride<L, Q>, NS = kStride<L, NP>, XS = kStride<L, kPT>;
  alignas(16) L br[Q * NS], bt[NP * QS], ct[NP * QS];
  struct Head {
    L xr[Q * XS], yr[Q * XS], yt[kPT * QS];
  };
  union {
    alignas(16) Head head;
    alignas(16) L cr[Q * NS];  // until the scores are formed
  };
  // (W L d) and (G L) by columns j
  alignas(16) L md[MT][Q * QS], me[MT][Q * QS];
  // what a head leaves for its sums over the chunk; two heads in turn
  struct Sums {
    float rs[TQ][Q]; // row sums of Z by column tile
    float cs[TQ][Q]; // column sums of Z / d by row tile
    float diag[Q];   // sum_{i >= t > j} Z_ij inside t's own tile
    float rpart[NP / 16][Q], cpart[4][Q], dpart[kWaves], lpart[kWaves];
  } sums[2];
  Decay<Q> dec[3];  // of a head, the one before and the next
  float v[3][Q];    // dt + dt_bias
};

// The matrix core's bfloat16 products round towards minus infinity when they
// are added up.  Where a long sum of such results has to keep float32 accuracy
// (A_bar was off by 2e-6 instead of 3e-7 at 4096 tokens) every other step of
// the inner index is formed with the opposite sign and subtracted, so that the
// two halves' bias cancels.
template <typename L>
struct Sum2 {
  static constexpr bool kFlip = sizeof(L) == 2;
  f32x4 plus = {0.0f, 0.0f, 0.0f, 0.0f}, minus = {0.0f, 0.0f, 0.0f, 0.0f};
  __device__ inline f32x4 &at(int step) { return kFlip && (step & 1) ? minus : plus; }
  __device__ inline f32x4 value() const { return kFlip ? plus - minus : plus; }
  // an operand's fragment or value as step `step` takes it
  template <typename F>
  static __device__ inline F sign(int step, F f) {
    return kFlip && (step & 1) ? negative(f) : f;
  }
};

// sums over the 16 lanes of a tile row, and over a wavefront
__device__ inline float sum16(float v) { return lane_sum<16>(v); }
__device__ inline float sum64(float v) { return lane_sum<64>(v); }

// sums over a row's lanes up to this one, and from this one on
__device__ inline float row_prefix(float v) {
  v += dpp_move<0x111>(v);
  v += dpp_move<0x112>(v);
  v += dpp_move<0x114>(v);
  return v + dpp_move<0x118>(v);
}
__device__ inline float row_suffix(float v) {
  v += dpp_move<0x101>(v);
  v += dpp_move<0x102>(v);
  v += dpp_move<0x104>(v);
  return v + dpp_move<0x108>(v);
}
__device__ inline float lane_at(float v, int lane) {
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), lane));
}

// v into a sum that starts with the head's first tile of P.  Every lane that
// holds v may write it: no branch, which would fence off the products around it.
__device__ inline void add_to(float &sum, bool first, float v) {
  const float old = sum;
  sum = first ? v : old + v;
}
// the sums of four rows over a tile's 16 columns, into sum[0 .. 3]
__device__ inline void add_rows(float *sum, bool first, f32x4 v, int r) {
  // a lane keeps the row of its last two bits and hands on the others
  const bool odd = r & 1, high = r & 2;
  float a = (odd ? v[1] : v[0]) + dpp_move<0xb1>(odd ? v[0] : v[1]);
  float b = (odd ? v[3] : v[2]) + dpp_move<0xb1>(odd ? v[2] : v[3]);
  a = (high ? b : a) + dpp_move<0x4e>(high ? a : b);
  a += dpp_move<0x124>(a);  // the quads of the row, by rotations of 4 and 8
  a += dpp_move<0x128>(a);
  add_to(sum[r & 3], first, a);
}

// From a state tile, four neighbours p of a lane's column n: rows 16 k + 4 g ..
// + 3 of the tile's column tile nt lie in the lanes that hold those rows, at
// place n % 4 of their four; `off`: the lane's own bytes of that.
__device__ inline unsigned down_offset(int r, int g) {
  return static_cast<unsigned>((4 * g + 16 * (r >> 2)) * 4 + (r & 3)) * 4;
}
__device__ inline f32x4 load_down(const float *tile, int nt, int k, unsigned off) {
  const float *s = reinterpret_cast<const float *>(
      reinterpret_cast<const char *>(tile + in_tile(nt, k, 0)) + off);
  return f32x4{s[0], s[4], s[8], s[12]};
}

// part: [B][chunks][H][3] sums for A, D, dt_bias; bc: [slices][2][B][T][G][N]
// partial B_bar, C_bar where the heads of a group are split (slices > 1)
template <typename E, int NP, bool V4>
__global__ __launch_bounds__(kThreads) void vjp_kernel(selinv_scan_args a, const float *states,
                                                       const float *costates, float *part,
                                                       float *bc, int slices, int total) {
  using S = VjpShared<E, NP>;
  using L = typename S::L;
  constexpr int Q = S::Q, TQ = S::TQ, MT = S::MT, QS = S::QS, NS = S::NS, XS = S::XS;
  constexpr int NT = NP / 16, KP = kPT / 16;
  constexpr int IS = kWaves / NT;                  // wavefronts that share a column tile n
  constexpr int TI = TQ > IS ? TQ / IS : 1;        // token tiles of each
  constexpr int TX = TQ / 2;                       // token tiles of x_bar per wavefront
  constexpr int NSC = TQ * (TQ + 1) / 2;           // score tiles on and below the diagonal
  constexpr int SC = 2, kScore = (NSC + SC - 1) / SC;  // two each, the others are free
  __shared__ S sh;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  int r = lane & 15, g = lane >> 4;
  int id = xcd_order(blockIdx.x, total);
  const int slice = id % slices;
  id /= slices;
  const int gr = id % a.G;
  id /= a.G;
  const int chunks = (static_cast<int>(a.T) + Q - 1) / Q;
  const int c = id % chunks;
  const int64_t b = id / chunks;
  const int per_group = a.H / a.G, per = (per_group + slices - 1) / slices;
  const int h0 = gr * per_group + slice * per, h1 = min(h0 + per, (gr + 1) * per_group);
  const int len = row_length(a.lengths, b, a.T), t0 = c * Q;
  const int rows = min(Q, len - t0), all = min(Q, static_cast<int>(a.T) - t0);
  const int64_t tok = b * a.T + t0;  // first token of the chunk, over the batch
  const int npt = (a.P + kPT - 1) / kPT;
  const int64_t row = static_cast<int64_t>(a.H) * a.P;  // of x_bar
  E *xbar = static_cast<E *>(a.x_bar), *dtbar = static_cast<E *>(a.dt_bar);

  f32x4 dB[TI], dC[TI];
#pragma unroll
  for (int i = 0; i < TI; ++i) dB[i] = dC[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  const int nt = wv % NT, i0 = IS == 1 ? 0 : wv / NT * TI;  // this wavefront's part of B_bar, C_bar
  int n = 16 * nt + r;
  const unsigned down = down_offset(r, g);

  if (rows <= 0) {  // no tokens: zeros
    for (int h = h0; h < h1; ++h) {
      for (int t = wv; t < all; t += kWaves)
        for (int p = lane; p < a.P; p += 64)
          xbar[((tok + t) * a.H + h) * a.P + p] = static_cast<E>(0.0f);
      if (tid < all) dtbar[(tok + tid) * a.H + h] = static_cast<E>(0.0f);
      if (tid < 3) part[((b * chunks + c) * a.H + h) * 3 + tid] = 0.0f;
    }
  } else {
    // ---- B, C and their scores
    for (int i = tid; i < 2 * MT * Q * QS; i += kThreads) sh.md[0][i] = static_cast<L>(0.0f);
    {
      Tile<E, Q, NP, kThreads> tb, tc;
      const E *Bm = static_cast<const E *>(a.Bm) + b * a.b_sb + gr * a.b_sg + t0 * a.b_st;
      const E *Cm = static_cast<const E *>(a.Cm) + b * a.c_sb + gr * a.c_sg + t0 * a.c_st;
      tb.template load<V4>(Bm, a.b_st, rows, a.N, tid);
      tc.template load<V4>(Cm, a.c_st, rows, a.N, tid);
      tb.each(tid, [&](int t, int k, const Block<E> &v) {
        put_rows<L>(sh.br, NS, t, k, v);
        put_cols<L>(sh.bt, QS, t, k, v);
      });
      tc.each(tid, [&](int t, int k, const Block<E> &v) {
        put_rows<L>(sh.cr, NS, t, k, v);
        put_cols<L>(sh.ct, QS, t, k, v);
      });
    }
    __syncthreads();
    f32x4 gt[SC];
    int sit[SC], sjt[SC];
#pragma unroll
    for (int q = 0; q < SC; ++q) {
      const int k = wv + q * kScore;
      int it = 0;
      while ((it + 1) * (it + 2) / 2 <= k) ++it;
      sit[q] = wv < kScore && k < NSC ? it : -1;
      sjt[q] = k - it * (it + 1) / 2;
      gt[q] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
      if (sit[q] < 0) continue;
      const L *pc = sh.cr + (16 * sit[q] + r) * NS + 4 * g;
      const L *pb = sh.br + (16 * sjt[q] + r) * NS + 4 * g;
      Sum2<L> acc;
#pragma unroll
      for (int m = 0; m < NP / 32; ++m)
        mma(acc.at(m), Sum2<L>::sign(m, frag<L>(pc + 32 * m)),
            Sum2<L>::sign(m, frag<L>(pc + 32 * m + 16)), frag<L>(pb + 32 * m),
            frag<L>(pb + 32 * m + 16));
      gt[q] = acc.value();
    }
    __syncthreads();  // the scores are formed: C's rows make room for a head

    // ---- the heads, by tiles of P: step q is tile q % npt of head h0 + q / npt
    const int steps = max(0, h1 - h0) * npt;
    const bool isx = wv < kWaves / 2;
    Tile<E, Q, kPT, kThreads / 2> tx;  // x in one half of the threads, y_bar in the other
    const int tx_tid = tid % (kThreads / 2);
    const E *src = isx ? static_cast<const E *>(a.x) + b * a.x_sb + t0 * a.x_st
                       : static_cast<const E *>(a.y_bar) + b * a.yb_sb + t0 * a.yb_st;
    const int64_t src_st = isx ? a.x_st : a.yb_st, src_sh = isx ? a.x_sh : a.yb_sh;
    f32x4 r2[NT];  // R, 16 rows p (for x_bar)
    auto fetch = [&](int q) {  // no branches, as in Tile::load; past the last step: nothing
      const bool any = q < steps;
      const int h = any ? h0 + q / npt : h0, pt = any ? q % npt * kPT : 0;
      tx.template load<V4>(src + h * src_sh + pt, src_st, any ? rows : 0, min(kPT, a.P - pt), tx_tid);
      const __amdgpu_buffer_rsrc_t Rh = buffer_rows(
          costates + (((b * chunks + c) * a.H + h) * npt + pt / kPT) * kTileSize<NP>, kTileSize<NP>,
          any);
#pragma unroll
      for (int k = 0; k < NT; ++k) r2[k] = buffer_load4<float>(Rh, in_tile(k, wv & 3, lane) * 4u);
    };
    // dt of a head; its decays, which the next to last wavefront forms while
    // others are at the scores of the head before
    auto load_dt = [&](int h) {
      return raw_step<E, Q>(a, static_cast<const E *>(a.dt) + b * a.dt_sb + min(h, h1 - 1), t0, lane);
    };
    auto form = [&](int h, E raw) {
      const float v = lane < rows ? static_cast<float>(raw) + (a.dt_bias ? a.dt_bias[h] : 0.0f) : 0.0f;
      decays<Q>(sh.dec[h % 3], step_of<E>(a, v, lane < rows), a.A[h], lane);
      if (lane < Q) sh.v[h % 3][lane] = v;
    };
    // a head's sums over the chunk: d_bar, A_bar, D_bar, dt_bias_bar
    auto finish = [&](int h) {
      const typename S::Sums &su = sh.sums[h & 1];
      const Decay<Q> &dec = sh.dec[h % 3];
      const int t = lane, tau = t >> 4;
      const bool in = lane < Q;
      const float d = in ? dec.d[t] : 0.0f;
      float rsum = 0.0f, csum = 0.0f, u = 0.0f, rect = in ? su.diag[t] : 0.0f;
#pragma unroll
      for (int k = 0; k < TQ; ++k) {
        const float rk = in && k < tau ? su.rs[k][t] : 0.0f;
        const float ck = in && k >= tau ? su.cs[k][t] : 0.0f;
        rsum += rk;
        u += ck;
        if (k > tau) csum += ck * d;
        // whole tiles (it, k) with it > tau > k
        const float whole = sum16(rk);
#pragma unroll
        for (int it = 1; it < TQ; ++it) {
          const float w = lane_at(whole, 16 * it);
          if (it > tau && k < tau) rect += w;
        }
      }
      float rr = 0.0f, cc = 0.0f;
      if (in) {
#pragma unroll
        for (int k = 0; k < NT; ++k) rr += su.rpart[k][t];
        cc = (su.cpart[0][t] + su.cpart[1][t]) + (su.cpart[2][t] + su.cpart[3][t]);
      }
      u += cc;
      cc *= d;
      // rows i >= t and columns j < t: within the tile, and over the chunk
      rect += row_suffix(rsum) + dpp_move<0x111>(row_prefix(csum));
      // rows of 16 lanes first, then the other rows' sums
      const float rs = row_suffix(rr), cp = row_prefix(cc);
      float later = rs, before = dpp_move<0x111>(cp);
#pragma unroll
      for (int k = 0; k < TQ; ++k) {
        const float rk = lane_at(rs, 16 * k), ck = lane_at(cp, 16 * k + 15);
        if (k > tau) later += rk;
        if (k < tau) before += ck;
      }
      float lam = 0.0f, dd = 0.0f;
#pragma unroll
      for (int k = 0; k < kWaves; ++k) lam += su.lpart[k], dd += su.dpart[k];
      const float l = rect + later + before + dec.total * lam;
      float dv = in && t < rows ? fmaf(a.A[h], l, u) : 0.0f;
      if (a.softplus && in) dv *= sigmoid(sh.v[h % 3][t]);
      if (t < all) dtbar[(tok + t) * a.H + h] = static_cast<E>(dv);
      const float sa = sum64(d * l), sb = sum64(dv);
      float *o = part + ((b * chunks + c) * a.H + h) * 3;
      if (lane == 0) o[0] = sa, o[1] = dd, o[2] = sb;
    };

    E rdt = static_cast<E>(0.0f);
    if (steps > 0) {
      fetch(0);
      if (wv == kWaves - 2) {
        form(h0, load_dt(h0));
        rdt = load_dt(h0 + 1);
      }
    }
    for (int q = 0; q < steps; ++q) {
      const int h = h0 + q / npt, pt = q % npt * kPT, cols = min(kPT, a.P - pt);
      const bool first = pt == 0;
      typename S::Sums &su = sh.sums[h & 1];
      const Decay<Q> &dec = sh.dec[h % 3];
      tx.each(tx_tid, [&](int t, int k, const Block<E> &w) {
        if (isx) {
          put_rows<L>(sh.head.xr, XS, t, k, w);
        } else {
          put_rows<L>(sh.head.yr, XS, t, k, w);
          put_cols<L>(sh.head.yt, QS, t, k, w);
        }
      });
      // S and R, the 16 columns n of this wavefront (for C_bar and B_bar)
      f32x4 sf[KP], rf[KP];
      {
        const int64_t o = (((b * chunks + c) * a.H + h) * npt + q % npt) * kTileSize<NP>;
#pragma unroll
        for (int k = 0; k < KP; ++k) {
          sf[k] = load_down(states + o, nt, k, down);
          rf[k] = load_down(costates + o, nt, k, down);
        }
      }
      __syncthreads();
      r = fresh(r), g = fresh(g);
      // ---- score tiles (rows i, columns j): W, Z and the weighted scores,
      // beside the sums of the head before
      if (wv == kWaves - 1 && first && q > 0) finish(h - 1);
      if (wv == kWaves - 2 && first && h + 1 < h1) {
        form(h + 1, rdt);
        rdt = load_dt(h + 2);
      }
#pragma unroll
      for (int k = 0; k < SC; ++k) {
        if (sit[k] < 0) continue;
        const int it = sit[k], jt = sjt[k], j = 16 * jt + r, ib = 16 * it + 4 * g;
        const L *py = sh.head.yr + (16 * it + r) * XS + 4 * g;
        const L *px = sh.head.xr + j * XS + 4 * g;
        Sum2<L> acc;
#pragma unroll
        for (int m = 0; m < kPT / 32; ++m)
          mma(acc.at(m), Sum2<L>::sign(m, frag<L>(py + 32 * m)),
              Sum2<L>::sign(m, frag<L>(py + 32 * m + 16)), frag<L>(px + 32 * m),
              frag<L>(px + 32 * m + 16));
        const f32x4 w = acc.value();
        const float dj = dec.d[j];
        const f32x4 x2 = (*reinterpret_cast<const f32x4 *>(dec.hi + ib) - dec.hi[j]) +
                         (*reinterpret_cast<const f32x4 *>(dec.lo + ib) - dec.lo[j]);
        f32x4 gl, wl;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float f = ib + e >= j ? __builtin_amdgcn_exp2f(x2[e]) : 0.0f;
          gl[e] = gt[k][e] * f;
          wl[e] = w[e] * f;
        }
        const f32x4 z = w * gl, zd = z * dj;
        const Terms<L, MT> tg = split<MT>(gl, L()), tw = split<MT>(wl * dj, L());
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          *reinterpret_cast<Frag<L> *>(&sh.md[m][j * QS + ib]) = tw.t[m];
          if (first) *reinterpret_cast<Frag<L> *>(&sh.me[m][j * QS + ib]) = tg.t[m];
        }
        f32x4 up;  // sums of the column from row ib + e down
        up[3] = zd[3], up[2] = zd[2] + up[3], up[1] = zd[1] + up[2], up[0] = zd[0] + up[1];
        if (it == jt) {
          // add what the groups of rows below hold, then sum the columns
          // before t
          const float s1 = __shfl_down(up[0], 16, 64), s2 = __shfl_down(up[0], 32, 64),
                      s3 = __shfl_down(up[0], 48, 64);
          const float below = (g < 3 ? s1 : 0.0f) + (g < 2 ? s2 : 0.0f) + (g < 1 ? s3 : 0.0f);
#pragma unroll
          for (int e = 0; e < 4; ++e) up[e] = j < ib + e ? up[e] + below : 0.0f;
          add_rows(su.diag + ib, first, up, r);
        } else {
          add_rows(su.rs[jt] + ib, first, zd, r);
        }
        float cs = (z[0] + z[1]) + (z[2] + z[3]);
        cs += __shfl_xor(cs, 16, 64);
        cs += __shfl_xor(cs, 32, 64);
        add_to(su.cs[it][j], first, cs);
      }
      __syncthreads();

      // ---- x_bar (rows p, columns j)
      r = fresh(r), g = fresh(g);
      {
        const int pw = wv & 3, pb = 16 * pw + 4 * g;
        const float D = a.D ? a.D[h] : 0.0f;
        // operands of a token tile are read from LDS ahead of the products before
        Frag<L> nb[NT], yt[Q / 16];
        auto fetch_b = [&](int k) {
          const L *q = sh.br + (16 * ((wv >> 2) * TX + k) + r) * NS + 4 * g;
#pragma unroll
          for (int m = 0; m < NT; ++m) nb[m] = frag<L>(q + 16 * m);
        };
        fetch_b(0);
#pragma unroll
        for (int i = 0; i < Q / 16; ++i)
          yt[i] = frag<L>(sh.head.yt + (16 * pw + r) * QS + 16 * i + 4 * g);
        __builtin_amdgcn_sched_barrier(0);
        Terms<L, MT> rr[NT];
#pragma unroll
        for (int k = 0; k < NT; ++k) rr[k] = split<MT>(Sum2<L>::sign(k / 2, r2[k]), L());
        float dd = 0.0f;
#pragma unroll
        for (int k = 0; k < TX; ++k) {
          const int jt = (wv >> 2) * TX + k, j = 16 * jt + r;
          Frag<L> bm[NT], me[MT][Q / 16];
#pragma unroll
          for (int m = 0; m < NT; ++m) bm[m] = nb[m];
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int i = 0; i < Q / 16; ++i) me[m][i] = frag<L>(&sh.me[m][j * QS + 16 * i + 4 * g]);
          const f32x4 xv = wide(frag<L>(sh.head.xr + j * XS + pb));
          const f32x4 yv = wide(frag<L>(sh.head.yr + j * XS + pb));
          __builtin_amdgcn_sched_barrier(0);
          Sum2<L> t2;
#pragma unroll
          for (int i = MT - 1; i >= 0; --i)
#pragma unroll
            for (int m = 0; m < NT; m += 2)
              mma(t2.at(m / 2), rr[m].t[i], rr[m + 1].t[i], bm[m], bm[m + 1]);
          f32x4 acc = t2.value() * dec.to[j];
          if (k + 1 < TX) fetch_b(k + 1);
          float cj = 0.0f;
#pragma unroll
          for (int e = 0; e < 4; ++e) cj = fmaf(acc[e], xv[e], cj), dd = fmaf(xv[e], yv[e], dd);
          cj += __shfl_xor(cj, 16, 64);
          cj += __shfl_xor(cj, 32, 64);
          add_to(su.cpart[pw][j], first, cj);
          // tiles of rows above the diagonal are zeros
#pragma unroll
          for (int m = MT - 1; m >= 0; --m)
#pragma unroll
            for (int i = 0; i < Q / 16; i += 2) mma(acc, yt[i], yt[i + 1], me[m][i], me[m][i + 1]);
          const float dj = dec.d[j];
          float f[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)  // past the row: chosen, as acc may not be finite
            f[e] = j < rows ? fmaf(dj, acc[e], D * yv[e]) : 0.0f;
          E *o = xbar + ((tok + 16 * jt) * a.H + h) * a.P + pt;
          if (V4) {  // rows past T are dropped
            buffer_store4(buffer_rows(o, row, all - 16 * jt),
                          pb < cols ? (r * static_cast<unsigned>(row) + pb) * sizeof(E) : kOutside,
                          narrow<E, 4>(f));
          } else if (j < all) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (pb + e < cols) o[r * row + pb + e] = static_cast<E>(f[e]);
          }
        }
        dd = sum64(dd);
        add_to(su.dpart[wv], first, dd);
      }
      __builtin_amdgcn_sched_barrier(0);
      fetch(q + 1);
      __builtin_amdgcn_sched_barrier(0);

      // ---- C_bar and B_bar: columns n of this wavefront
      {
        float s = 0.0f;
#pragma unroll
        for (int k = 0; k < KP; ++k)
#pragma unroll
          for (int e = 0; e < 4; ++e) s = fmaf(sf[k][e], rf[k][e], s);
        s = sum64(wv < NT ? s : 0.0f);  // each column tile once
        add_to(su.lpart[wv], first, s);
      }
      if (i0 < TQ) {
        r = fresh(r), g = fresh(g), n = 16 * nt + r;
        Terms<L, MT> ss[KP], rr[KP];
        // as above: the next token tile's operands are on their way
        Frag<L> nx[KP], ny[KP], bt[Q / 16], ct[Q / 16];
        auto fetch_xy = [&](int i) {
          const int o = (16 * (i0 + i) + r) * XS + 4 * g;
#pragma unroll
          for (int k = 0; k < KP; ++k)
            nx[k] = frag<L>(sh.head.xr + o + 16 * k), ny[k] = frag<L>(sh.head.yr + o + 16 * k);
        };
        fetch_xy(0);
#pragma unroll
        for (int j = 0; j < Q / 16; ++j) {
          bt[j] = frag<L>(sh.bt + n * QS + 16 * j + 4 * g);
          ct[j] = frag<L>(sh.ct + n * QS + 16 * j + 4 * g);
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int k = 0; k < KP; ++k)
          ss[k] = split<MT>(Sum2<L>::sign(k / 2, sf[k]), L()), rr[k] = split<MT>(rf[k], L());
#pragma unroll
        for (int i = 0; i < TI; ++i) {
          r = fresh(r), g = fresh(g);
          const int it = i0 + i, ib = 16 * it + 4 * g;
          Frag<L> x[KP], y[KP], mc[2][Q / 16], md[2][Q / 16];
#pragma unroll
          for (int k = 0; k < KP; ++k) x[k] = nx[k], y[k] = ny[k];
          // columns j of (W L d) up to the diagonal, and its rows from there on: a
          // term, and the next one while it is multiplied
          auto fetch_w = [&](int m) {
#pragma unroll
            for (int j = 0; j < Q / 16; ++j) {
              if (j / 2 * 2 <= it)
                mc[m & 1][j] = frag_down(&sh.md[m][16 * j * QS + 16 * it], QS, r, g);
              if (j / 2 * 2 + 2 > it)
                md[m & 1][j] = frag<L>(&sh.md[m][(16 * it + r) * QS + 16 * j + 4 * g]);
            }
          };
          fetch_w(MT - 1);
          if (i + 1 < TI) fetch_xy(i + 1);
          const f32x4 from = *reinterpret_cast<const f32x4 *>(dec.from + ib);
          const f32x4 weight = *reinterpret_cast<const f32x4 *>(dec.weight + ib);
          const f32x4 cw = wide(frag<L>(sh.ct + n * QS + ib));
          __builtin_amdgcn_sched_barrier(0);
          Sum2<L> s1;
          f32x4 t3 = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int m = MT - 1; m >= 0; --m)
#pragma unroll
            for (int k = 0; k < KP; k += 2) {
              mma(s1.at(k / 2), y[k], y[k + 1], ss[k].t[m], ss[k + 1].t[m]);
              mma(t3, x[k], x[k + 1], rr[k].t[m], rr[k + 1].t[m]);
            }
          const f32x4 t1 = s1.value() * from;
          add_rows(su.rpart[nt] + ib, first, t1 * cw, r);
          dC[i] += t1;
          dB[i] += t3 * weight;
#pragma unroll
          for (int m = MT - 1; m >= 0; --m) {
            if (m > 0) fetch_w(m - 1);
#pragma unroll
            for (int j = 0; j < Q / 16; j += 2) {
              if (j <= it) mma(dC[i], mc[m & 1][j], mc[m & 1][j + 1], bt[j], bt[j + 1]);
              if (j + 2 > it) mma(dB[i], md[m & 1][j], md[m & 1][j + 1], ct[j], ct[j + 1]);
            }
          }
        }
      }
      __syncthreads();  // done with the head's x, y_bar and scores
    }
    if (steps > 0 && wv == kWaves - 1) finish(h1 - 1);
  }

  // ---- B_bar, C_bar of the group (or this slice of its heads)
  if (i0 < TQ && n < a.N) {
#pragma unroll
    for (int i = 0; i < TI; ++i) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int t = 16 * (i0 + i) + 4 * g + e;
        if (t >= all) continue;
        const int64_t o = ((tok + t) * a.G + gr) * a.N + n;
        const float db = t < rows ? dB[i][e] : 0.0f, dc = t < rows ? dC[i][e] : 0.0f;
        if (slices == 1) {
          static_cast<E *>(a.B_bar)[o] = static_cast<E>(db);
          static_cast<E *>(a.C_bar)[o] = static_cast<E>(dc);
        } else {
          const int64_t size = a.B * a.T * a.G * a.N;
          bc[2 * slice * size + o] = db;
          bc[(2 * slice + 1) * size + o] = dc;
        }
      }
    }
  }
}

// What is left once the chunks are done, in one launch: A_bar, D_bar, dt_bias_bar
// of a head from its chunks, a workgroup each (the first H), and B_bar, C_bar from
// the slices, in their order.
template <typename E>
__global__ __launch_bounds__(256) void sums_kernel(selinv_scan_args a, const float *part,
                                                   int64_t chunks, const float *bc, int slices,
                                                   int64_t size) {
  __shared__ float red[4][3];
  const int h = blockIdx.x, lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  if (h >= a.H) {
    const int64_t i = static_cast<int64_t>(h - a.H) * 256 + threadIdx.x;
    if (i >= 2 * size) return;
    float s = 0.0f;
    for (int k = 0; k < slices; ++k) s += bc[2 * k * size + i];
    if (i < size) static_cast<E *>(a.B_bar)[i] = static_cast<E>(s);
    else static_cast<E *>(a.C_bar)[i - size] = static_cast<E>(s);
    return;
  }
  float s[3] = {};
  for (int64_t k = threadIdx.x; k < chunks; k += 256)
#pragma unroll
    for (int i = 0; i < 3; ++i) s[i] += part[(k * a.H + h) * 3 + i];
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    s[i] = sum64(s[i]);
    if (lane == 0) red[wv][i] = s[i];
  }
  __syncthreads();
  if (threadIdx.x) return;
#pragma unroll
  for (int i = 0; i < 3; ++i) s[i] = (red[0][i] + red[1][i]) + (red[2][i] + red[3][i]);
  a.A_bar[h] = s[0];
  if (a.D_bar) a.D_bar[h] = s[1];
  if (a.dt_bias_bar) a.dt_bias_bar[h] = s[2];
}

template <typename E, bool V4, int NP>
hipError_t run_vjp(const selinv_scan_args &a, const float *states, const float *costates,
                   float *part, float *bc, int slices, int chunks, hipStream_t s) {
  const int total = static_cast<int>(a.B * chunks * a.G * slices);
  hipLaunchKernelGGL((vjp_kernel<E, NP, V4>), dim3(total), dim3(kThreads), 0, s, a, states,
                     costates, part, bc, slices, total);
  return hipGetLastError();
}

// Workspace: the two kinds of states per chunk, the segments of a sweep, the
// heads' sums, and B_bar, C_bar of the slices.
struct Plan {
  int chunks, nseg, cps, slices;
  bool cut;
  int64_t heads, state;
  float *states, *costates, *local[2], *decay[2], *part, *bc;
  size_t bytes;
  Plan(int64_t B, int64_t T, int32_t H, int32_t P, int32_t G, int32_t N, int Q, void *ws) {
    chunks = chunks_of(T, Q);
    nseg = segments_for(2 * B, H, P, N, chunks, &cut);  // both sweeps at once
    cps = (chunks + nseg - 1) / nseg;
    heads = B * H, state = state_size(P, N);
    // One workgroup fits a CU.  The heads of a group are split, at the price
    // of writing and reading B_bar and C_bar once more per slice, until every
    // CU has one (32 heads of 64 x 128, bfloat16: 1 x 1024 tokens in one group
    // 300 us whole, 69 in sixteen; 4 x 4096 in two groups 466 whole, 506 in two).
    slices = 1;
    while (slices * 2 <= H / G && B * chunks * G * slices < 256) slices *= 2;
    size_t off = 0;
    auto take = [&](int64_t n) {
      float *p = ws ? reinterpret_cast<float *>(static_cast<char *>(ws) + off) : nullptr;
      off += (static_cast<size_t>(n) * sizeof(float) + 255) / 256 * 256;
      return p;
    };
    states = take(heads * chunks * state);
    costates = take(heads * chunks * state);
    for (int rev = 0; rev < 2; ++rev) {
      local[rev] = take(nseg > 1 ? heads * nseg * state : 0);
      decay[rev] = take(nseg > 1 ? heads * nseg : 0);
    }
    part = take(heads * chunks * 3);
    bc = take(slices > 1 ? 2 * slices * B * T * G * N : 0);
    bytes = off;
  }
};

}  // namespace
}  // namespace scan

using namespace scan;

template <typename E>
size_t scan_vjp_workspace_bytes(int64_t B, int64_t T, int32_t H, int32_t P, int32_t G, int32_t N) {
  return Plan(B, T, H, P, G, N, Path<E>::Q, nullptr).bytes;
}

template <typename E>
bool scan_vjp_fits(int64_t B, int64_t T, int32_t G) {
  // below 2^32 threads; there are slices only where there are less than 256 of these
  return B * chunks_of(T, Path<E>::Q) * G < (int64_t(1) << 32) / kThreads;
}

template <typename E>
hipError_t scan_vjp_launch(const selinv_scan_args &a, void *ws, hipStream_t s) {
  const Plan p(a.B, a.T, a.H, a.P, a.G, a.N, Path<E>::Q, ws);
  hipError_t e = hipSuccess;
  if (a.B > 0) {
    Sweeps sw = {};
    sw.ways = 2, sw.nseg = p.nseg, sw.cps = p.cps, sw.cut = p.cut;
    for (int rev = 0; rev < 2; ++rev) {
      Sweep &w = sw.way[rev];
      w.first = rev ? a.state_out_bar : a.state;
      w.chunk = a.T > 0 ? (rev ? p.costates : p.states) : nullptr;
      w.last = rev ? a.state_bar : nullptr;
      w.local = p.local[rev], w.decay = p.decay[rev];
    }
    if (p.nseg > 1) {
      sw.local = true;
      e = sweep_states<E>(a, sw, s);
      if (e == hipSuccess && p.nseg > 2) e = chain_segments(p.heads, p.state, sw, s);
      if (e != hipSuccess) return e;
      sw.local = false;
    }
    e = sweep_states<E>(a, sw, s);
  }
  if (e != hipSuccess) return e;
  if (a.B > 0 && a.T > 0) {
#define SELINV_RUN(V4, NP) \
  e = run_vjp<E, V4, NP>(a, p.states, p.costates, p.part, p.bc, p.slices, p.chunks, s)
    SELINV_SCAN_VARIANT(rows_of_four<E>(a, true), a.N, SELINV_RUN);
#undef SELINV_RUN
    if (e != hipSuccess) return e;
  }
  const bool any = a.B > 0 && a.T > 0;
  const int64_t size = any && p.slices > 1 ? a.B * a.T * a.G * a.N : 0;
  hipLaunchKernelGGL(sums_kernel<E>, dim3(a.H + blocks_for(2 * size)), dim3(256), 0, s, a, p.part,
                     any ? a.B * p.chunks : 0, p.bc, p.slices, size);
  return hipGetLastError();
}

#define SELINV_SCAN_VJP_INSTANCE(E) \
  template bool scan_vjp_fits<E>(int64_t, int64_t, int32_t); \
  template size_t scan_vjp_workspace_bytes<E>(int64_t, int64_t, int32_t, int32_t, int32_t, int32_t); \
  template hipError_t scan_vjp_launch<E>(const selinv_scan_args &, void *, hipStream_t);
SELINV_SCAN_VJP_INSTANCE(float)
SELINV_SCAN_VJP_INSTANCE(_Float16)
SELINV_SCAN_VJP_INSTANCE(__bf16)

}  // namespace selinv
