// scan_tile.h -- tiles of the chunked selective scan on the matrix cores.
//
// Inside a chunk of Q tokens, with s_t the sum of d A from the chunk's start
// through t (inclusive),
//   y_i = sum_{j <= i} e^{s_i - s_j} d_j (C_i . B_j) x_j + e^{s_i} S C_i
//   S'  = e^{s_Q} S + sum_t e^{s_Q - s_t} d_t x_t B_t^T
// so that a chunk is a handful of small matrix products.
//
// Fragments.  Every operand of a product is kept with its inner index K
// contiguous, and a lane (row r = lane % 16, group g = lane / 16) holds four
// neighbours K = 16 k + 4 g .. + 3 of its row.  That is also how a result tile
// leaves the matrix core (column r, rows 4 g .. + 3), so a result is the next
// product's operand without a move, for the state and for the chunk's scores
// alike.  Two such fragments make one K = 32 step.
//
// Types.  bfloat16 inputs go into v_mfma_f32_16x16x32_bf16 as they are; an
// operand that was computed in float32 is written as a sum of three bfloat16
// terms (8 bits each: they leave 2^-25 of it, two would leave 2^-17), one
// instruction per term.
// float32 and float16 inputs use v_mfma_f32_16x16x4_f32 on float32 fragments.
#pragma once

#include "seq.h"

namespace selinv {
namespace scan {

using namespace seq;

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kPT = 64;  // rows of the state (elements of x) per workgroup

// L: what the fragments hold; Q: tokens of a chunk; kMain: of the forward main
// pass's; kTerms: terms of an operand that was computed in float32 (two round one
// 16-bit output in a thousand another way than float32 does)
template <typename E>
struct Path {
  using L = float;
  static constexpr int Q = 32, kMain = 32, kTerms = 1;
};
template <>
struct Path<__bf16> {
  using L = __bf16;
  static constexpr int Q = 64, kMain = 32, kTerms = 3;
};

template <typename L>
struct FragOf;
template <>
struct FragOf<float> {
  using type = f32x4;
};
template <>
struct FragOf<__bf16> {
  using type = bf16x4;
};
template <typename L>
using Frag = typename FragOf<L>::type;

__device__ inline f32x4 wide(f32x4 v) { return v; }
__device__ inline f32x4 wide(bf16x4 v) {
  typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
  const u32x2 w = __builtin_bit_cast(u32x2, v);
  return f32x4{__uint_as_float(w[0] << 16), __uint_as_float(w[0] & 0xffff0000u),
               __uint_as_float(w[1] << 16), __uint_as_float(w[1] & 0xffff0000u)};
}

template <typename L>
__device__ inline Frag<L> frag(const L *p) {
  return *reinterpret_cast<const Frag<L> *>(p);
}

// four neighbours down column r of a 16 x 16 tile that lies by rows, rows 4 g ..
// + 3: the fragment of the transposed tile
__device__ inline bf16x4 frag_down(const __bf16 *tile, int stride, int r, int g) {
  // 16 lanes read four rows of 16 elements, four elements each, and the load hands
  // every lane its column
  const __bf16 *p = tile + (4 * g + (r >> 2)) * stride + 4 * (r & 3);
  return __builtin_amdgcn_ds_read_tr16_b64_v4bf16(
      (__attribute__((address_space(3))) bf16x4 *)const_cast<__bf16 *>(p));
}
__device__ inline f32x4 frag_down(const float *tile, int stride, int r, int g) {
  const float *p = tile + 4 * g * stride + r;
  return f32x4{p[0], p[stride], p[2 * stride], p[3 * stride]};
}

// acc += A B over K = 32: fragments k and k + 16 of either operand
__device__ inline void mma(f32x4 &acc, bf16x4 a0, bf16x4 a1, bf16x4 b0, bf16x4 b1) {
  const bf16x8 a = __builtin_shufflevector(a0, a1, 0, 1, 2, 3, 4, 5, 6, 7);
  const bf16x8 b = __builtin_shufflevector(b0, b1, 0, 1, 2, 3, 4, 5, 6, 7);
  acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, acc, 0, 0, 0);
}
__device__ inline void mma(f32x4 &acc, f32x4 a0, f32x4 a1, f32x4 b0, f32x4 b1) {
#pragma unroll
  for (int i = 0; i < 4; ++i) acc = __builtin_amdgcn_mfma_f32_16x16x4f32(a0[i], b0[i], acc, 0, 0, 0);
#pragma unroll
  for (int i = 0; i < 4; ++i) acc = __builtin_amdgcn_mfma_f32_16x16x4f32(a1[i], b1[i], acc, 0, 0, 0);
}

// a float32 fragment as a sum of N terms of L
template <typename L, int N>
struct Terms {
  Frag<L> t[N];
};
template <int N>
__device__ inline Terms<float, N> split(f32x4 v, float) {
  static_assert(N == 1, "float32 fragments are exact");
  return {{v}};
}
template <int N>
__device__ inline Terms<__bf16, N> split(f32x4 v, __bf16) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
  // (-1, 0) and (0, -1), from registers: as an inline constant -1.0 stands for
  // one word of either
  unsigned first, second;
  asm("s_mov_b32 %0, 0x0000bf80" : "=s"(first));
  asm("s_mov_b32 %0, 0xbf800000" : "=s"(second));
  Terms<__bf16, N> o;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    u32x2 w;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const f32x2 pair = {v[2 * k], v[2 * k + 1]};
      const bf16x2 t = __builtin_convertvector(pair, bf16x2);
      w[k] = __builtin_bit_cast(unsigned, t);
      if (i + 1 < N) {  // what is left, exactly: one product-sum each
        v[2 * k] = __builtin_amdgcn_fdot2_f32_bf16(t, __builtin_bit_cast(bf16x2, first), v[2 * k], false);
        v[2 * k + 1] = __builtin_amdgcn_fdot2_f32_bf16(t, __builtin_bit_cast(bf16x2, second), v[2 * k + 1], false);
      }
    }
    o.t[i] = __builtin_bit_cast(bf16x4, w);
  }
  return o;
}

// -v; of a bfloat16 fragment by its sign bits
__device__ inline f32x4 negative(f32x4 v) { return -v; }
__device__ inline bf16x4 negative(bf16x4 v) {
  return __builtin_bit_cast(bf16x4, __builtin_bit_cast(uint64_t, v) ^ 0x8000800080008000ull);
}

// ------------------------------------------------------------ global -> LDS
// Four tokens x four neighbouring channels, the unit that a thread moves: it
// can be put into LDS by rows (token-major) or transposed, four at a time
// either way.
template <typename E>
struct Block {
  Vec<E, 4> r[4];
};
template <typename L, typename E>
__device__ inline void put_rows(L *dst, int stride, int t, int c, const Block<E> &b) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const typename Vec<E, 4>::Reg v = b.r[i].e;
    *reinterpret_cast<Frag<L> *>(dst + (t + i) * stride + c) = __builtin_convertvector(v, Frag<L>);
  }
}
template <typename L, typename E>
__device__ inline void put_cols(L *dst, int stride, int t, int c, const Block<E> &b) {
  // whole vectors first: reading elements of the block in place would keep it
  // in memory
  const typename Vec<E, 4>::Reg v0 = b.r[0].e, v1 = b.r[1].e, v2 = b.r[2].e, v3 = b.r[3].e;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const typename Vec<E, 4>::Reg v = {v0[k], v1[k], v2[k], v3[k]};
    *reinterpret_cast<Frag<L> *>(dst + (c + k) * stride + t) = __builtin_convertvector(v, Frag<L>);
  }
}

// Rows of an array as a buffer: a lane's 32-bit offset is checked against the
// rows' bytes by the load itself, which gives zero (and a store that does
// nothing) past them.  The offset past all of them:
constexpr unsigned kOutside = 0xffffffffu;
// The size of a buffer is 32 bits wide, so it holds a chunk's rows and not what
// is left of an array: at most kBufferRows rows, kBufferStride elements apart at
// most.
constexpr int kBufferRows = 64, kBufferStride = 1 << 21;
constexpr int buffer_bytes(int64_t st, int rows, int size) {
  return rows <= 0 ? 0
                   : static_cast<int>((rows < kBufferRows ? rows : kBufferRows) * st * size);
}
static_assert(buffer_bytes(kBufferStride, 1 << 30, 4) == int64_t{kBufferRows} * kBufferStride * 4);
static_assert(buffer_bytes(65536, 32768, 2) == kBufferRows * 65536 * 2, "rows of 2^32 bytes");
template <typename E>
__device__ inline __amdgpu_buffer_rsrc_t buffer_rows(const E *p, int64_t st, int rows) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<E *>(p), 0,
                                           buffer_bytes(st, rows, sizeof(E)), 0x00027000);
}
template <typename E>
__device__ inline typename Vec<E, 4>::Reg buffer_load4(__amdgpu_buffer_rsrc_t rows, unsigned off) {
  if constexpr (sizeof(E) == 2) {
    return __builtin_bit_cast(typename Vec<E, 4>::Reg,
                              __builtin_amdgcn_raw_buffer_load_b64(rows, off, 0, 0));
  } else {
    return __builtin_bit_cast(typename Vec<E, 4>::Reg,
                              __builtin_amdgcn_raw_buffer_load_b128(rows, off, 0, 0));
  }
}
template <typename E>
__device__ inline void buffer_store4(__amdgpu_buffer_rsrc_t rows, unsigned off, const Vec<E, 4> &v) {
  if constexpr (sizeof(E) == 2) {
    typedef unsigned R __attribute__((ext_vector_type(2)));
    __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(R, v.e), rows, off, 0, 0);
  } else {
    typedef unsigned R __attribute__((ext_vector_type(4)));
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(R, v.e), rows, off, 0, 0);
  }
}

// The blocks of a Q x W tile that one of NT threads moves.  What lies past
// `rows` or `cols` reads as zero and is not touched.  With V4 a row is whole
// vectors, and the strides are at least `cols` and keep a tile's bytes in 31
// bits (rows_of_four): a block is then four loads at one offset, which stays the
// same from tile to tile, in the rows from the first, second, third and fourth.
//
// LDS serves 16 lanes of eight bytes at a time, so these are four by four blocks
// (a wavefront's eight by eight): by rows and by columns alike they then meet
// every bank once.
template <typename E, int Q, int W, int NT>
struct Tile {
  // four elements at any alignment of one: the hardware takes those in one load
  typedef E Loose __attribute__((ext_vector_type(4), aligned(sizeof(E)), may_alias));
  static constexpr int kBlocks = (Q / 4) * (W / 4), kPer = (kBlocks + NT - 1) / NT;
  Block<E> b[kPer];
  static __device__ inline int token(int i) {
    return (i >> 6) / (W / 32) * 32 + ((i >> 2 & 3) | (i >> 3 & 4)) * 4;
  }
  static __device__ inline int channel(int i) {
    return (i >> 6) % (W / 32) * 32 + ((i & 3) | (i >> 2 & 4)) * 4;
  }
  template <bool V4>
  __device__ inline void load(const E *p, int64_t st, int rows, int cols, int tid) {
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const int i = tid + k * NT;
      if (kBlocks % NT && i >= kBlocks) continue;  // whole wavefronts
      const int t = token(i), c = channel(i);
      if (V4) {
        const unsigned off =
            c < cols ? (static_cast<unsigned>(t) * static_cast<unsigned>(st) + c) * sizeof(E)
                     : kOutside;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          b[k].r[j].e = buffer_load4<E>(buffer_rows(p + j * st, st, rows - j), off);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          typename Vec<E, 4>::Reg v = static_cast<E>(0.0f);
          const E *q = p + (t + j) * st + c;
          if (t + j < rows) {
            if (c + 4 <= cols) {
              v = *reinterpret_cast<const Loose *>(q);
            } else {
#pragma unroll
              for (int n = 0; n < 4; ++n)
                if (c + n < cols) v[n] = q[n];
            }
          }
          b[k].r[j].e = v;
        }
      }
    }
  }
  template <typename F>
  __device__ inline void each(int tid, F &&f) const {
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const int i = tid + k * NT;
      if (kBlocks % NT == 0 || i < kBlocks) f(token(i), channel(i), b[k]);
    }
  }
};

// LDS row strides.  Fragments are read 16 rows at a time, eight bytes a lane and
// 16 lanes at once: four elements past a multiple of 32 put the rows' words
// (2 r odd mod 32) on distinct banks.
template <typename L, int W>
constexpr int kStride = W + 4;

// ------------------------------------------------------------------ decays
// Per token of a chunk, from its step d and the scan of d A (in float64: the
// differences of sums over a chunk keep float32 accuracy whatever they are
// taken between).  s = hi + lo in units of log2.
template <int Q>
struct Decay {
  alignas(16) float hi[Q], lo[Q];
  float d[Q];      // step
  float from[Q];   // e^{s_t}: from the chunk's start
  float to[Q];     // e^{s_Q - s_t}: to the chunk's end
  float weight[Q]; // d_t e^{s_Q - s_t}
  float total;     // e^{s_Q}
  double sum;      // s_Q, log2
};

// the step of token t of a row: 0 past its length
template <typename E>
__device__ inline float step_of(const selinv_scan_args &a, float v, bool in) {
  if (!in) return 0.0f;
  return a.softplus ? fmaxf(v, 0.0f) + log1pf(expf(-fabsf(v))) : v;
}

// dt of the chunk's tokens from t0, lane = token, as it comes: a conversion would
// wait for the load, and with it for every load before.  Past the row's length or
// the chunk: any of the array's values, which step_of drops.
template <typename E, int Q>
__device__ inline E raw_step(const selinv_scan_args &a, const E *dt, int t0, int lane) {
  return dt[max(0, min(t0 + min(lane, Q - 1), static_cast<int>(a.T) - 1)) * a.dt_st];
}

// s plus its value CTRL lanes away (zero from outside the row or a masked row)
template <int CTRL, int ROWS>
__device__ inline double plus_moved(double s) {
  const uint64_t u = __builtin_bit_cast(uint64_t, s);
  const int lo = __builtin_amdgcn_update_dpp(0, static_cast<int>(u), CTRL, ROWS, 0xf, true);
  const int hi = __builtin_amdgcn_update_dpp(0, static_cast<int>(u >> 32), CTRL, ROWS, 0xf, true);
  return s + __builtin_bit_cast(double, static_cast<uint64_t>(static_cast<unsigned>(hi)) << 32 |
                                            static_cast<unsigned>(lo));
}
// the sum over this lane and those before it
__device__ inline double scan64(double s) {
  s = plus_moved<0x111, 0xf>(s);  // lanes of a row of 16, by 1, 2, 4, 8
  s = plus_moved<0x112, 0xf>(s);
  s = plus_moved<0x114, 0xf>(s);
  s = plus_moved<0x118, 0xf>(s);
  s = plus_moved<0x142, 0xa>(s);  // the row before, into rows 1 and 3
  s = plus_moved<0x143, 0xc>(s);  // the first half, into rows 2 and 3
  return s;
}

// by one whole wavefront; lane = token
template <int Q>
__device__ inline void decays(Decay<Q> &o, float d, float A, int lane) {
  const double s =
      scan64(static_cast<double>(d) * static_cast<double>(A) * 1.4426950408889634);
  const uint64_t u = __builtin_bit_cast(uint64_t, s);
  const double all = __builtin_bit_cast(
      double, static_cast<uint64_t>(static_cast<unsigned>(
                  __builtin_amdgcn_readlane(static_cast<int>(u >> 32), Q - 1))) << 32 |
                  static_cast<unsigned>(__builtin_amdgcn_readlane(static_cast<int>(u), Q - 1)));
  if (lane < Q) {
    const float hi = static_cast<float>(s);
    o.hi[lane] = hi;
    o.lo[lane] = static_cast<float>(s - hi);
    o.d[lane] = d;
    o.from[lane] = __builtin_amdgcn_exp2f(hi);
    o.to[lane] = __builtin_amdgcn_exp2f(static_cast<float>(all - s));
    o.weight[lane] = d * o.to[lane];
    if (lane == 0) {
      o.total = __builtin_amdgcn_exp2f(static_cast<float>(all));
      o.sum = all;
    }
  }
}

// A lane index that the compiler takes for a new value: LDS addresses made from
// it are formed where they are used.  Otherwise some hundred of them are hoisted
// out of the loop over chunks or heads, and spilled.
__device__ inline int fresh(int v) {
  asm volatile("" : "+v"(v));
  return v;
}

// Blocks go round robin over the eight XCDs; give each XCD a contiguous range
// of work, so that the heads that read the same B and C share its L2.
__device__ inline int xcd_order(int blk, int total) {
  const int per = total / 8, rest = total % 8, x = blk % 8, k = blk / 8;
  return x * per + (x < rest ? x : rest) + k;
}

// ------------------------------------------------------------- state update
// St (P x N transposed: lane column = row of the state, rows = n) of one
// wavefront's 16 rows: St = total St + sum_t Bt[n][t] w_t Xt[p][t].  A
// wavefront that keeps -St passes sign = -1.
template <typename E, int NP, int Q, int QS>
__device__ inline void state_update(f32x4 (&st)[NP / 16], const typename Path<E>::L *xt,
                                    const typename Path<E>::L *bt, const float *w, float total,
                                    float sign, int r, int g) {
  using L = typename Path<E>::L;
  constexpr int N3 = Path<E>::kTerms;
#pragma unroll
  for (int k = 0; k < NP / 16; ++k) st[k] *= total;
  // Four column tiles at a time, the next four's fragments under way while
  // these are multiplied; the products of one term are independent.
  constexpr int KB = NP / 16 < 4 ? NP / 16 : 4;
#pragma unroll
  for (int t = 0; t < Q; t += 32) {
    Frag<L> b[KB][2];
    auto fetch = [&](int k0) {
#pragma unroll
      for (int k = 0; k < KB; ++k) {
        const L *q = bt + (16 * (k0 + k) + r) * QS + t + 4 * g;
        b[k][0] = frag<L>(q), b[k][1] = frag<L>(q + 16);
      }
    };
    __builtin_amdgcn_sched_barrier(0);  // one step's operands at a time
    Frag<L> x[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) x[h] = frag<L>(xt + r * QS + t + 16 * h + 4 * g);
    fetch(0);
    __builtin_amdgcn_sched_barrier(0);
    Terms<L, N3> xw[2];
#pragma unroll
    for (int h = 0; h < 2; ++h)
      xw[h] = split<N3>(
          wide(x[h]) * (*reinterpret_cast<const f32x4 *>(w + t + 16 * h + 4 * g) * sign), L());
#pragma unroll
    for (int k0 = 0; k0 < NP / 16; k0 += KB) {
      Frag<L> now[KB][2];
#pragma unroll
      for (int k = 0; k < KB; ++k) now[k][0] = b[k][0], now[k][1] = b[k][1];
      if (k0 + KB < NP / 16) fetch(k0 + KB);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int i = 0; i < N3; ++i)
#pragma unroll
        for (int k = 0; k < KB; ++k)
          mma(st[k0 + k], now[k][0], now[k][1], xw[0].t[i], xw[1].t[i]);
    }
  }
}

// four neighbours n.. of a state row in memory (cols = N)
template <bool V4>
__device__ inline f32x4 load4(const float *p, int n, int cols) {
  f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
  if (V4) {
    if (n < cols) v = *reinterpret_cast<const f32x4 *>(p + n);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (n + i < cols) v[i] = p[n + i];
  }
  return v;
}
template <bool V4>
__device__ inline void store4(float *p, int n, int cols, f32x4 v) {
  if (V4) {
    if (n < cols) *reinterpret_cast<f32x4 *>(p + n) = v;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (n + i < cols) p[n + i] = v[i];
  }
}

// ------------------------------------------------------- passes over states
// States in the workspace lie as the wavefronts hold them: tiles of kPT rows
// and NP columns (zeros where those are more than P and N), in each for
// [column tile][wavefront][lane] the lane's four neighbours.
template <int NP>
constexpr int kTileSize = kPT * NP;
__device__ inline int in_tile(int k, int wv, int lane) { return ((k * 4 + wv) * 64 + lane) * 4; }

// What a sweep over a row's chunks carries, forwards (S, from x and B) or
// backwards (its cotangent R, from y_bar and C).
struct Sweep {
  const float *first;  // [B][H][P][N] the state that the sweep begins with, or null
  float *chunk;        // [B][chunks][H] tiles: the state that meets each chunk, or null
  float *last;         // [B][H][P][N] the state that the sweep ends with, or null
  float *local;        // [B][H][nseg] tiles: what a segment makes of nothing (the first
                       // one of `first`); once chained, what segment i + 1 begins with
  float *decay;        // [B][H][nseg]: a segment's decay
};
struct Sweeps {
  Sweep way[2];   // forwards, backwards
  int ways;       // 1: forwards alone
  int nseg, cps;  // segments of a row, chunks of a segment
  bool local;     // the pass that forms what segments add, or the one that starts from it
  bool cut;       // a workgroup holds 64 columns of the state, not all 128
};

inline int chunks_of(int64_t T, int Q) { return T < 1 ? 1 : static_cast<int>((T + Q - 1) / Q); }

inline int padded_n(int N) { return N <= 32 ? 32 : N <= 64 ? 64 : 128; }
// floats of a head's state in the workspace
inline int64_t state_size(int P, int N) {
  return static_cast<int64_t>((P + kPT - 1) / kPT) * kPT * padded_n(N);
}

// Segments of a row's chunks so that a sweep has enough workgroups; `cut` is set
// where the columns of the state are shared out too (null: they are not).
int segments_for(int64_t B, int32_t H, int32_t P, int32_t N, int chunks, bool *cut);

// a segment's pass of the sweeps in `sw`, in one launch
template <typename E>
hipError_t sweep_states(const selinv_scan_args &a, const Sweeps &sw, hipStream_t s);
// the segments one after the other, in place: local[i] = decay[i] local[i - 1] + local[i]
hipError_t chain_segments(int64_t heads, int64_t state, const Sweeps &sw, hipStream_t s);

// rows of four elements everywhere: the N and P of the call and all strides;
// and token strides that Tile can take (rows that overlap go the other way)
template <typename E>
inline bool rows_of_four(const selinv_scan_args &a, bool vjp) {
  auto near = [](int64_t st, int cols) { return st >= cols && st < kBufferStride; };
  const bool ok = a.N % 4 == 0 && a.P % 4 == 0 && near(a.x_st, a.P) && near(a.b_st, a.N) &&
                  near(a.c_st, a.N) && (!vjp || near(a.yb_st, a.P)) &&
                  near(static_cast<int64_t>(a.H) * a.P, a.P) &&
                  whole_vectors<E, 4>(a.x, a.P, a.x_sb, a.x_st, a.x_sh) &&
                  whole_vectors<E, 4>(a.Bm, a.N, a.b_sb, a.b_st, a.b_sg) &&
                  whole_vectors<E, 4>(a.Cm, a.N, a.c_sb, a.c_st, a.c_sg) &&
                  whole_vectors<float, 4>(a.state, a.N);
  if (!vjp) return ok && whole_vectors<E, 4>(a.y, a.P) && whole_vectors<float, 4>(a.state_out, a.N);
  return ok && whole_vectors<E, 4>(a.y_bar, a.P, a.yb_sb, a.yb_st, a.yb_sh) &&
         whole_vectors<E, 4>(a.x_bar, a.P) && whole_vectors<E, 4>(a.B_bar, a.N) &&
         whole_vectors<E, 4>(a.C_bar, a.N) && whole_vectors<float, 4>(a.state_out_bar, a.N) &&
         whole_vectors<float, 4>(a.state_bar, a.N);
}

// f(V4, NP) with the compile-time variants: N padded to 32, 64 or 128
#define SELINV_SCAN_VARIANT(V4_, N_, CALL)                 \
  do {                                                     \
    if (V4_) {                                             \
      if ((N_) <= 32) { CALL(true, 32); }                  \
      else if ((N_) <= 64) { CALL(true, 64); }             \
      else { CALL(true, 128); }                            \
    } else {                                               \
      if ((N_) <= 32) { CALL(false, 32); }                 \
      else if ((N_) <= 64) { CALL(false, 64); }            \
      else { CALL(false, 128); }                           \
    }                                                      \
  } while (0)

}  // namespace scan
}  // namespace selinv
