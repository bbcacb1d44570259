// Differential attention over the incoming edges of each destination row,
// forward and backward (see egnn.h).
//
//   l[e,h,s] = scale <q[d,h,s], k[src,h,s]> + bias[e,h,s]      s = 0, 1
//   a[.,h,s] = softmax of l over the row's edges
//   w[e,h]   = m[e,h] (a[e,h,0] - lam[h] a[e,h,1]),  m = dropout factor
//   out[d,k,c] = sum_e w[e,h(c)] v[src,k,c]
//
// Two shapes of work carry both directions:
//   products   per edge and head, a dot of a destination's row with a source's row
//              (the logits, and <grad_out, v> in the backward), with the row's softmax
//              (or its backward) in the same block;
//   sums       per row and column, a weighted sum of gathered rows (out, and the
//              gradients of q, k and v; the latter two over edges grouped by source).
//
// Rows are handled by one block (products) or one wave per column slice
// (sums).  A row longer than the kernel's limit T is cut at the multiples of T
// of the edge array, so pieces need no list and no host knowledge of the row
// lengths: window x = [xT, (x+1)T) holds at most the end of one long row
// (piece 2x: the row that owns edge xT) and the start of another (piece 2x+1:
// the row that owns the window's last edge, if it starts inside the window).
// Pieces are joined by a later launch, in edge order.
#include <cmath>

#include "common.h"
#include "philox.h"
#include "timing.h"

using namespace egnn;

namespace {

constexpr int kWave = 64;
constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;
constexpr int kMaxHeads = 32;
constexpr int kMaxBlocks = 1 << 22;        // of a launch: its threads are counted in 32 bits
constexpr int64_t kMaxEdges = 1 << 28;     // at most 2^23 pieces of 64 edges or more
constexpr int kMaxRows = kMaxBlocks / 2;

// ------------------------------------------------------------------ helpers

template <typename T, int VW> struct Vec;
template <> struct Vec<float, 1> {
  __device__ static inline void ld(const float *p, float (&v)[1]) { v[0] = *p; }
  __device__ static inline void st(float *p, const float (&v)[1]) { *p = v[0]; }
};
template <> struct Vec<uint16_t, 1> {
  __device__ static inline void ld(const uint16_t *p, float (&v)[1]) { v[0] = bf16_to_f32(*p); }
  __device__ static inline void st(uint16_t *p, const float (&v)[1]) { *p = f32_to_bf16(v[0]); }
};
template <> struct Vec<float, 4> {
  __device__ static inline void ld(const float *p, float (&v)[4]) {
    const float4 a = *reinterpret_cast<const float4 *>(p);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  }
  __device__ static inline void st(float *p, const float (&v)[4]) {
    *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
  }
};
template <> struct Vec<float, 8> {
  __device__ static inline void ld(const float *p, float (&v)[8]) {
    const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
  __device__ static inline void st(float *p, const float (&v)[8]) {
    reinterpret_cast<float4 *>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4 *>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
  }
};
template <> struct Vec<uint16_t, 8> {
  __device__ static inline void ld(const uint16_t *p, float (&v)[8]) {
    const uint4 a = *reinterpret_cast<const uint4 *>(p);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
  __device__ static inline void st(uint16_t *p, const float (&v)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = static_cast<uint32_t>(f32_to_bf16(v[2 * i])) | (static_cast<uint32_t>(f32_to_bf16(v[2 * i + 1])) << 16);
    *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  }
};

__device__ inline int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// Edges [b, e) of row d; bounds from memory are held inside [0, E].
__device__ inline void row_bounds(const int *ptr, int d, int E, int *b, int *e) {
  const int lo = min(max(ptr[d], 0), E);
  *b = lo;
  *e = min(max(ptr[d + 1], lo), E);
}

struct Piece {
  int row, begin, end;  // row < 0: none
};

// The part of a long row (more than T edges) that piece p is, given the row
// that owns an edge position (see the file comment).
template <typename RowOf>
__device__ inline Piece find_piece(int p, int T, const int *ptr, int n_rows, int E, RowOf row_of) {
  Piece r{-1, 0, 0};
  const int total = min(max(ptr[n_rows], 0), E);
  const int64_t w0 = static_cast<int64_t>(p >> 1) * T;
  if (w0 >= total) return r;
  const int w1 = static_cast<int>(w0 + T < total ? w0 + T : total);
  const int row = row_of((p & 1) ? w1 - 1 : static_cast<int>(w0));
  if (row < 0 || row >= n_rows) return r;
  int b, e;
  row_bounds(ptr, row, E, &b, &e);
  if (e - b <= T || ((p & 1) && b <= w0)) return r;
  r.begin = max(b, static_cast<int>(w0));
  r.end = min(e, w1);
  if (r.begin < r.end) r.row = row;
  return r;
}

// Pieces of the long row [b, e): number and the id of the i-th
__device__ inline int piece_count(int b, int e, int T) { return (e - 1) / T - b / T + 1; }
__device__ inline int piece_id(int b, int T, int i) {
  const int x = b / T + i;
  return 2 * x + (i == 0 && b % T != 0 ? 1 : 0);
}

__device__ inline int row_by_search(const int *ptr, int n, int pos) {  // last d with ptr[d] <= pos
  int lo = 0, hi = n;                                                  // ptr[lo] <= pos assumed
  while (hi - lo > 1) {
    const int mid = lo + ((hi - lo) >> 1);
    if (ptr[mid] <= pos) lo = mid;
    else hi = mid;
  }
  return lo;
}

// Reduction over the threads that share column tid % Hp (Hp a power of two <=
// 64): butterflies inside a wave, then the waves in order.  Every thread gets
// the result.
template <typename F>
__device__ inline float column_reduce(float v, int Hp, float (*red)[kWave], F f) {
  for (int o = Hp; o < kWave; o <<= 1) v = f(v, __shfl_xor(v, o));
  const int lane = threadIdx.x & (kWave - 1);
  __syncthreads();
  red[threadIdx.x >> 6][lane] = v;
  __syncthreads();
  float r = red[0][lane];
#pragma unroll
  for (int i = 1; i < kWaves; ++i) r = f(r, red[i][lane]);
  return r;
}
struct MaxOp { __device__ float operator()(float a, float b) const { return fmaxf(a, b); } };
struct SumOp { __device__ float operator()(float a, float b) const { return a + b; } };

// softmax weight of a logit: (M, 1/S) of its row.  Rows with nothing left have
// M = 0, 1/S = 0; a masked logit is -inf and gives 0.
__device__ inline float weight_of(float l, float2 st) { return __expf(l - st.x) * st.y; }

__device__ inline float2 finish_stats(float M, float S) {
  if (M == -INFINITY) return make_float2(0.0f, 0.0f);
  return make_float2(M, 1.0f / S);
}

// Walk the (edge, head) decisions of edges [b, b + cnt) in aligned groups of
// eight, one generator call each; f(local index i * H + h, i, h, factor).
template <typename F>
__device__ inline void for_decisions(int b, int cnt, int H, const Drop &dr, F f) {
  const int64_t first = static_cast<int64_t>(b) * H;
  const int n = cnt * H;
  DropKey key{};
  if (dr.t != 0) key = drop_key(dr);
  for (int64_t g = (first >> 3) + threadIdx.x; g * 8 < first + n; g += kThreads) {
    uint4 w = make_uint4(0, 0, 0, 0);
    if (dr.t != 0) w = philox4x32(static_cast<uint64_t>(g), key);
    int at = static_cast<int>(g * 8 - first), u0 = 0;
    if (at < 0) {
      u0 = -at;
      at = 0;
    }
    int i = at / H, h = at - i * H;
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      if (u < u0 || at >= n) continue;
      f(at, i, h, dr.t == 0 || drop_draw(w, u) >= dr.t ? dr.factor : 0.0f);
      ++at;
      if (++h == H) {
        h = 0;
        ++i;
      }
    }
  }
}

// ------------------------------------------------------------------ products

// Lane layout of a dot product over `H` heads of `P` vectors each: lane =
// (edge sub, head, part), powers of two.
struct Team {
  int LTl, Hpl;  // log2 of parts per head, of padded heads
};

inline int log2_ceil(int n) {
  int l = 0;
  while ((1 << l) < n) ++l;
  return l;
}

inline Team make_team(int H, int vectors) {
  Team t;
  t.Hpl = log2_ceil(H);
  const int want = log2_ceil(vectors);
  t.LTl = want < 6 - t.Hpl ? want : 6 - t.Hpl;
  return t;
}

template <int CTRL> __device__ inline float dpp_move(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xF, 0xF, true));
}

// dot[u] summed over teams of 2^LTl lanes; every lane of a team gets the sum.
// Up to 16 lanes the steps are DPP moves inside a row of 16 (a quad's lanes
// hold the same value when the mirrors swap quads), no LDS permutes.
template <int U>
__device__ inline void team_sum(float (&dot)[U], int LTl) {
  if (LTl > 0)
#pragma unroll
    for (int u = 0; u < U; ++u) dot[u] += dpp_move<0xB1>(dot[u]);   // quad [1,0,3,2]
  if (LTl > 1)
#pragma unroll
    for (int u = 0; u < U; ++u) dot[u] += dpp_move<0x4E>(dot[u]);   // quad [2,3,0,1]
  if (LTl > 2)
#pragma unroll
    for (int u = 0; u < U; ++u) dot[u] += dpp_move<0x141>(dot[u]);  // mirror within 8
  if (LTl > 3)
#pragma unroll
    for (int u = 0; u < U; ++u) dot[u] += dpp_move<0x140>(dot[u]);  // mirror within 16
  if (LTl > 4)
#pragma unroll
    for (int u = 0; u < U; ++u) dot[u] += __shfl_xor(dot[u], 16);
  if (LTl > 5)
#pragma unroll
    for (int u = 0; u < U; ++u) dot[u] += __shfl_xor(dot[u], 32);
}

// lds[i * H + h] = sum over the head's vectors of A . B[scol[i]], i < cnt.
// A stays in registers, NIT vectors a lane.  Head h's vector j lies at
// (j / P) C + h Ch + (j % P) VW.  ONE: a wave takes one edge at a time (teams
// fill it), so the row's address is scalar work and the loads are scalar base
// plus the lane's fixed offset.
template <typename TA, typename TB, int VW, int NIT, bool ONE>
__device__ inline void edge_dots(const TA *arow, const TB *B, int64_t ldb, const int *scol, int cnt, int H, int C,
                                 int Ch, int nvec, Team tm, float *lds) {
  constexpr int U = NIT >= 8 ? 1 : 8 / NIT;  // eight loads in flight
  const int lane = threadIdx.x & (kWave - 1), wave = uniform(threadIdx.x >> 6);
  const int LT = 1 << tm.LTl;
  const int t = lane & (LT - 1), hh = (lane >> tm.LTl) & ((1 << tm.Hpl) - 1);
  const int es = ONE ? 0 : lane >> (tm.LTl + tm.Hpl);
  const int EPW = ONE ? 1 : kWave >> (tm.LTl + tm.Hpl);
  const int h = min(hh, H - 1);
  const int P = Ch / VW;
  for (int c0 = 0; c0 < nvec; c0 += LT * NIT) {
    float af[NIT][VW];
    int off[NIT];
    bool ok[NIT];
#pragma unroll
    for (int i = 0; i < NIT; ++i) {
      const int j = c0 + i * LT + t;
      ok[i] = j < nvec;
      const int jj = ok[i] ? j : nvec - 1;
      off[i] = (jj / P) * C + h * Ch + (jj % P) * VW;
      Vec<TA, VW>::ld(arow + off[i], af[i]);
    }
    for (int i0 = wave * EPW; i0 < cnt; i0 += kWaves * EPW * U) {
      float v[U][NIT][VW], dot[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = min(i0 + u * kWaves * EPW + es, cnt - 1);
        const int s = ONE ? uniform(scol[i]) : scol[i];
        const TB *row = B + static_cast<int64_t>(s) * ldb;
#pragma unroll
        for (int n = 0; n < NIT; ++n) Vec<TB, VW>::ld(row + off[n], v[u][n]);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        dot[u] = 0.0f;
#pragma unroll
        for (int n = 0; n < NIT; ++n) {
          float part = 0.0f;
#pragma unroll
          for (int x = 0; x < VW; ++x) part += af[n][x] * v[u][n][x];
          dot[u] += ok[n] ? part : 0.0f;
        }
      }
      team_sum<U>(dot, tm.LTl);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = i0 + u * kWaves * EPW + es;
        if (t == 0 && hh < H && i < cnt) lds[i * H + hh] = c0 == 0 ? dot[u] : lds[i * H + hh] + dot[u];
      }
    }
  }
}

// The source of each of cnt edges, sources outside the list as row 0 (their
// logits are masked).
__device__ inline void stage_sources(const int *src, int b, int cnt, int n_src, int *scol) {
  for (int i = threadIdx.x; i < cnt; i += kThreads) {
    const int s = src[b + i];
    scol[i] = static_cast<unsigned>(s) < static_cast<unsigned>(n_src) ? s : 0;
  }
}

struct LogitArgs {
  const int *row_ptr, *src;
  int n_dst, n_src, E, T, H, D;   // H heads of two maps
  int64_t ldq, ldk;
  float scale;
  const float *bias;              // [E][2H] or null
  const uint8_t *mask;            // [E] or null
  const float *lam;
  Drop drop;
  Team team;
  float *logits;                  // [E][2H] or null (no backward and no long row)
  float *w;                       // [E][H]
  float2 *stats;                  // [n_dst][2H]
  int *dst;                       // [E]
  float2 *piece_stats;            // [pieces][2H]
};

// One block per row (or piece): logits, softmax statistics and, for whole
// rows, the edge weights.
template <typename T, int VW, int NIT, bool ONE>
__global__ void __launch_bounds__(kThreads) logits_kernel(LogitArgs a, const T *__restrict__ q,
                                                          const T *__restrict__ k) {
  extern __shared__ float lg[];  // [T][2H], then the sources [T]
  int *scol = reinterpret_cast<int *>(lg + a.T * 2 * a.H);
  __shared__ float red[kWaves][kWave];
  __shared__ float2 fin[kWave];
  const int H2 = 2 * a.H;
  int d, b, e;
  const int p = static_cast<int>(blockIdx.x) - a.n_dst;
  if (p < 0) {
    d = blockIdx.x;
    row_bounds(a.row_ptr, d, a.E, &b, &e);
    if (e - b > a.T || e == b) return;
  } else {
    const Piece pc = find_piece(p, a.T, a.row_ptr, a.n_dst, a.E,
                                [&](int pos) { return row_by_search(a.row_ptr, a.n_dst, pos); });
    if (pc.row < 0) return;
    d = pc.row;
    b = pc.begin;
    e = pc.end;
  }
  const int cnt = e - b;
  for (int i = threadIdx.x; i < cnt; i += kThreads) a.dst[b + i] = d;
  stage_sources(a.src, b, cnt, a.n_src, scol);
  __syncthreads();
  edge_dots<T, T, VW, NIT, ONE>(q + static_cast<int64_t>(d) * a.ldq, k, a.ldk, scol, cnt, H2, H2 * a.D, a.D, a.D / VW,
                                a.team, lg);
  __syncthreads();
  const int Hp = 1 << a.team.Hpl;
  const int col = threadIdx.x & (Hp - 1), r0 = threadIdx.x >> a.team.Hpl, R = kThreads >> a.team.Hpl;
  float M = -INFINITY;
  if (col < H2) {
    for (int i = r0; i < cnt; i += R) {
      const int64_t o = static_cast<int64_t>(b + i) * H2 + col;
      float l = lg[i * H2 + col] * a.scale;
      if (a.bias) {
        const float bv = a.bias[o];
        l = bv == -INFINITY ? -INFINITY : l + bv;  // a bias of -inf masks, whatever the product is
      }
      if ((a.mask && a.mask[b + i] == 0) || static_cast<unsigned>(a.src[b + i]) >= static_cast<unsigned>(a.n_src))
        l = -INFINITY;
      lg[i * H2 + col] = l;
      if (a.logits) a.logits[o] = l;
      M = fmaxf(M, l);
    }
  }
  M = column_reduce(M, Hp, red, MaxOp());
  float S = 0.0f;
  if (col < H2 && M != -INFINITY)
    for (int i = r0; i < cnt; i += R) S += __expf(lg[i * H2 + col] - M);
  S = column_reduce(S, Hp, red, SumOp());
  if (p >= 0) {
    if (r0 == 0 && col < H2) a.piece_stats[static_cast<int64_t>(p) * H2 + col] = make_float2(M, S);
    return;
  }
  if (r0 == 0 && col < H2) {
    const float2 st = finish_stats(M, S);
    fin[col] = st;
    a.stats[static_cast<int64_t>(d) * H2 + col] = st;
  }
  __syncthreads();
  for_decisions(b, cnt, a.H, a.drop, [&](int at, int, int h, float m) {
    const float a0 = weight_of(lg[2 * at], fin[2 * h]), a1 = weight_of(lg[2 * at + 1], fin[2 * h + 1]);
    a.w[static_cast<int64_t>(b) * a.H + at] = m == 0.0f ? 0.0f : m * (a0 - a.lam[h] * a1);
  });
}

// Long rows: the pieces' statistics joined, then their edge weights.
__global__ void __launch_bounds__(kThreads) long_weights_kernel(LogitArgs a) {
  __shared__ float red[kWaves][kWave];
  __shared__ float2 fin[kWave];
  const Piece pc = find_piece(blockIdx.x, a.T, a.row_ptr, a.n_dst, a.E, [&](int pos) { return a.dst[pos]; });
  if (pc.row < 0) return;
  int b, e;
  row_bounds(a.row_ptr, pc.row, a.E, &b, &e);
  const int H2 = 2 * a.H, Hp = 1 << a.team.Hpl;
  const int col = threadIdx.x & (Hp - 1), r0 = threadIdx.x >> a.team.Hpl, R = kThreads >> a.team.Hpl;
  const int n = piece_count(b, e, a.T);
  float M = -INFINITY;
  if (col < H2)
    for (int i = r0; i < n; i += R)
      M = fmaxf(M, a.piece_stats[static_cast<int64_t>(piece_id(b, a.T, i)) * H2 + col].x);
  M = column_reduce(M, Hp, red, MaxOp());
  float S = 0.0f;
  if (col < H2 && M != -INFINITY)
    for (int i = r0; i < n; i += R) {
      const float2 st = a.piece_stats[static_cast<int64_t>(piece_id(b, a.T, i)) * H2 + col];
      if (st.x != -INFINITY) S += st.y * __expf(st.x - M);
    }
  S = column_reduce(S, Hp, red, SumOp());
  if (r0 == 0 && col < H2) {
    fin[col] = finish_stats(M, S);
    if (pc.begin == b) a.stats[static_cast<int64_t>(pc.row) * H2 + col] = fin[col];
  }
  __syncthreads();
  const float2 *lg = reinterpret_cast<const float2 *>(a.logits) + static_cast<int64_t>(pc.begin) * a.H;
  for_decisions(pc.begin, pc.end - pc.begin, a.H, a.drop, [&](int at, int, int h, float m) {
    const float2 l = lg[at];
    const float a0 = weight_of(l.x, fin[2 * h]), a1 = weight_of(l.y, fin[2 * h + 1]);
    a.w[static_cast<int64_t>(pc.begin) * a.H + at] = m == 0.0f ? 0.0f : m * (a0 - a.lam[h] * a1);
  });
}

struct GradArgs {
  const int *row_ptr, *src, *dst;
  int n_dst, n_src, E, T, H, C, K;
  int64_t ldv;
  const float *lam;
  Drop drop;
  Team team;
  const float2 *logits;  // [E][H] pairs of maps
  const float2 *stats;   // [n_dst][H] pairs of (M, 1/S): two entries a head
  float2 *dl;            // [E][H] pairs: gradient of the logits before the scale
  float *t1;             // [n_dst][H] sum_e a1 u
  float *u;              // [E][H] m <grad_out, v> of long rows, or null
  float2 *piece_t;       // [pieces][H] (sum a0 u, sum a1 u)
};

__device__ inline void logit_grads(const GradArgs &a, int64_t o, int h, float u, float2 t, const float4 *st) {
  const float2 l = a.logits[o];
  const float a0 = weight_of(l.x, make_float2(st[h].x, st[h].y)), a1 = weight_of(l.y, make_float2(st[h].z, st[h].w));
  // a weight of exactly 0 (masked) has no gradient, whatever the row of v holds
  a.dl[o] = make_float2(a0 == 0.0f ? 0.0f : a0 * (u - t.x), a1 == 0.0f ? 0.0f : -a.lam[h] * a1 * (u - t.y));
}

// One block per row (or piece): u = m <grad_out, v> per edge and head, then the
// softmax's backward for both maps.
template <typename T, int VW, int NIT, bool ONE>
__global__ void __launch_bounds__(kThreads) logit_grad_kernel(GradArgs a, const float *__restrict__ go,
                                                              const T *__restrict__ v) {
  extern __shared__ float us[];  // [T][H], then the sources [T]
  int *scol = reinterpret_cast<int *>(us + a.T * a.H);
  __shared__ float red[kWaves][kWave];
  __shared__ float4 st[kMaxHeads];
  __shared__ float2 tt[kMaxHeads];
  int d, b, e;
  const int p = static_cast<int>(blockIdx.x) - a.n_dst;
  if (p < 0) {
    d = blockIdx.x;
    row_bounds(a.row_ptr, d, a.E, &b, &e);
    if (e - b > a.T) return;
    if (e == b) {
      if (threadIdx.x < static_cast<unsigned>(a.H)) a.t1[static_cast<int64_t>(d) * a.H + threadIdx.x] = 0.0f;
      return;
    }
  } else {
    const Piece pc = find_piece(p, a.T, a.row_ptr, a.n_dst, a.E, [&](int pos) { return a.dst[pos]; });
    if (pc.row < 0) return;
    d = pc.row;
    b = pc.begin;
    e = pc.end;
  }
  const int cnt = e - b, H = a.H;
  if (threadIdx.x < static_cast<unsigned>(H))
    st[threadIdx.x] = reinterpret_cast<const float4 *>(a.stats)[static_cast<int64_t>(d) * H + threadIdx.x];
  const int Ch = a.C / H;
  stage_sources(a.src, b, cnt, a.n_src, scol);
  __syncthreads();
  edge_dots<float, T, VW, NIT, ONE>(go + static_cast<int64_t>(d) * a.K * a.C, v, a.ldv, scol, cnt, H, a.C, Ch,
                                    a.K * (Ch / VW), a.team, us);
  __syncthreads();
  for_decisions(b, cnt, H, a.drop, [&](int at, int, int, float m) {
    const float x = m == 0.0f ? 0.0f : m * us[at];
    us[at] = x;
    if (p >= 0) a.u[static_cast<int64_t>(b) * H + at] = x;
  });
  __syncthreads();
  const int Hp = 1 << a.team.Hpl;
  const int h = threadIdx.x & (Hp - 1), r0 = threadIdx.x >> a.team.Hpl, R = kThreads >> a.team.Hpl;
  float t0 = 0.0f, t1 = 0.0f;
  if (h < H)
    for (int i = r0; i < cnt; i += R) {
      const float2 l = a.logits[static_cast<int64_t>(b + i) * H + h];
      const float a0 = weight_of(l.x, make_float2(st[h].x, st[h].y));
      const float a1 = weight_of(l.y, make_float2(st[h].z, st[h].w));
      const float x = us[i * H + h];
      t0 += a0 == 0.0f ? 0.0f : a0 * x;
      t1 += a1 == 0.0f ? 0.0f : a1 * x;
    }
  t0 = column_reduce(t0, Hp, red, SumOp());
  t1 = column_reduce(t1, Hp, red, SumOp());
  if (p >= 0) {
    if (r0 == 0 && h < H) a.piece_t[static_cast<int64_t>(p) * H + h] = make_float2(t0, t1);
    return;
  }
  if (r0 == 0 && h < H) {
    tt[h] = make_float2(t0, t1);
    a.t1[static_cast<int64_t>(d) * H + h] = t1;
  }
  __syncthreads();
  if (h < H)
    for (int i = r0; i < cnt; i += R)
      logit_grads(a, static_cast<int64_t>(b + i) * H + h, h, us[i * H + h], tt[h], st);
}

// Long rows: the pieces' sums joined, then the logits' gradients.
__global__ void __launch_bounds__(kThreads) long_grad_kernel(GradArgs a) {
  __shared__ float red[kWaves][kWave];
  __shared__ float4 st[kMaxHeads];
  __shared__ float2 tt[kMaxHeads];
  const Piece pc = find_piece(blockIdx.x, a.T, a.row_ptr, a.n_dst, a.E, [&](int pos) { return a.dst[pos]; });
  if (pc.row < 0) return;
  int b, e;
  row_bounds(a.row_ptr, pc.row, a.E, &b, &e);
  const int H = a.H, Hp = 1 << a.team.Hpl;
  const int h = threadIdx.x & (Hp - 1), r0 = threadIdx.x >> a.team.Hpl, R = kThreads >> a.team.Hpl;
  if (threadIdx.x < static_cast<unsigned>(H))
    st[threadIdx.x] = reinterpret_cast<const float4 *>(a.stats)[static_cast<int64_t>(pc.row) * H + threadIdx.x];
  const int n = piece_count(b, e, a.T);
  float t0 = 0.0f, t1 = 0.0f;
  if (h < H)
    for (int i = r0; i < n; i += R) {
      const float2 t = a.piece_t[static_cast<int64_t>(piece_id(b, a.T, i)) * H + h];
      t0 += t.x;
      t1 += t.y;
    }
  t0 = column_reduce(t0, Hp, red, SumOp());
  t1 = column_reduce(t1, Hp, red, SumOp());
  if (r0 == 0 && h < H) {
    tt[h] = make_float2(t0, t1);
    if (pc.begin == b) a.t1[static_cast<int64_t>(pc.row) * H + h] = t1;
  }
  __syncthreads();
  if (h < H)
    for (int i = pc.begin + r0; i < pc.end; i += R) {
      const int64_t o = static_cast<int64_t>(i) * H + h;
      logit_grads(a, o, h, a.u[o], tt[h], st);
    }
}

// grad_lam[h] = -sum_d t1[d][h], one block a head, in a fixed order
__global__ void __launch_bounds__(kThreads) lam_grad_kernel(const float *__restrict__ t1, int n_dst, int H,
                                                            float *__restrict__ grad_lam) {
  __shared__ double red[kThreads];
  double s = 0.0;
  for (int d = threadIdx.x; d < n_dst; d += kThreads) s += t1[static_cast<int64_t>(d) * H + blockIdx.x];
  red[threadIdx.x] = s;
  __syncthreads();
  for (int o = kThreads / 2; o > 0; o >>= 1) {
    if (threadIdx.x < static_cast<unsigned>(o)) red[threadIdx.x] += red[threadIdx.x + o];
    __syncthreads();
  }
  if (threadIdx.x == 0) grad_lam[blockIdx.x] = static_cast<float>(-red[0]);
}

// ---------------------------------------------------------------------- sums

struct SumArgs {
  const int *ptr;       // [n_rows + 1]
  const int *perm;      // edge ids in row order (PERM)
  const int *col;       // [E] row of X of an edge
  const int *row_of;    // [E] row of an edge
  int n_rows, n_x, E, T;
  int64_t ldx;
  const float *w;       // [E][H]
  int H, C, Ch, width;  // out row = width elements; column c of width has head (c % C) / Ch
  int S, SV, Gl;        // slices, vectors a slice, log2 of lanes an edge
  int BE;               // edges staged at a time
  int unit0, units, blocks;  // first unit of the launch; rows + pieces; blocks a slice in the launch
  float scale;
  float *part;          // [pieces][width]
};

constexpr int kStage = 1024;  // weights a wave stages at a time (4 KB)

template <bool PERM> __device__ inline int owner(const SumArgs &a, int pos) {
  if constexpr (PERM) {
    const int ed = a.perm[pos];
    return static_cast<unsigned>(ed) < static_cast<unsigned>(a.E) ? a.row_of[ed] : -1;
  }
  return a.row_of[pos];
}

// The next BE edges of a list: lane i < BE holds edge j0 + i's row of X, and
// the lanes together the BE x H weights, four a register where H allows.
// Edges past the end and rows outside X have weight 0 and row 0.
template <bool PERM, bool W4> struct Batch {
  int x;
  float4 w4[kStage / 4 / kWave];
  float w1[kStage / kWave];

  __device__ inline void fetch(const SumArgs &a, int j0, int e, int lane) {
    int ed = -1;
    x = 0;
    if (lane < a.BE && j0 + lane < e) {
      ed = PERM ? a.perm[j0 + lane] : j0 + lane;
      if (PERM && static_cast<unsigned>(ed) >= static_cast<unsigned>(a.E)) ed = -1;
      if (ed >= 0) {
        const int s = a.col[ed];
        if (static_cast<unsigned>(s) < static_cast<unsigned>(a.n_x)) x = s;
        else ed = -1;
      }
    }
    const int per = W4 ? a.H / 4 : a.H, n = a.BE * per;
#pragma unroll
    for (int t = 0; t < (W4 ? kStage / 4 / kWave : kStage / kWave); ++t) {
      const int f = t * kWave + lane;
      if (t * kWave >= n) break;
      const int i = f / per;
      const int from = __shfl(ed, i & (kWave - 1));
      const bool live = f < n && from >= 0;
      const int64_t at = static_cast<int64_t>(from) * a.H + (f - i * per) * (W4 ? 4 : 1);
      if constexpr (W4)
        w4[t] = live ? *reinterpret_cast<const float4 *>(a.w + at) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      else
        w1[t] = live ? a.w[at] : 0.0f;
    }
  }

  __device__ inline void stage(const SumArgs &a, int lane, float *sw, int *sx) const {
    const int n = a.BE * (W4 ? a.H / 4 : a.H);
#pragma unroll
    for (int t = 0; t < (W4 ? kStage / 4 / kWave : kStage / kWave); ++t) {
      const int f = t * kWave + lane;
      if (t * kWave >= n) break;
      if (f < n) {
        if constexpr (W4) reinterpret_cast<float4 *>(sw)[f] = w4[t];
        else sw[f] = w1[t];
      }
    }
    sx[lane] = x;
  }
};

// acc += sum over edges [b, e) of w X.  ONE: the whole wave takes one edge at
// a time and its row's address is scalar work; else 64 >> Gl edges at once.
// SAFE skips weights of 0, so that what such a row of X holds stays out.
template <typename TX, int VW, bool PERM, bool ONE, bool W4, bool SAFE>
__device__ inline void gather_rows(const SumArgs &a, const TX *X, int b, int e, int c, int head, int lane, float *sw,
                                   int *sx, float (&acc)[VW]) {
  constexpr int U = 8;
  const int grp = ONE ? 0 : lane >> a.Gl, EPW = ONE ? 1 : kWave >> a.Gl;
  Batch<PERM, W4> next;
  next.fetch(a, b, e, lane);
  for (int j0 = b; j0 < e; j0 += a.BE) {
    next.stage(a, lane, sw, sx);
    const int x = next.x;
    wave_lds_order();
    if (j0 + a.BE < e) next.fetch(a, j0 + a.BE, e, lane);  // under way while this batch is summed
    const int n = min(a.BE, e - j0);
    for (int i0 = 0; i0 < n; i0 += EPW * U) {
      float v[U][VW], w[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        int i, s;
        if constexpr (ONE) {
          i = i0 + u;
          s = __builtin_amdgcn_readlane(x, i);
        } else {
          i = min(i0 + u * EPW + grp, a.BE - 1);
          s = sx[i];
        }
        w[u] = sw[i * a.H + head];
        if constexpr (!ONE)
          if (i0 + u * EPW + grp >= a.BE) w[u] = 0.0f;
        Vec<TX, VW>::ld(X + static_cast<int64_t>(s) * a.ldx + c, v[u]);
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int k = 0; k < VW; ++k) acc[k] = fmaf(w[u], SAFE && w[u] == 0.0f ? 0.0f : v[u][k], acc[k]);
    }
    wave_lds_order();
  }
}

// out[r] = scale sum over the row's edges of w[e][head] X[col[e]].  One wave
// per (row or piece, slice of columns).
template <typename TX, typename TO, int VW, bool PERM, bool ONE, bool W4>
__global__ void __launch_bounds__(kThreads) gather_sum_kernel(SumArgs a, const TX *__restrict__ X,
                                                              TO *__restrict__ out) {
  __shared__ __align__(16) float sw[kWaves][kStage];
  __shared__ int sx[kWaves][kWave];
  // consecutive blocks go to the eight XCDs in turn: a slice stays on one XCD
  // (S a multiple of 8), so each L2 holds an eighth of X
  int slice, rb;
  if (a.S <= 8) {
    slice = blockIdx.x % a.S;
    rb = blockIdx.x / a.S;
  } else {
    const int qd = blockIdx.x >> 3;
    slice = (qd / a.blocks) * 8 + (blockIdx.x & 7);
    rb = qd % a.blocks;
  }
  const int lane = threadIdx.x & (kWave - 1), wave = uniform(threadIdx.x >> 6);
  const int unit = a.unit0 + rb * kWaves + wave;
  if (unit >= a.units) return;
  int row, b, e;
  const int p = unit - a.n_rows;
  if (p < 0) {
    row = unit;
    row_bounds(a.ptr, row, a.E, &b, &e);
    if (e - b > a.T) return;
  } else {
    const Piece pc = find_piece(p, a.T, a.ptr, a.n_rows, a.E, [&](int pos) { return owner<PERM>(a, pos); });
    if (pc.row < 0) return;
    row = pc.row;
    b = pc.begin;
    e = pc.end;
  }
  b = uniform(b);
  e = uniform(e);
  const int gl = ONE ? lane : lane & ((1 << a.Gl) - 1);
  const int nv = a.width / VW;
  const int vj = slice * a.SV + gl;
  const bool on = gl < a.SV && vj < nv;
  const int c = (on ? vj : nv - 1) * VW;
  const int head = (c % a.C) / a.Ch;
  float acc[VW];
#pragma unroll
  for (int k = 0; k < VW; ++k) acc[k] = 0.0f;
  gather_rows<TX, VW, PERM, ONE, W4, false>(a, X, b, e, c, head, lane, sw[wave], sx[wave], acc);
  // A sum that is finite had no infinity or NaN in it, so its weights of 0
  // added 0.  One that is not is taken again with those edges left out.
  bool odd = false;
#pragma unroll
  for (int k = 0; k < VW; ++k) odd = odd || !(fabsf(acc[k]) < INFINITY);
  if (__any(odd)) {
#pragma unroll
    for (int k = 0; k < VW; ++k) acc[k] = 0.0f;
    gather_rows<TX, VW, PERM, ONE, W4, true>(a, X, b, e, c, head, lane, sw[wave], sx[wave], acc);
  }
  if constexpr (!ONE)
    for (int o = 1 << a.Gl; o < kWave; o <<= 1)
#pragma unroll
      for (int k = 0; k < VW; ++k) acc[k] += __shfl_xor(acc[k], o);
  if (!on || (!ONE && (lane >> a.Gl) != 0)) return;
  if (p >= 0) {
    Vec<float, VW>::st(a.part + static_cast<int64_t>(p) * a.width + c, acc);
    return;
  }
#pragma unroll
  for (int k = 0; k < VW; ++k) acc[k] *= a.scale;
  Vec<TO, VW>::st(out + static_cast<int64_t>(row) * a.width + c, acc);
}

// Long rows: the pieces' sums, added in edge order.  One block per window and
// 256 columns; it acts for the long row that starts in its window, if any.
template <typename TO, bool PERM>
__global__ void __launch_bounds__(kThreads) long_sum_kernel(SumArgs a, TO *__restrict__ out) {
  const int total = min(max(a.ptr[a.n_rows], 0), a.E);
  const int64_t w0 = static_cast<int64_t>(blockIdx.x) * a.T;
  if (w0 >= total) return;
  const int row = owner<PERM>(a, static_cast<int>(min(w0 + a.T, static_cast<int64_t>(total)) - 1));
  if (row < 0 || row >= a.n_rows) return;
  int b, e;
  row_bounds(a.ptr, row, a.E, &b, &e);
  if (e - b <= a.T || b < w0) return;
  const int c = blockIdx.y * kThreads + threadIdx.x;
  if (c >= a.width) return;
  const int n = piece_count(b, e, a.T);
  float s = 0.0f;
  for (int i = 0; i < n; ++i) s += a.part[static_cast<int64_t>(piece_id(b, a.T, i)) * a.width + c];
  Store<TO>::st(out + static_cast<int64_t>(row) * a.width + c, s * a.scale);
}

// ---------------------------------------------------------------------- host

struct Shape {
  int lmax, K, C, H, D, storage;
  int64_t ldq, ldk, ldv;
  int n_dst, n_src, E;
  float scale;
  int t;         // dropout threshold
  int T;         // edges of a row one block of the products holds
  int64_t pieces;
};

egnn_status make_shape_of(const egnn_attn_desc *d, const egnn_graph *g, Shape *s) {
  clear_error();
  EGNN_REQUIRE(d, "attention description is null");
  EGNN_REQUIRE(d->lmax >= 0 && d->lmax <= 8, "lmax (%d) must lie in 0..8", d->lmax);
  EGNN_REQUIRE(d->n_heads >= 1 && d->n_heads <= kMaxHeads, "n_heads (%d) must lie in 1..%d", d->n_heads, kMaxHeads);
  EGNN_REQUIRE(d->C >= 1 && d->C <= 1024 && d->C % d->n_heads == 0,
               "C (%d) must be a multiple of n_heads (%d) in 1..1024", d->C, d->n_heads);
  EGNN_REQUIRE(d->head_dim >= 1 && d->head_dim <= 256, "head_dim (%d) must lie in 1..256", d->head_dim);
  EGNN_REQUIRE(d->storage == EGNN_F32 || d->storage == EGNN_BF16, "unknown storage type (%d)", d->storage);
  EGNN_REQUIRE(std::isfinite(d->scale), "scale must be finite");
  s->t = drop_threshold(d->drop_p);
  EGNN_REQUIRE(s->t >= 0, "dropout probability %g must lie in [0, 1) after rounding to 1/65536", d->drop_p);
  s->lmax = d->lmax;
  s->K = (d->lmax + 1) * (d->lmax + 1);
  s->C = d->C;
  s->H = d->n_heads;
  s->D = d->head_dim;
  s->storage = d->storage;
  s->scale = static_cast<float>(d->scale);
  const int64_t qk = 2LL * s->H * s->D, vals = static_cast<int64_t>(s->K) * s->C;
  s->ldq = d->q_stride ? d->q_stride : qk;
  s->ldk = d->k_stride ? d->k_stride : qk;
  s->ldv = d->v_stride ? d->v_stride : vals;
  EGNN_REQUIRE(s->ldq >= qk && s->ldk >= qk, "q and k row strides must be 0 or at least 2 n_heads head_dim");
  EGNN_REQUIRE(s->ldv >= vals, "v row stride must be 0 or at least (lmax+1)^2 C");
  EGNN_REQUIRE(g, "graph is null");
  EGNN_REQUIRE(g->n_dst >= 0 && g->n_src >= 0, "negative row counts");
  EGNN_REQUIRE(g->n_edges >= 0, "negative edge count");
  if (g->n_edges > kMaxEdges || g->n_dst > kMaxRows || g->n_src > kMaxRows) {
    set_error("at most %lld edges, %d rows and %d sources", static_cast<long long>(kMaxEdges), kMaxRows, kMaxRows);
    return EGNN_E_UNSUPPORTED;
  }
  EGNN_REQUIRE(g->n_edges == 0 || (g->n_dst > 0 && g->n_src > 0), "edges need rows and sources");
  s->n_dst = g->n_dst;
  s->n_src = g->n_src;
  s->E = static_cast<int>(g->n_edges);
  const int fit = 4096 / (2 * s->H);  // 16 KB of logits
  s->T = fit < 64 ? 64 : fit > 512 ? 512 : fit;
  s->pieces = s->E > s->T ? 2 * ((static_cast<int64_t>(s->E) + s->T - 1) / s->T) : 0;
  return EGNN_OK;
}

struct SumPlan {
  int nv, S, SV, Gl, T;
  int64_t pieces;
};

// Slices and piece length of a weighted sum with rows of `nv` vectors.
SumPlan sum_plan(int n_rows, int E, int nv) {
  SumPlan p;
  p.nv = nv;
  p.S = nv <= kWave ? 1 : 8 * ((nv + 8 * kWave - 1) / (8 * kWave));
  p.SV = (nv + p.S - 1) / p.S;
  p.Gl = log2_ceil(p.SV);
  p.T = static_cast<int64_t>(n_rows) * p.S >= 4096 ? 2048 : 128;
  p.pieces = E > p.T ? 2 * ((static_cast<int64_t>(E) + p.T - 1) / p.T) : 0;
  return p;
}

size_t align256(size_t n) { return (n + 255) & ~size_t(255); }

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// Vector width: 16-byte vectors that lie in one head and one row; else single
// elements (any width, stride and alignment).
template <typename T> int vec_width(int Ch, int64_t ld, const void *p) {
  constexpr int V = 16 / sizeof(T);
  return Ch % V == 0 && ld % V == 0 && aligned16(p) ? V : 1;
}

struct Saved {
  float *logits, *w;
  float2 *stats;
  int *dst;
};

size_t saved_bytes_of(const Shape &s) {
  const size_t E = s.E, H = s.H;
  return align256(E * 2 * H * 4) + align256(E * H * 4) + align256(static_cast<size_t>(s.n_dst) * 2 * H * 8) +
         align256(E * 4);
}

Saved carve_saved(const Shape &s, char *p) {
  const size_t E = s.E, H = s.H;
  Saved v;
  v.logits = reinterpret_cast<float *>(p);
  p += align256(E * 2 * H * 4);
  v.w = reinterpret_cast<float *>(p);
  p += align256(E * H * 4);
  v.stats = reinterpret_cast<float2 *>(p);
  p += align256(static_cast<size_t>(s.n_dst) * 2 * H * 8);
  v.dst = reinterpret_cast<int *>(p);
  return v;
}

// Pieces of a sum's partial rows: the most any vector width may ask for.
size_t sum_part_bytes(int n_rows, int E, int width) {
  size_t most = 0;
  for (int vw : {1, 4, 8}) {
    const SumPlan p = sum_plan(n_rows, E, (width + vw - 1) / vw);
    const size_t n = align256(static_cast<size_t>(p.pieces) * width * 4);
    if (n > most) most = n;
  }
  return most;
}

size_t ws_fwd_of(const Shape &s, bool train) {
  return (train ? 0 : saved_bytes_of(s)) + align256(static_cast<size_t>(s.pieces) * 2 * s.H * 8) +
         sum_part_bytes(s.n_dst, s.E, s.K * s.C);
}

size_t ws_bwd_of(const Shape &s) {
  const size_t E = s.E, H = s.H;
  size_t part = sum_part_bytes(s.n_dst, s.E, 2 * s.H * s.D);
  for (int width : {2 * s.H * s.D, s.K * s.C}) {
    const size_t n = sum_part_bytes(s.n_src, s.E, width);
    if (n > part) part = n;
  }
  return align256(E * 2 * H * 4) + align256(static_cast<size_t>(s.n_dst) * H * 4) +
         (s.pieces ? align256(E * H * 4) + align256(static_cast<size_t>(s.pieces) * H * 8) : 0) + part;
}

template <typename TX, typename TO, bool PERM>
void launch_sum(unsigned grid, bool vec, bool one, bool w4, hipStream_t st, const SumArgs &a, const TX *X, TO *out) {
  constexpr int V = 16 / sizeof(TX);
  if (vec && one && w4) gather_sum_kernel<TX, TO, V, PERM, true, true><<<grid, kThreads, 0, st>>>(a, X, out);
  else if (vec && one) gather_sum_kernel<TX, TO, V, PERM, true, false><<<grid, kThreads, 0, st>>>(a, X, out);
  else if (vec && w4) gather_sum_kernel<TX, TO, V, PERM, false, true><<<grid, kThreads, 0, st>>>(a, X, out);
  else if (vec) gather_sum_kernel<TX, TO, V, PERM, false, false><<<grid, kThreads, 0, st>>>(a, X, out);
  else if (one) gather_sum_kernel<TX, TO, 1, PERM, true, false><<<grid, kThreads, 0, st>>>(a, X, out);
  else gather_sum_kernel<TX, TO, 1, PERM, false, false><<<grid, kThreads, 0, st>>>(a, X, out);
}

template <typename TX, typename TO, bool PERM>
egnn_status run_sum(SumArgs a, const TX *X, TO *out, const char *name, hipStream_t st) {
  if (a.n_rows == 0) return EGNN_OK;
  const int vw = vec_width<TX>(a.Ch, a.ldx, X) > 1 && aligned16(out) ? 16 / sizeof(TX) : 1;
  const SumPlan p = sum_plan(a.n_rows, a.E, a.width / vw);
  a.S = p.S;
  a.SV = p.SV;
  a.Gl = p.Gl;
  a.T = p.T;
  a.units = static_cast<int>(a.n_rows + p.pieces);
  a.BE = a.H <= kStage / kWave ? kWave : kStage / kMaxHeads / 2;
  const int most = kMaxBlocks / a.S;  // blocks a slice in one launch
  for (a.unit0 = 0; a.unit0 < a.units; a.unit0 += most * kWaves) {
    Timed t(st, name, a.unit0 ? 0.0 : 2.0 * a.E * a.width,
            a.unit0 ? 0.0
                    : static_cast<double>(a.E) * (4.0 * a.H + 4) + static_cast<double>(a.n_x) * a.width * sizeof(TX) +
                          static_cast<double>(a.n_rows) * a.width * sizeof(TO));
    const int left = (a.units - a.unit0 + kWaves - 1) / kWaves;
    a.blocks = left < most ? left : most;
    const unsigned grid = static_cast<unsigned>(a.blocks) * a.S;
    launch_sum<TX, TO, PERM>(grid, vw > 1, p.Gl == 6, a.H % 4 == 0 && aligned16(a.w), st, a, X, out);
    EGNN_CHECK_LAUNCH();
  }
  if (p.pieces) {
    Timed t(st, "attn_long_sum", 0.0, 0.0);
    long_sum_kernel<TO, PERM><<<dim3(static_cast<unsigned>(p.pieces / 2), ceil_div(a.width, kThreads)), kThreads, 0,
                                st>>>(a, out);
    EGNN_CHECK_LAUNCH();
  }
  return EGNN_OK;
}

template <typename T, int VW, bool ONE>
void launch_logits(unsigned grid, size_t lds, int nit, hipStream_t st, const LogitArgs &a, const T *q, const T *k) {
  if (nit <= 1) logits_kernel<T, VW, 1, ONE><<<grid, kThreads, lds, st>>>(a, q, k);
  else if (nit <= 2) logits_kernel<T, VW, 2, ONE><<<grid, kThreads, lds, st>>>(a, q, k);
  else logits_kernel<T, VW, 4, ONE><<<grid, kThreads, lds, st>>>(a, q, k);
}

template <typename T, int VW, bool ONE>
void launch_logit_grad(unsigned grid, size_t lds, int nit, hipStream_t st, const GradArgs &a, const float *go,
                       const T *v) {
  if (nit <= 1) logit_grad_kernel<T, VW, 1, ONE><<<grid, kThreads, lds, st>>>(a, go, v);
  else if (nit <= 4) logit_grad_kernel<T, VW, 4, ONE><<<grid, kThreads, lds, st>>>(a, go, v);
  else logit_grad_kernel<T, VW, 8, ONE><<<grid, kThreads, lds, st>>>(a, go, v);
}

int rounds_of(int vectors, const Team &t) {
  const int LT = 1 << t.LTl;
  return (vectors + LT - 1) / LT;
}

template <typename T>
egnn_status forward(const Shape &s, const egnn_graph *g, const T *q, const T *k, const T *v, const float *lam,
                    const float *bias, const uint8_t *mask, const uint64_t *rng, uint32_t site, T *out, void *saved,
                    char *ws, hipStream_t st) {
  const bool train = saved != nullptr;
  const Saved sv = carve_saved(s, train ? static_cast<char *>(saved) : ws);
  if (!train) ws += saved_bytes_of(s);
  auto *piece_stats = reinterpret_cast<float2 *>(ws);
  ws += align256(static_cast<size_t>(s.pieces) * 2 * s.H * 8);
  if (s.n_dst == 0) return EGNN_OK;
  LogitArgs a{};
  a.row_ptr = g->row_ptr;
  a.src = g->src;
  a.n_dst = s.n_dst;
  a.n_src = s.n_src;
  a.E = s.E;
  a.T = s.T;
  a.H = s.H;
  a.D = s.D;
  a.ldq = s.ldq;
  a.ldk = s.ldk;
  a.scale = s.scale;
  a.bias = bias;
  a.mask = mask;
  a.lam = lam;
  a.drop = make_drop(rng, site, s.t);
  a.logits = train || s.pieces ? sv.logits : nullptr;
  a.w = sv.w;
  a.stats = sv.stats;
  a.dst = sv.dst;
  a.piece_stats = piece_stats;
  if (s.E > 0) {
    constexpr int V = 16 / sizeof(T);
    const bool vec = vec_width<T>(s.D, s.ldq, q) > 1 && vec_width<T>(s.D, s.ldk, k) > 1;
    const int vectors = vec ? s.D / V : s.D;
    a.team = make_team(2 * s.H, vectors);
    const unsigned grid = static_cast<unsigned>(s.n_dst + s.pieces);
    const size_t lds = static_cast<size_t>(s.T) * (2 * s.H + 1) * 4;
    {
      Timed t(st, "attn_logits", 4.0 * s.E * s.H * s.D,
              static_cast<double>(s.E) * (12.0 * s.H + 8 + (bias ? 8.0 * s.H : 0)) +
                  2.0 * s.H * s.D * sizeof(T) * (static_cast<double>(s.n_dst) + s.n_src));
      const int nit = rounds_of(vectors, a.team);
      const bool one = a.team.LTl + a.team.Hpl == 6;
      if (vec && one) launch_logits<T, V, true>(grid, lds, nit, st, a, q, k);
      else if (vec) launch_logits<T, V, false>(grid, lds, nit, st, a, q, k);
      else launch_logits<T, 1, false>(grid, lds, nit, st, a, q, k);
      EGNN_CHECK_LAUNCH();
    }
    if (s.pieces) {
      Timed t(st, "attn_long_weights", 0.0, 0.0);
      long_weights_kernel<<<static_cast<unsigned>(s.pieces), kThreads, 0, st>>>(a);
      EGNN_CHECK_LAUNCH();
    }
  }
  SumArgs m{};
  m.ptr = g->row_ptr;
  m.col = g->src;
  m.row_of = sv.dst;
  m.n_rows = s.n_dst;
  m.n_x = s.n_src;
  m.E = s.E;
  m.ldx = s.ldv;
  m.w = sv.w;
  m.H = s.H;
  m.C = s.C;
  m.Ch = s.C / s.H;
  m.width = s.K * s.C;
  m.scale = 1.0f;
  m.part = reinterpret_cast<float *>(ws);
  return run_sum<T, T, false>(m, v, out, "attn_out", st);
}

template <typename T>
egnn_status backward(const Shape &s, const egnn_graph *g, const T *q, const T *k, const T *v, const float *lam,
                     const uint64_t *rng, uint32_t site, const void *saved, const float *go, float *gq, float *gk,
                     float *gv, float *glam, float *gbias, char *ws, hipStream_t st) {
  const Saved sv = carve_saved(s, static_cast<char *>(const_cast<void *>(saved)));
  const size_t E = s.E, H = s.H;
  float *dl = gbias ? gbias : reinterpret_cast<float *>(ws);
  ws += align256(E * 2 * H * 4);
  auto *t1 = reinterpret_cast<float *>(ws);
  ws += align256(static_cast<size_t>(s.n_dst) * H * 4);
  float *u = nullptr;
  float2 *piece_t = nullptr;
  if (s.pieces) {
    u = reinterpret_cast<float *>(ws);
    ws += align256(E * H * 4);
    piece_t = reinterpret_cast<float2 *>(ws);
    ws += align256(static_cast<size_t>(s.pieces) * H * 8);
  }
  auto *part = reinterpret_cast<float *>(ws);
  constexpr int V = 16 / sizeof(T);
  const int Ch = s.C / s.H;
  if (s.n_dst > 0) {
    GradArgs a{};
    a.row_ptr = g->row_ptr;
    a.src = g->src;
    a.dst = sv.dst;
    a.n_dst = s.n_dst;
    a.n_src = s.n_src;
    a.E = s.E;
    a.T = s.T;
    a.H = s.H;
    a.C = s.C;
    a.K = s.K;
    a.ldv = s.ldv;
    a.lam = lam;
    a.drop = make_drop(rng, site, s.t);
    a.logits = reinterpret_cast<const float2 *>(sv.logits);
    a.stats = sv.stats;
    a.dl = reinterpret_cast<float2 *>(dl);
    a.t1 = t1;
    a.u = u;
    a.piece_t = piece_t;
    const bool vec = vec_width<T>(Ch, s.ldv, v) > 1 && aligned16(go);
    const int vectors = s.K * (vec ? Ch / V : Ch);
    a.team = make_team(s.H, vectors);
    const unsigned grid = static_cast<unsigned>(s.n_dst + s.pieces);
    const size_t lds = static_cast<size_t>(s.T) * (s.H + 1) * 4;
    {
      Timed t(st, "attn_logit_grad", 2.0 * s.E * s.K * s.C,
              static_cast<double>(s.E) * (16.0 * s.H + 4) +
                  static_cast<double>(s.K) * s.C * (4.0 * s.n_dst + sizeof(T) * static_cast<double>(s.n_src)));
      const int nit = rounds_of(vectors, a.team);
      const bool one = a.team.LTl + a.team.Hpl == 6;
      if (vec && one) launch_logit_grad<T, V, true>(grid, lds, nit, st, a, go, v);
      else if (vec) launch_logit_grad<T, V, false>(grid, lds, nit, st, a, go, v);
      else launch_logit_grad<T, 1, false>(grid, lds, nit, st, a, go, v);
      EGNN_CHECK_LAUNCH();
    }
    if (s.pieces) {
      Timed t(st, "attn_long_grad", 0.0, 0.0);
      long_grad_kernel<<<static_cast<unsigned>(s.pieces), kThreads, 0, st>>>(a);
      EGNN_CHECK_LAUNCH();
    }
  }
  {
    Timed t(st, "attn_lam_grad", 0.0, 4.0 * s.n_dst * s.H);
    lam_grad_kernel<<<s.H, kThreads, 0, st>>>(t1, s.n_dst, s.H, glam);
    EGNN_CHECK_LAUNCH();
  }
  SumArgs m{};
  m.ptr = g->row_ptr;
  m.col = g->src;
  m.row_of = sv.dst;
  m.n_rows = s.n_dst;
  m.n_x = s.n_src;
  m.E = s.E;
  m.ldx = s.ldk;
  m.w = dl;
  m.H = 2 * s.H;
  m.C = 2 * s.H * s.D;
  m.Ch = s.D;
  m.width = 2 * s.H * s.D;
  m.scale = s.scale;
  m.part = part;
  egnn_status r = run_sum<T, float, false>(m, k, gq, "attn_grad_q", st);
  if (r != EGNN_OK) return r;
  m.ptr = g->src_ptr;
  m.perm = g->src_perm;
  m.col = sv.dst;
  m.row_of = g->src;
  m.n_rows = s.n_src;
  m.n_x = s.n_dst;
  m.ldx = s.ldq;
  r = run_sum<T, float, true>(m, q, gk, "attn_grad_k", st);
  if (r != EGNN_OK) return r;
  m.ldx = static_cast<int64_t>(s.K) * s.C;
  m.w = sv.w;
  m.H = s.H;
  m.C = s.C;
  m.Ch = Ch;
  m.width = s.K * s.C;
  m.scale = 1.0f;
  return run_sum<float, float, true>(m, go, gv, "attn_grad_v", st);
}

}  // namespace

extern "C" egnn_status egnn_diff_attention_sizes(const egnn_attn_desc *d, const egnn_graph *g, size_t *saved_bytes,
                                                 size_t *ws_infer_bytes, size_t *ws_train_bytes) {
  Shape s;
  const egnn_status st = make_shape_of(d, g, &s);
  if (st != EGNN_OK) return st;
  EGNN_REQUIRE(saved_bytes && ws_infer_bytes && ws_train_bytes, "size outputs are required");
  *saved_bytes = saved_bytes_of(s);
  *ws_infer_bytes = ws_fwd_of(s, false);
  const size_t f = ws_fwd_of(s, true), b = ws_bwd_of(s);
  *ws_train_bytes = f > b ? f : b;
  return EGNN_OK;
}

extern "C" egnn_status egnn_diff_attention_fwd(const egnn_attn_desc *d, const egnn_graph *g, const void *q,
                                               const void *k, const void *v, const float *lam, const float *bias,
                                               const uint8_t *mask, const uint64_t *rng, void *out, void *saved,
                                               void *ws, size_t ws_bytes, hipStream_t stream) {
  Shape s;
  const egnn_status st = make_shape_of(d, g, &s);
  if (st != EGNN_OK) return st;
  if (s.n_dst == 0) return EGNN_OK;
  EGNN_REQUIRE(g->row_ptr && (s.E == 0 || g->src), "the graph's row_ptr and src are required");
  EGNN_REQUIRE(out && (s.E == 0 || (q && k && v && lam)), "q, k, v, lam and out are required");
  EGNN_REQUIRE(rng || s.t == 0, "rng state is required when the dropout probability is not zero");
  EGNN_REQUIRE((reinterpret_cast<uintptr_t>(rng) & 7) == 0, "rng state must be 8-byte aligned");
  EGNN_REQUIRE(aligned16(saved) && aligned16(ws), "saved and workspace must be 16-byte aligned");
  const size_t need = ws_fwd_of(s, saved != nullptr);
  if (need > 0 && (!ws || ws_bytes < need)) {
    set_error("workspace of %zu bytes, needs %zu", ws ? ws_bytes : size_t(0), need);
    return EGNN_E_WORKSPACE;
  }
  if (s.storage == EGNN_BF16)
    return forward<uint16_t>(s, g, static_cast<const uint16_t *>(q), static_cast<const uint16_t *>(k),
                             static_cast<const uint16_t *>(v), lam, bias, mask, rng, d->site,
                             static_cast<uint16_t *>(out), saved, static_cast<char *>(ws), stream);
  return forward<float>(s, g, static_cast<const float *>(q), static_cast<const float *>(k),
                        static_cast<const float *>(v), lam, bias, mask, rng, d->site, static_cast<float *>(out), saved,
                        static_cast<char *>(ws), stream);
}

extern "C" egnn_status egnn_diff_attention_bwd(const egnn_attn_desc *d, const egnn_graph *g, const void *q,
                                               const void *k, const void *v, const float *lam, const uint64_t *rng,
                                               const void *saved, const float *grad_out, float *grad_q, float *grad_k,
                                               float *grad_v, float *grad_lam, float *grad_bias, void *ws,
                                               size_t ws_bytes, hipStream_t stream) {
  Shape s;
  const egnn_status st = make_shape_of(d, g, &s);
  if (st != EGNN_OK) return st;
  EGNN_REQUIRE(g->row_ptr && (s.E == 0 || g->src), "the graph's row_ptr and src are required");
  EGNN_REQUIRE(g->src_ptr && (s.E == 0 || g->src_perm), "the backward needs the graph's src_ptr and src_perm");
  EGNN_REQUIRE(grad_lam && (s.n_dst == 0 || grad_q) && (s.n_src == 0 || (grad_k && grad_v)),
               "grad_q, grad_k, grad_v and grad_lam are required");
  EGNN_REQUIRE(s.E == 0 || (q && k && v && lam && saved && grad_out), "q, k, v, lam, saved and grad_out are required");
  EGNN_REQUIRE(rng || s.t == 0, "rng state is required when the dropout probability is not zero");
  EGNN_REQUIRE((reinterpret_cast<uintptr_t>(rng) & 7) == 0, "rng state must be 8-byte aligned");
  EGNN_REQUIRE(aligned16(saved) && aligned16(ws), "saved and workspace must be 16-byte aligned");
  EGNN_REQUIRE((reinterpret_cast<uintptr_t>(grad_bias) & 7) == 0, "grad_bias must be 8-byte aligned");
  const size_t need = ws_bwd_of(s);
  if (need > 0 && (!ws || ws_bytes < need)) {
    set_error("workspace of %zu bytes, needs %zu", ws ? ws_bytes : size_t(0), need);
    return EGNN_E_WORKSPACE;
  }
  if (s.storage == EGNN_BF16)
    return backward<uint16_t>(s, g, static_cast<const uint16_t *>(q), static_cast<const uint16_t *>(k),
                              static_cast<const uint16_t *>(v), lam, rng, d->site, saved, grad_out, grad_q, grad_k,
                              grad_v, grad_lam, grad_bias, static_cast<char *>(ws), stream);
  return backward<float>(s, g, static_cast<const float *>(q), static_cast<const float *>(k),
                         static_cast<const float *>(v), lam, rng, d->site, saved, grad_out, grad_q, grad_k, grad_v,
                         grad_lam, grad_bias, static_cast<char *>(ws), stream);
}
