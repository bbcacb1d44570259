// Differential attention over the incoming edges of each destination row,
// forward and backward (see egnn.h).
//
//   l[e,h,s] = scale <q[d,h,s], k[src,h,s]> + bias[e,h,s]      s = 0, 1
//   a[.,h,s] = softmax of l over the row's edges
//   w[e,h]   = m[e,h] (a[e,h,0] - lam[h] a[e,h,1]),  m = dropout factor
//   out[d,k,c] = sum_e w[e,h(c)] v[src,k,c]
//
// Two shapes of work carry both directions:
//   products   per edge and head, a dot of a destination's row with a source's
//              row: the logits, with the row's softmax in the same block, and
//              <grad_out, v>, whose softmax backward is a launch of its own;
//   sums       per row and column, a weighted sum of gathered rows: out, and the
//              gradients of q, k and v (of k and v over edges grouped by source).
//
// What bounds them: not HBM (the operands are some tens of MB) but the gathered
// rows, edges x row bytes, through the L2s and the vector caches.  So a sum is
// sliced by columns and a product's rows are cut by source, one slice or part
// an XCD, so that each 4 MB L2 holds its own share of the gathered array: the
// rows then come from L2 rather than over the fabric (HfO2-like cell, 544,000
// edges of 6.4 KB: out 340 us unsliced with vector addressing, 168 us now, 21
// TB/s, 92% of the line requests hits; dots 374 us in one part, 152 in eight).
// In bf16 the conversion to fp32 (two instructions a pair) beside the
// multiply-adds is the limit: vector units busy 92% in out of the GeSbTe-like
// cell (1.11 M edges of 6.4 KB, 361 us); its fp32 gradient of v (rows of 12.8
// KB, 702 us, 20 TB/s) is at the lines again.
//
// Rows are handled by one block (logits, softmax) or one wave per slice or
// part (sums, dots).  A row longer than the launch's limit T is cut at the
// multiples of T of the edge array, so pieces need no list and no host
// knowledge of the row lengths: window x = [xT, (x+1)T) holds at most the end
// of one long row (piece 2x: the row that owns edge xT) and the start of
// another (piece 2x+1: the row that owns the window's last edge, if it starts
// inside the window).  Pieces are joined by a later launch, in edge order.
#include <algorithm>
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
constexpr int64_t kMaxStride = 1 << 29;    // a row's pitch in bytes is counted in 32 bits
constexpr int64_t kSliceBytes = 3200000;   // of X in one XCD's L2
constexpr int64_t kPartBytes = 3600000;    // of v in one XCD's L2 (dot products)
constexpr int64_t kPairBytes = 8000000;    // of both X of two sums that share a launch

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
template <> struct Vec<float, 2> {
  __device__ static inline void ld(const float *p, float (&v)[2]) {
    const float2 a = *reinterpret_cast<const float2 *>(p);
    v[0] = a.x; v[1] = a.y;
  }
};
template <> struct Vec<uint16_t, 4> {
  __device__ static inline void ld(const uint16_t *p, float (&v)[4]) {
    const uint2 a = *reinterpret_cast<const uint2 *>(p);
    v[0] = __uint_as_float(a.x << 16); v[1] = __uint_as_float(a.x & 0xFFFF0000u);
    v[2] = __uint_as_float(a.y << 16); v[3] = __uint_as_float(a.y & 0xFFFF0000u);
  }
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

// A byte offset the wave shares, kept on the scalar unit (the compiler
// otherwise folds the row's product into a 64-bit multiply-add per lane).
// Unoptimised code keeps no value there.
__device__ inline uint64_t scalar(uint64_t v) {
#ifdef __OPTIMIZE__
  asm("" : "+s"(v));
#endif
  return v;
}

// One vector as it lies in memory (16 or 8 bytes, or one element), so that loads can
// be issued apart from the conversion; zero bits are zeros in either type.
template <typename T, int VW> struct Raw;
template <> struct Raw<float, 4> {
  float4 r = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  __device__ inline void ld(const float *p) { r = *reinterpret_cast<const float4 *>(p); }
  __device__ inline void get(float (&v)[4]) const { v[0] = r.x; v[1] = r.y; v[2] = r.z; v[3] = r.w; }
};
template <> struct Raw<uint16_t, 8> {
  uint4 r = make_uint4(0, 0, 0, 0);
  __device__ inline void ld(const uint16_t *p) { r = *reinterpret_cast<const uint4 *>(p); }
  __device__ inline void get(float (&v)[8]) const {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
};
template <> struct Raw<float, 2> {
  float2 r = make_float2(0.0f, 0.0f);
  __device__ inline void ld(const float *p) { r = *reinterpret_cast<const float2 *>(p); }
  __device__ inline void get(float (&v)[2]) const { v[0] = r.x; v[1] = r.y; }
};
template <> struct Raw<uint16_t, 4> {
  uint2 r = make_uint2(0, 0);
  __device__ inline void ld(const uint16_t *p) { r = *reinterpret_cast<const uint2 *>(p); }
  __device__ inline void get(float (&v)[4]) const {
    v[0] = __uint_as_float(r.x << 16); v[1] = __uint_as_float(r.x & 0xFFFF0000u);
    v[2] = __uint_as_float(r.y << 16); v[3] = __uint_as_float(r.y & 0xFFFF0000u);
  }
};
template <typename T> struct Raw<T, 1> {
  T r = 0;
  __device__ inline void ld(const T *p) { r = *p; }
  __device__ inline void get(float (&v)[1]) const { v[0] = Store<T>::ld(&r); }
};

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

// exp(x), x <= 0 (or NaN): 2^t with t = x log2 e, whose rounding error r is
// put back as a factor 1 + r ln 2.  Within 2 ulp for any x, where 2^t alone is
// off by |x| / 2 ulp; infinity and what underflows give 0.
__device__ inline float exp_of(float x) {
  constexpr float kHi = 1.44269502f, kLo = 1.92596299e-8f, kLn2 = 0.693147181f;  // log2 e in two parts
  x = x < -150.0f ? -150.0f : x;
  const float t = x * kHi;
  const float r = fmaf(x, kLo, fmaf(x, kHi, -t));
  const float y = __builtin_amdgcn_exp2f(t);
  return fmaf(y, r * kLn2, y);
}

struct MaxOp { __device__ float operator()(float a, float b) const { return fmaxf(a, b); } };
struct SumOp { __device__ float operator()(float a, float b) const { return a + b; } };

// softmax weight of a logit: (M, 1/S) of its row.  Rows with nothing left have
// M = 0, 1/S = 0; a masked logit is -inf and gives 0.
__device__ inline float weight_of(float l, float2 st) { return exp_of(l - st.x) * st.y; }

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

// Block b's slice (or part) of `slices`, and its number among the slice's
// `blocks` blocks.  Consecutive blocks go to the eight XCDs in turn; eight
// slices at a time keep one XCD each, and the last r = slices % 8 (1, 2 or 4)
// are dealt over all XCDs, 8 / r to a slice, so that none idles.
struct Slot {
  int slice, block;
};
__device__ inline Slot slot_of(int slices, int blocks, int b) {
  const int full = slices >> 3, r = slices & 7, t = b - full * 8 * blocks;
  if (t < 0) return Slot{((b >> 3) / blocks) * 8 + (b & 7), (b >> 3) % blocks};
  if (r == 0) return Slot{slices, 0};  // padding behind the last slice
  return Slot{full * 8 + t % r, t / r};
}

// ------------------------------------------------------------------ products

// Lane layout of the dot products of rows [K][C] over H heads, in vectors of
// VW elements.
//   natural (H and the vectors of a head powers of two, a component's vectors
//   at most a wave): lane = (edge sub, component sub, vector of the
//   component), so that four neighbouring lanes read 64 contiguous bytes: the
//   vector cache looks up one line for four lanes at a time, and a head's
//   lanes side by side instead (the other layout) cost twice the lookups
//   where a head has 32 bytes of a component;
//   by head (any shape): lane = (edge sub, head, part).
// The partial products of a head are summed over the lane bits [0, low) and
// [hi0, hi1).
struct Team {
  bool natural;
  int low, hi0, hi1;
  int esh;           // log2 of the lanes an edge takes
  int NCl, KSl;      // natural: log2 of a component's vectors, of the components side by side
  int rounds, nit;   // vectors a lane: rounds of nit
};

constexpr int kMaxNit = 7;  // vectors of A a lane keeps in registers

inline int log2_ceil(int n) {
  int l = 0;
  while ((1 << l) < n) ++l;
  return l;
}

inline bool pow2(int n) { return (n & (n - 1)) == 0; }

inline Team make_team(int K, int H, int P) {
  Team t{};
  const int NC = H * P;
  t.natural = pow2(H) && pow2(P) && NC <= kWave;
  if (t.natural) {
    t.NCl = log2_ceil(NC);
    const int want = log2_ceil(K);
    t.KSl = want < 6 - t.NCl ? want : 6 - t.NCl;
    t.low = log2_ceil(P);
    t.hi0 = t.NCl;
    t.hi1 = t.esh = t.NCl + t.KSl;
    t.nit = (K + (1 << t.KSl) - 1) >> t.KSl;
  } else {
    const int Hpl = log2_ceil(H), want = log2_ceil(K * P);
    t.low = want < 6 - Hpl ? want : 6 - Hpl;
    t.hi0 = t.hi1 = 0;
    t.esh = t.low + Hpl;
    t.nit = (K * P + (1 << t.low) - 1) >> t.low;
  }
  t.rounds = (t.nit + kMaxNit - 1) / kMaxNit;
  t.nit = (t.nit + t.rounds - 1) / t.rounds;
  return t;
}

template <int CTRL> __device__ inline float dpp_move(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xF, 0xF, true));
}

// v plus the value in the lane that differs in bit `bit` only
__device__ inline float add_across(float v, int bit) {
  if (bit == 5) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
  if (bit == 4) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
  return v + __shfl_xor(v, 1 << bit);
}

// dot[u] summed over the team; every lane of a team gets the sum.  The low
// bits take DPP moves inside a row of 16 (a quad's lanes hold the same value
// when the mirrors swap quads).
template <int U>
__device__ inline void team_sum(float (&dot)[U], const Team &tm) {
  if (tm.low > 0)
#pragma unroll
    for (int u = 0; u < U; ++u) dot[u] += dpp_move<0xB1>(dot[u]);   // quad [1,0,3,2]
  if (tm.low > 1)
#pragma unroll
    for (int u = 0; u < U; ++u) dot[u] += dpp_move<0x4E>(dot[u]);   // quad [2,3,0,1]
  if (tm.low > 2)
#pragma unroll
    for (int u = 0; u < U; ++u) dot[u] += dpp_move<0x141>(dot[u]);  // mirror within 8
  if (tm.low > 3)
#pragma unroll
    for (int u = 0; u < U; ++u) dot[u] += dpp_move<0x140>(dot[u]);  // mirror within 16
  for (int bit = 4; bit < tm.low; ++bit)
#pragma unroll
    for (int u = 0; u < U; ++u) dot[u] = add_across(dot[u], bit);
  for (int bit = tm.hi0; bit < tm.hi1; ++bit)
#pragma unroll
    for (int u = 0; u < U; ++u) dot[u] = add_across(dot[u], bit);
}

// put(i, h, dot, first) for the edges i < cnt of i_first, i_first + stride, ...
// (and, where a wave takes several at once, those that follow each), dot = sum
// over the head's vectors of A . B[scol[i]] (row 0 for a source of -1).  A
// stays in registers, NIT vectors a lane; what does not fit is added by further
// rounds (first = false).  ONE: a wave takes one edge at a time, so the row's
// address is scalar work.
template <typename TA, typename TB, int VW, int NIT, bool ONE, typename Put>
__device__ inline void edge_dots(const TA *arow, const TB *B, int64_t ldb, const int *scol, int i_first, int stride,
                                 int cnt, int K, int H, int C, const Team &tm, Put put) {
  // edges in flight: 6 to 10 loads (two edges of 7 took 522 us where one takes
  // 477: bf16 rows of 6.4 KB, 1.1 M edges; their registers cost a wave)
  constexpr int U = NIT == 1 ? 8 : NIT == 2 ? 4 : NIT == 3 ? 3 : NIT <= 5 ? 2 : 1;
  const int lane = threadIdx.x & (kWave - 1);
  const int Ch = C / H, P = Ch / VW;
  const int es = ONE ? 0 : lane >> tm.esh;
  const uint32_t pitch = static_cast<uint32_t>(ldb * sizeof(TB));
  // this lane's head, first vector and step: vector n of the lane lies at
  // component k(n), and exists while k(n) < K
  int h, t0;
  if (tm.natural) {
    const int col = lane & ((1 << tm.NCl) - 1);
    h = col >> tm.low;
    t0 = (lane >> tm.NCl) & ((1 << tm.KSl) - 1);
  } else {
    h = (lane >> tm.low) & ((1 << (tm.esh - tm.low)) - 1);
    t0 = lane & ((1 << tm.low) - 1);
  }
  const bool writes = (lane & ((1 << tm.low) - 1)) == 0 && (!tm.natural || t0 == 0) && h < H;
  const int hc = min(h, H - 1);
  // vector m of the lane goes to round m % rounds, so that only a round's last
  // (n = NIT - 1) may be missing in some or all lanes
  for (int r = 0; r < tm.rounds; ++r) {
    float af[NIT][VW];
    uint32_t off[NIT];
    bool have = true;
#pragma unroll
    for (int n = 0; n < NIT; ++n) {
      const int m = n * tm.rounds + r;
      if (tm.natural) {
        const int k = (m << tm.KSl) + t0;
        have = k < K;
        off[n] = min(k, K - 1) * C + (lane & ((1 << tm.NCl) - 1)) * VW;
      } else {
        const int j = (m << tm.low) + t0;
        have = j < K * P;
        const int jj = min(j, K * P - 1);
        off[n] = (jj / P) * C + hc * Ch + (jj % P) * VW;
      }
      Vec<TA, VW>::ld(arow + off[n], af[n]);
      off[n] *= sizeof(TB);
    }
#pragma unroll
    for (int x = 0; x < VW; ++x) af[NIT - 1][x] = have ? af[NIT - 1][x] : 0.0f;
    for (int i0 = i_first; i0 < cnt; i0 += stride * U) {
      Raw<TB, VW> v[U][NIT];
      float dot[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = min(i0 + u * stride + es, cnt - 1);
        const uint32_t s = max(ONE ? uniform(scol[i]) : scol[i], 0);
        uint64_t at = static_cast<uint64_t>(s) * pitch;
        if constexpr (ONE) at = scalar(at);
        const char *row = reinterpret_cast<const char *>(B) + at;
#pragma unroll
        for (int n = 0; n < NIT - 1; ++n) v[u][n].ld(reinterpret_cast<const TB *>(row + off[n]));
        // a vector that is not there is not read: what lies at a clamped place
        // (an infinity) must not meet the 0 in A, nor cost a lookup
        if (have) v[u][NIT - 1].ld(reinterpret_cast<const TB *>(row + off[NIT - 1]));
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        dot[u] = 0.0f;
#pragma unroll
        for (int n = 0; n < NIT; ++n) {
          float x[VW];
          v[u][n].get(x);
#pragma unroll
          for (int y = 0; y < VW; ++y) dot[u] = fmaf(af[n][y], x[y], dot[u]);
        }
      }
      team_sum<U>(dot, tm);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = i0 + u * stride + es;
        if (writes && i < cnt) put(i, h, dot[u], r == 0);
      }
    }
  }
}

struct LogitArgs {
  const int *row_ptr, *src;
  int n_dst, n_src, E, H, D;      // H heads of two maps
  int T, TP;                      // edges in LDS at a time; of a piece (longer rows are cut)
  int Hpl;                        // log2 of the maps' columns, padded
  int64_t ldq, ldk;
  float scale;
  const float *bias;              // [E][2H] or null
  const uint8_t *mask;            // [E] or null
  const float *lam;
  Drop drop;
  Team team;
  float2 *maps;                   // [E][H] weights of both maps; logits until a row beyond T is done
  bool keep;                      // the backward wants maps
  float *w;                       // [H][ldw]
  int64_t ldw;
  int *dst;                       // [E]
  float2 *piece_stats;            // [pieces][2H]
};

// Writes the weights m x(i, h) of edges [b, b + cnt) to their planes.  A thread
// writes its edge's heads, so that a wave's lanes write neighbouring edges of a
// plane, and draws eight decisions at a time.
template <typename X> __device__ inline void put_weights(const LogitArgs &a, int b, int cnt, X x) {
  DropKey key{};
  if (a.drop.t != 0) key = drop_key(a.drop);
  for (int i = threadIdx.x; i < cnt; i += kThreads) {
    const int64_t at = static_cast<int64_t>(b + i) * a.H;
    // heads of one draw group after another; the groups start at multiples of 8 of at + h
    for (int h0 = -static_cast<int>(at & 7); h0 < a.H; h0 += 8) {
      uint4 draws = make_uint4(0, 0, 0, 0);
      if (a.drop.t != 0) draws = philox4x32(static_cast<uint64_t>((at + h0) >> 3), key);
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int h = h0 + u;
        if (h < 0 || h >= a.H) continue;
        float w = x(i, h);
        if (a.drop.t != 0) w = drop_draw(draws, u) >= a.drop.t ? w * a.drop.factor : 0.0f;
        a.w[h * a.ldw + b + i] = w;
      }
    }
  }
}

// Edge weights of [b, e) whose logits are in a.maps, T edges at a time through
// lds [T][H + 1].  (Pieces of 373,000 edges, 16 heads, training: 75 us with a
// thread's eight weights straight to their planes, 43 so.)
__device__ inline void edge_weights(const LogitArgs &a, const float2 *fin, int b, int e, float *lds) {
  const int H = a.H, pitch = H + 1;
  for (int c0 = b; c0 < e; c0 += a.T) {
    const int cnt = min(a.T, e - c0);
    float2 *maps = a.maps + static_cast<int64_t>(c0) * H;
    __syncthreads();  // the last chunk's are no longer read
    for (int f = threadIdx.x; f < cnt * H; f += kThreads) {
      const int i = f / H, h = f - i * H;
      const float2 l = maps[f];
      const float2 al = make_float2(weight_of(l.x, fin[2 * h]), weight_of(l.y, fin[2 * h + 1]));
      if (a.keep) maps[f] = al;
      lds[i * pitch + h] = al.x - a.lam[h] * al.y;
    }
    __syncthreads();
    put_weights(a, c0, cnt, [&](int i, int h) { return lds[i * pitch + h]; });
  }
}

// One block per row (or piece): logits, T edges at a time, with the running
// maximum and sum of each map, and, for whole rows, the edge weights.
template <typename T, int VW, int NIT, bool ONE>
__global__ void __launch_bounds__(kThreads) logits_kernel(LogitArgs a, const T *__restrict__ q,
                                                          const T *__restrict__ k) {
  extern __shared__ float lg[];  // [T][2H + 1], then the sources [T]
  int *scol = reinterpret_cast<int *>(lg + a.T * (2 * a.H + 1));
  __shared__ float red[kWaves][kWave];
  __shared__ float2 fin[kWave];
  __shared__ float slam[kMaxHeads];
  const int H2 = 2 * a.H, pitch = H2 + 1;
  if (threadIdx.x < static_cast<unsigned>(a.H)) slam[threadIdx.x] = a.lam[threadIdx.x];
  int d, b, e;
  const int p = static_cast<int>(blockIdx.x) - a.n_dst;
  if (p < 0) {
    d = blockIdx.x;
    row_bounds(a.row_ptr, d, a.E, &b, &e);
    if (e - b > a.TP || e == b) return;
  } else {
    const Piece pc = find_piece(p, a.TP, a.row_ptr, a.n_dst, a.E,
                                [&](int pos) { return row_by_search(a.row_ptr, a.n_dst, pos); });
    if (pc.row < 0) return;
    d = pc.row;
    b = pc.begin;
    e = pc.end;
  }
  const int Hp = 1 << a.Hpl;
  const int col = threadIdx.x & (Hp - 1), r0 = threadIdx.x >> a.Hpl, R = kThreads >> a.Hpl;
  const bool whole = p < 0 && e - b <= a.T;
  float M = -INFINITY, S = 0.0f;
  for (int c0 = b; c0 < e; c0 += a.T) {
    const int cnt = min(a.T, e - c0);
    __syncthreads();  // the last chunk's logits are no longer read
    for (int i = threadIdx.x; i < cnt; i += kThreads) {
      const int s = a.src[c0 + i];
      // -1: takes no part; its products are taken with row 0 and not used
      const bool live = static_cast<unsigned>(s) < static_cast<unsigned>(a.n_src) && !(a.mask && a.mask[c0 + i] == 0);
      scol[i] = live ? s : -1;
      a.dst[c0 + i] = d;
    }
    __syncthreads();
    const int step = ONE ? 1 : kWave >> a.team.esh;
    edge_dots<T, T, VW, NIT, ONE>(q + static_cast<int64_t>(d) * a.ldq, k, a.ldk, scol,
                                  uniform(threadIdx.x >> 6) * step, kWaves * step, cnt, 1, H2, H2 * a.D, a.team,
                                  [&](int i, int h, float x, bool first) {
                                    lg[i * pitch + h] = first ? x : lg[i * pitch + h] + x;
                                  });
    __syncthreads();
    float Mc = -INFINITY;
    if (col < H2)
      for (int i0 = r0; i0 < cnt; i0 += 4 * R) {
        const int64_t o = static_cast<int64_t>(c0) * H2 + col;
        float bv[4];  // loaded together; places past the end are clamped
#pragma unroll
        for (int u = 0; u < 4; ++u) bv[u] = a.bias ? a.bias[o + min(i0 + u * R, cnt - 1) * H2] : 0.0f;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int i = i0 + u * R;
          if (i >= cnt) break;
          float l = lg[i * pitch + col] * a.scale + bv[u];
          if (bv[u] == -INFINITY || scol[i] < 0) l = -INFINITY;  // masked, whatever the product is
          lg[i * pitch + col] = l;
          if (!whole) reinterpret_cast<float *>(a.maps)[o + i * H2] = l;
          Mc = fmaxf(Mc, l);
        }
      }
    const float Mn = fmaxf(M, column_reduce(Mc, Hp, red, MaxOp()));
    float Sc = 0.0f;
    if (col < H2 && Mn != -INFINITY)
      for (int i = r0; i < cnt; i += R) Sc += exp_of(lg[i * pitch + col] - Mn);
    S = (M == -INFINITY ? 0.0f : S * exp_of(M - Mn)) + column_reduce(Sc, Hp, red, SumOp());
    M = Mn;
  }
  if (p >= 0) {
    if (r0 == 0 && col < H2) a.piece_stats[static_cast<int64_t>(p) * H2 + col] = make_float2(M, S);
    return;
  }
  const float2 st = finish_stats(M, S);
  if (!whole) {
    if (r0 == 0 && col < H2) fin[col] = st;
    __syncthreads();  // orders the logits that this block wrote to memory, too
    edge_weights(a, fin, b, e, lg);
    return;
  }
  const int cnt = e - b;
  if (col < H2)
    for (int i = r0; i < cnt; i += R) {
      const float al = weight_of(lg[i * pitch + col], st);
      lg[i * pitch + col] = al;
      if (a.keep) reinterpret_cast<float *>(a.maps)[static_cast<int64_t>(b + i) * H2 + col] = al;
    }
  __syncthreads();
  put_weights(a, b, cnt, [&](int i, int h) { return lg[i * pitch + 2 * h] - slam[h] * lg[i * pitch + 2 * h + 1]; });
}

// Long rows: the pieces' statistics joined, then their edge weights.
__global__ void __launch_bounds__(kThreads) long_weights_kernel(LogitArgs a) {
  extern __shared__ float lds[];  // [T][H + 1]
  __shared__ float red[kWaves][kWave];
  __shared__ float2 fin[kWave];
  const Piece pc = find_piece(blockIdx.x, a.TP, a.row_ptr, a.n_dst, a.E, [&](int pos) { return a.dst[pos]; });
  if (pc.row < 0) return;
  int b, e;
  row_bounds(a.row_ptr, pc.row, a.E, &b, &e);
  const int H2 = 2 * a.H, Hp = 1 << a.Hpl;
  const int col = threadIdx.x & (Hp - 1), r0 = threadIdx.x >> a.Hpl, R = kThreads >> a.Hpl;
  const int n = piece_count(b, e, a.TP);
  float own = -INFINITY, S = 0.0f;  // of this thread's pieces
  if (col < H2)
    for (int i0 = r0; i0 < n; i0 += 8 * R) {
      float2 st[8];  // loaded together
#pragma unroll
      for (int u = 0; u < 8; ++u)
        st[u] = a.piece_stats[static_cast<int64_t>(piece_id(b, a.TP, min(i0 + u * R, n - 1))) * H2 + col];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        if (i0 + u * R >= n || st[u].x == -INFINITY) continue;
        const float top = fmaxf(own, st[u].x);
        S = (own == -INFINITY ? 0.0f : S * exp_of(own - top)) + st[u].y * exp_of(st[u].x - top);
        own = top;
      }
    }
  const float M = column_reduce(own, Hp, red, MaxOp());
  S = column_reduce(own == -INFINITY ? 0.0f : S * exp_of(own - M), Hp, red, SumOp());
  if (r0 == 0 && col < H2) fin[col] = finish_stats(M, S);
  __syncthreads();
  edge_weights(a, fin, pc.begin, pc.end, lds);
}

struct DotArgs {
  const int *row_ptr, *src, *dst;
  int n_dst, n_src, E, T;
  int K, C, H;
  int64_t ldv;
  Team team;
  int parts, unit0, units, blocks;
  float *u;  // [E][H]
};

// u[e][h] = <grad_out[d], v[src]> over the head's channels.  One wave per (row
// or piece, part of its edges).  Part p of every row goes to XCD p % 8 and
// starts after as many edges as there are sources below p n_src / parts: a
// partition of the row whatever its order, and where the sources ascend (as
// egnn_build_graph writes them) the part's sources are one stretch of v, which
// the XCD's L2 then holds for all rows.
template <typename T, int VW, int NIT, bool ONE>
__global__ void __launch_bounds__(kThreads) value_dots_kernel(DotArgs a, const float *__restrict__ go,
                                                              const T *__restrict__ v) {
  __shared__ int scol[kWaves][kWave];
  const Slot sl = slot_of(a.parts, a.blocks, blockIdx.x);
  const int lane = threadIdx.x & (kWave - 1), wave = uniform(threadIdx.x >> 6);
  const int unit = a.unit0 + sl.block * kWaves + wave;
  if (unit >= a.units) return;
  int d = unit, b, e;
  if (unit < a.n_dst) {
    row_bounds(a.row_ptr, d, a.E, &b, &e);
    if (e - b > a.T) return;
  } else {
    const Piece pc = find_piece(unit - a.n_dst, a.T, a.row_ptr, a.n_dst, a.E, [&](int pos) { return a.dst[pos]; });
    if (pc.row < 0) return;
    d = pc.row;
    b = pc.begin;
    e = pc.end;
  }
  b = uniform(b);
  e = uniform(e);
  if (unit >= a.n_dst) {  // a piece's sources are near each other already
    const int64_t len = e - b;
    e = uniform(b + static_cast<int>(len * (sl.slice + 1) / a.parts));
    b = uniform(b + static_cast<int>(len * sl.slice / a.parts));
  } else if (a.parts > 1) {
    const int from = static_cast<int>(static_cast<int64_t>(a.n_src) * sl.slice / a.parts);
    const int to = static_cast<int>(static_cast<int64_t>(a.n_src) * (sl.slice + 1) / a.parts);
    int below = 0, upto = 0;
    for (int c0 = b; c0 < e; c0 += kWave) {
      const int s = c0 + lane < e ? a.src[c0 + lane] : INT32_MAX;
      below += __popcll(__ballot(s < from));
      upto += __popcll(__ballot(s < to));
    }
    // the first part starts at the row's start and the last ends at its end, whatever the sources are
    e = sl.slice + 1 < a.parts ? uniform(b + upto) : e;
    b = sl.slice > 0 ? uniform(b + below) : b;
  }
  for (int c0 = b; c0 < e; c0 += kWave) {
    const int cnt = min(kWave, e - c0);
    const int s = lane < cnt ? a.src[c0 + lane] : -1;
    scol[wave][lane] = static_cast<unsigned>(s) < static_cast<unsigned>(a.n_src) ? s : -1;
    wave_lds_order();
    edge_dots<float, T, VW, NIT, ONE>(go + static_cast<int64_t>(d) * a.K * a.C, v, a.ldv, scol[wave], 0,
                                      ONE ? 1 : kWave >> a.team.esh, cnt, a.K, a.H, a.C, a.team,
                                      [&](int i, int h, float x, bool first) {
                                        float *o = a.u + static_cast<int64_t>(c0 + i) * a.H + h;
                                        *o = first ? x : *o + x;
                                      });
    wave_lds_order();
  }
}

struct GradArgs {
  const int *row_ptr, *dst;
  int n_dst, E, H;
  int T, TP, Hpl;
  const float *lam;
  Drop drop;
  const float2 *maps;    // [E][H] the forward's weights of both maps
  float2 *dl;            // [E][H] pairs: gradient of the logits before the scale
  float *dlp;            // the same as planes [2H][ldw]
  int64_t ldw;
  float *wr;             // [E][H] the forward's edge weights, again
  float *t1;             // [n_dst][H] sum_e a1 u
  float *u;              // [E][H] in: <grad_out, v>; where a row does not stay in LDS, m times that
  float2 *piece_t;       // [pieces][H] (sum a0 u, sum a1 u)
};

// The logits' gradients of edges [c0, c0 + cnt), whose weights lie in al
// (pitch 2H + 1) and u in us: rows first, then through al into planes.
__device__ inline void logit_grads(const GradArgs &a, int c0, int cnt, const float2 *tt, const float *slam, float *al,
                                   const float *us) {
  const int H = a.H, pitch = 2 * H + 1;
  float2 *dl = a.dl + static_cast<int64_t>(c0) * H;
  for (int f = threadIdx.x; f < cnt * H; f += kThreads) {
    const int i = f / H, h = f - i * H;
    float *w = al + i * pitch + 2 * h;
    const float u = us[f];
    // a weight of exactly 0 (masked) has no gradient, whatever the row of v holds
    const float2 g = make_float2(w[0] == 0.0f ? 0.0f : w[0] * (u - tt[h].x),
                                 w[1] == 0.0f ? 0.0f : -slam[h] * w[1] * (u - tt[h].y));
    dl[f] = g;
    w[0] = g.x;
    w[1] = g.y;
  }
  __syncthreads();
  const int lane = threadIdx.x & (kWave - 1);
  for (int p = threadIdx.x >> 6; p < 2 * H; p += kWaves)
    for (int i = lane; i < cnt; i += kWave) a.dlp[p * a.ldw + c0 + i] = al[i * pitch + p];
}

__device__ inline void load_maps(const GradArgs &a, int c0, int cnt, float *al) {
  const int H = a.H, pitch = 2 * H + 1;
  const float2 *maps = a.maps + static_cast<int64_t>(c0) * H;
  for (int f = threadIdx.x; f < cnt * H; f += kThreads) {
    const int i = f / H, h = f - i * H;
    const float2 w = maps[f];
    al[i * pitch + 2 * h] = w.x;
    al[i * pitch + 2 * h + 1] = w.y;
  }
}

// Rows and pieces of more than T edges: their gradients once the row's sums
// are known.
__device__ inline void logit_grads_again(const GradArgs &a, int b, int e, const float2 *tt, const float *slam, float *al,
                                         float *us) {
  for (int c0 = b; c0 < e; c0 += a.T) {
    const int cnt = min(a.T, e - c0);
    __syncthreads();
    load_maps(a, c0, cnt, al);
    for (int f = threadIdx.x; f < cnt * a.H; f += kThreads) us[f] = a.u[static_cast<int64_t>(c0) * a.H + f];
    __syncthreads();
    logit_grads(a, c0, cnt, tt, slam, al, us);
  }
}

// One block per row (or piece): the softmax's backward for both maps, T edges
// at a time.
__global__ void __launch_bounds__(kThreads) logit_grad_kernel(GradArgs a) {
  extern __shared__ float al[];  // [T][2H + 1], then u [T][H] and the decisions [T][H]
  float *us = al + a.T * (2 * a.H + 1);
  uint8_t *kept = reinterpret_cast<uint8_t *>(us + a.T * a.H);
  __shared__ float red[kWaves][kWave];
  __shared__ float2 tt[kMaxHeads];
  __shared__ float slam[kMaxHeads];
  int d, b, e;
  const int p = static_cast<int>(blockIdx.x) - a.n_dst;
  if (p < 0) {
    d = blockIdx.x;
    row_bounds(a.row_ptr, d, a.E, &b, &e);
    if (e - b > a.TP) return;
    if (e == b) {
      if (threadIdx.x < static_cast<unsigned>(a.H)) a.t1[static_cast<int64_t>(d) * a.H + threadIdx.x] = 0.0f;
      return;
    }
  } else {
    const Piece pc = find_piece(p, a.TP, a.row_ptr, a.n_dst, a.E, [&](int pos) { return a.dst[pos]; });
    if (pc.row < 0) return;
    d = pc.row;
    b = pc.begin;
    e = pc.end;
  }
  const int H = a.H, Hp = 1 << a.Hpl, pitch = 2 * H + 1;
  if (threadIdx.x < static_cast<unsigned>(H)) slam[threadIdx.x] = a.lam[threadIdx.x];  // null only without edges
  const int h = threadIdx.x & (Hp - 1), r0 = threadIdx.x >> a.Hpl, R = kThreads >> a.Hpl;
  const bool again = p >= 0 || e - b > a.T;  // u does not stay in LDS until the row's sums are known
  float t0 = 0.0f, t1 = 0.0f;
  for (int c0 = b; c0 < e; c0 += a.T) {
    const int cnt = min(a.T, e - c0);
    const int64_t o0 = static_cast<int64_t>(c0) * H;
    __syncthreads();
    load_maps(a, c0, cnt, al);
    __syncthreads();
    if (a.drop.t != 0) {
      for_decisions(c0, cnt, H, a.drop, [&](int at, int, int, float m) { kept[at] = m != 0.0f; });
      __syncthreads();
    }
    for (int f = threadIdx.x; f < cnt * H; f += kThreads) {
      const int i = f / H, hd = f - i * H;
      const float *w = al + i * pitch + 2 * hd;
      const bool on = a.drop.t == 0 || kept[f] != 0;
      a.wr[o0 + f] = on ? a.drop.factor * (w[0] - slam[hd] * w[1]) : 0.0f;
      const float x = on ? a.drop.factor * a.u[o0 + f] : 0.0f;
      us[f] = x;
      if (again) a.u[o0 + f] = x;
    }
    __syncthreads();
    if (h < H)
      for (int i = r0; i < cnt; i += R) {
        const float w0 = al[i * pitch + 2 * h], w1 = al[i * pitch + 2 * h + 1], x = us[i * H + h];
        t0 += w0 == 0.0f ? 0.0f : w0 * x;
        t1 += w1 == 0.0f ? 0.0f : w1 * x;
      }
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
  if (again) logit_grads_again(a, b, e, tt, slam, al, us);
  else logit_grads(a, b, e - b, tt, slam, al, us);
}

// Long rows: the pieces' sums joined, then the logits' gradients.
__global__ void __launch_bounds__(kThreads) long_grad_kernel(GradArgs a) {
  extern __shared__ float al[];
  float *us = al + a.T * (2 * a.H + 1);
  __shared__ float red[kWaves][kWave];
  __shared__ float2 tt[kMaxHeads];
  __shared__ float slam[kMaxHeads];
  if (threadIdx.x < static_cast<unsigned>(a.H)) slam[threadIdx.x] = a.lam[threadIdx.x];
  const Piece pc = find_piece(blockIdx.x, a.TP, a.row_ptr, a.n_dst, a.E, [&](int pos) { return a.dst[pos]; });
  if (pc.row < 0) return;
  int b, e;
  row_bounds(a.row_ptr, pc.row, a.E, &b, &e);
  const int H = a.H, Hp = 1 << a.Hpl;
  const int h = threadIdx.x & (Hp - 1), r0 = threadIdx.x >> a.Hpl, R = kThreads >> a.Hpl;
  const int n = piece_count(b, e, a.TP);
  float t0 = 0.0f, t1 = 0.0f;
  if (h < H)
    for (int i0 = r0; i0 < n; i0 += 8 * R) {
      float2 t[8];  // loaded together
#pragma unroll
      for (int u = 0; u < 8; ++u)
        t[u] = a.piece_t[static_cast<int64_t>(piece_id(b, a.TP, min(i0 + u * R, n - 1))) * H + h];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        t0 += i0 + u * R < n ? t[u].x : 0.0f;
        t1 += i0 + u * R < n ? t[u].y : 0.0f;
      }
    }
  t0 = column_reduce(t0, Hp, red, SumOp());
  t1 = column_reduce(t1, Hp, red, SumOp());
  if (r0 == 0 && h < H) {
    tt[h] = make_float2(t0, t1);
    if (pc.begin == b) a.t1[static_cast<int64_t>(pc.row) * H + h] = t1;
  }
  __syncthreads();
  logit_grads_again(a, pc.begin, pc.end, tt, slam, al, us);
}

// ---------------------------------------------------------------------- sums

// Edges in the order of their sources: the row each came to and its weights
// and logit gradients as planes, so that every slice of the sums below reads
// them in sequence.  One wave per 64 edges; a lane reads its edge's rows.
// The last H blocks sum the gradient of lam instead: -sum_d t1[d][h], in a
// fixed order.
template <bool V4>
__global__ void __launch_bounds__(kThreads) regroup_kernel(const int *__restrict__ perm, const int *__restrict__ src_ptr,
                                                           int n_src, int E, int H, const int *__restrict__ dst,
                                                           const float *__restrict__ wr, const float *__restrict__ dl,
                                                           int64_t ldw, int *__restrict__ dst_out,
                                                           float *__restrict__ w_out, float *__restrict__ dl_out,
                                                           const float *__restrict__ t1, int n_dst,
                                                           float *__restrict__ grad_lam) {
  if (blockIdx.x + H >= gridDim.x) {
    __shared__ double red[kThreads];
    const int h = blockIdx.x + H - gridDim.x;
    double sum = 0.0;
    for (int d0 = threadIdx.x; d0 < n_dst; d0 += 16 * kThreads) {
      float v[16];
#pragma unroll
      for (int u = 0; u < 16; ++u) v[u] = t1[static_cast<int64_t>(min(d0 + u * kThreads, n_dst - 1)) * H + h];
#pragma unroll
      for (int u = 0; u < 16; ++u) sum += d0 + u * kThreads < n_dst ? v[u] : 0.0f;
    }
    red[threadIdx.x] = sum;
    __syncthreads();
    for (int o = kThreads / 2; o > 0; o >>= 1) {
      if (threadIdx.x < static_cast<unsigned>(o)) red[threadIdx.x] += red[threadIdx.x + o];
      __syncthreads();
    }
    if (threadIdx.x == 0) grad_lam[h] = static_cast<float>(-red[0]);
    return;
  }
  const int j = blockIdx.x * kThreads + threadIdx.x;
  if (j >= min(max(src_ptr[n_src], 0), E)) return;
  const int e = perm[j];
  const bool live = static_cast<unsigned>(e) < static_cast<unsigned>(E);
  dst_out[j] = live ? dst[e] : -1;
  const int64_t at = static_cast<int64_t>(live ? e : 0) * H;
  if constexpr (V4) {
    for (int h = 0; h < H; h += 4) {
      const float4 x = *reinterpret_cast<const float4 *>(wr + at + h);
      const float4 y = *reinterpret_cast<const float4 *>(dl + 2 * (at + h));
      const float4 z = *reinterpret_cast<const float4 *>(dl + 2 * (at + h) + 4);
      const float w[4] = {x.x, x.y, x.z, x.w}, g[8] = {y.x, y.y, y.z, y.w, z.x, z.y, z.z, z.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) w_out[(h + k) * ldw + j] = live ? w[k] : 0.0f;
#pragma unroll
      for (int k = 0; k < 8; ++k) dl_out[(2 * h + k) * ldw + j] = live ? g[k] : 0.0f;
    }
  } else {
    for (int h = 0; h < H; ++h) w_out[h * ldw + j] = live ? wr[at + h] : 0.0f;
    for (int h = 0; h < 2 * H; ++h) dl_out[h * ldw + j] = live ? dl[2 * at + h] : 0.0f;
  }
}

struct SumArgs {
  const int *ptr;       // [n_rows + 1]
  const int *col;       // [E] row of X of an edge, in row order
  const int *row_of;    // [E] row of an edge; of edge perm[j] at position j where perm is given
  const int *perm;
  int n_rows, n_x, E, T;
  int64_t ldx;
  const float *w;       // planes [H][ldw], in row order
  int64_t ldw;
  int H, C, Ch, width;  // out row = width elements; column c of width has head (c % C) / Ch
  int S, SV, EPW;       // slices, vectors a slice, edges a wave takes at once
  int BE;               // edges staged at a time, a multiple of what a wave takes in flight
  int planes;           // heads a slice meets: all, or where a row is one component those of its columns
  int unit0, units, blocks;  // first unit of the launch; rows + pieces; blocks a slice in the launch
  float scale;
  float *part;          // [pieces][width]
};

__device__ inline int owner(const SumArgs &a, int pos) {
  if (!a.perm) return a.row_of[pos];
  const int ed = a.perm[pos];
  return static_cast<unsigned>(ed) < static_cast<unsigned>(a.E) ? a.row_of[ed] : -1;
}

// A wave stages BE edges: each head's weights side by side (a pitch apart), so
// that a lane reads four edges' weights at once, and the edges' rows of X.  NR
// registers a lane hold the next edges' weights on their way: 64 edges of up
// to NR heads, or (NARROW) 16 edges of up to 4 NR.
template <int NR, bool NARROW> struct Batch {
  static constexpr int kEdges = NARROW ? 16 : kWave, kPitch = kEdges + 4;
  static constexpr int kFloats = (NARROW ? 4 * NR : NR) * kPitch;
  int x;
  float w[NR];

  // Edges past the end and rows outside X have weight 0 and row 0.
  __device__ inline void fetch(const SumArgs &a, const float *planes, int n_planes, int j0, int e, int lane) {
    x = -1;
    if (lane < a.BE && j0 + lane < e) x = a.col[j0 + lane];
    const bool live = static_cast<unsigned>(x) < static_cast<unsigned>(a.n_x);
    const uint64_t there = __ballot(live);
    x = live ? x : 0;
#pragma unroll
    for (int t = 0; t < NR; ++t) w[t] = 0.0f;
    if constexpr (NARROW) {
      const int i = lane & 15, h0 = lane >> 4;
      if ((there >> i) & 1)
#pragma unroll
        for (int t = 0; t < NR; ++t)
          w[t] = planes[min(4 * t + h0, n_planes - 1) * a.ldw + j0 + i];
    } else if (live) {
      // plane t's address is the wave's; planes past the last are read again and not used
#pragma unroll
      for (int t = 0; t < NR; ++t) w[t] = (planes + min(t, n_planes - 1) * a.ldw + j0)[static_cast<uint32_t>(lane)];
    }
  }

  __device__ inline void stage(int lane, float *sw) const {
#pragma unroll
    for (int t = 0; t < NR; ++t) sw[(NARROW ? 4 * t + (lane >> 4) : t) * kPitch + (NARROW ? lane & 15 : lane)] = w[t];
  }
};

// How the rows of X are addressed: one edge at a time with the wave's address
// on the scalar unit; several with 32-bit byte offsets (X below 4 GB); several
// with 64-bit products.
enum { kScalar, kOffset, kLong };

// acc += sum over edges [b, e) of w X; lanes of a group of SV take the vectors
// of their slice, EPW groups an edge each.  Lanes without a vector read
// nothing (a lookup of the vector cache serves four lanes: idle ones would
// cost as much as others).  SAFE skips weights of 0, so that what such a row
// of X holds stays out.
template <typename TX, int VW, int MODE, int NR, bool NARROW, bool MIX, bool SAFE>
__device__ inline void gather_rows(const SumArgs &a, const TX *X, const float *planes, int n_planes, int b, int e,
                                   int c, const int (&head)[VW], int grp, bool on, int lane, float *sw, uint32_t *sx,
                                   float (&acc)[VW]) {
  constexpr int U = MODE == kScalar ? 8 : 4;  // edges a group has in flight
  const int step = MODE == kScalar ? U : a.EPW * U;
  const uint32_t pitch = static_cast<uint32_t>(a.ldx * sizeof(TX));
  using B = Batch<NR, NARROW>;
  constexpr int NH = MIX ? VW : 1;  // heads of a vector
  const float *swh[NH];
#pragma unroll
  for (int k = 0; k < NH; ++k) swh[k] = sw + head[k] * B::kPitch;
  B next;
  next.fetch(a, planes, n_planes, b, e, lane);
  for (int j0 = b; j0 < e; j0 += a.BE) {
    next.stage(lane, sw);
    const int x = next.x;
    if constexpr (MODE == kOffset) sx[lane] = static_cast<uint32_t>(x) * pitch;
    if constexpr (MODE == kLong) sx[lane] = x;
    wave_lds_order();
    if (j0 + a.BE < e) next.fetch(a, planes, n_planes, j0 + a.BE, e, lane);  // under way while this batch is summed
    const int n = min(a.BE, e - j0);
    for (int i0 = 0; i0 < n; i0 += step) {
      const int i = MODE == kScalar ? i0 : i0 + grp * U;
      if (on) {
        Raw<TX, VW> v[U];
        uint32_t rows[4] = {0, 0, 0, 0};
        if constexpr (MODE != kScalar) {
          const uint4 r = *reinterpret_cast<const uint4 *>(sx + i);
          rows[0] = r.x;
          rows[1] = r.y;
          rows[2] = r.z;
          rows[3] = r.w;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          // byte offsets of 32 bits on a scalar base; the row's own offset goes
          // to the base where a row is the wave's
          const char *base = reinterpret_cast<const char *>(X);
          uint32_t at = c * static_cast<uint32_t>(sizeof(TX));
          if constexpr (MODE == kScalar)
            base += scalar(static_cast<uint64_t>(static_cast<uint32_t>(__builtin_amdgcn_readlane(x, i + u))) * pitch);
          else if constexpr (MODE == kOffset)
            at += rows[u & 3];
          else
            base += static_cast<uint64_t>(rows[u & 3]) * pitch;
          v[u].ld(reinterpret_cast<const TX *>(base + at));
        }
        float w[U][NH];
#pragma unroll
        for (int k = 0; k < NH; ++k)
#pragma unroll
          for (int u = 0; u < U; u += 4) {
            const float4 f = *reinterpret_cast<const float4 *>(swh[k] + i + u);
            w[u][k] = f.x;
            w[u + 1][k] = f.y;
            w[u + 2][k] = f.z;
            w[u + 3][k] = f.w;
          }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          float r[VW];
          v[u].get(r);
#pragma unroll
          for (int k = 0; k < VW; ++k) {
            const float wk = w[u][MIX ? k : 0];
            acc[k] = fmaf(wk, SAFE && wk == 0.0f ? 0.0f : r[k], acc[k]);
          }
        }
      }
    }
    wave_lds_order();
  }
}

// Two sums of one launch: blocks from `split` (a multiple of 8) on take the
// second.
template <typename TX, typename TO> struct SumPair {
  SumArgs a[2];
  const TX *X[2];
  TO *out[2];
  unsigned split;
};

// out[r] = scale sum over the row's edges of w[e][head] X[col[e]].  One wave
// per (row or piece, slice of columns).
template <typename TX, typename TO, int VW, int MODE, int NR, bool NARROW, bool MIX>
__global__ void __launch_bounds__(kThreads) gather_sum_kernel(const SumPair<TX, TO> two) {
  __shared__ __align__(16) float sw[kWaves][Batch<NR, NARROW>::kFloats];
  __shared__ __align__(16) uint32_t sx[kWaves][kWave];
  const int which = blockIdx.x >= two.split ? 1 : 0;
  const SumArgs &a = two.a[which];
  const TX *__restrict__ X = two.X[which];
  TO *__restrict__ out = two.out[which];
  const Slot sl = slot_of(a.S, a.blocks, blockIdx.x - (which ? two.split : 0));
  const int slice = sl.slice, rb = sl.block;
  const int lane = threadIdx.x & (kWave - 1), wave = uniform(threadIdx.x >> 6);
  const int unit = a.unit0 + rb * kWaves + wave;
  const int nv = a.width / VW;
  if (unit >= a.units || slice * a.SV >= nv) return;
  int row, b, e;
  const int p = unit - a.n_rows;
  if (p < 0) {
    row = unit;
    row_bounds(a.ptr, row, a.E, &b, &e);
    if (e - b > a.T) return;
  } else {
    const Piece pc = find_piece(p, a.T, a.ptr, a.n_rows, a.E, [&](int pos) { return owner(a, pos); });
    if (pc.row < 0) return;
    row = pc.row;
    b = pc.begin;
    e = pc.end;
  }
  b = uniform(b);
  e = uniform(e);
  const int grp = MODE == kScalar ? 0 : lane / a.SV, gl = lane - grp * a.SV;
  const int vj = slice * a.SV + gl;
  const bool on = gl < a.SV && grp < a.EPW && vj < nv;
  const int c = (on ? vj : nv - 1) * VW;
  // heads are counted from the first that the slice meets
  const int first = a.width == a.C ? slice * a.SV * VW / a.Ch : 0;
  int head[VW];
#pragma unroll
  for (int k = 0; k < VW; ++k) head[k] = ((c + k) % a.C) / a.Ch - first;
  const float *planes = a.w + first * a.ldw;
  const int n_planes = min(a.planes, a.H - first);
  float acc[VW];
#pragma unroll
  for (int k = 0; k < VW; ++k) acc[k] = 0.0f;
  gather_rows<TX, VW, MODE, NR, NARROW, MIX, false>(a, X, planes, n_planes, b, e, c, head, grp, on, lane, sw[wave],
                                                    sx[wave], acc);
  // A sum that is finite had no infinity or NaN in it, so its weights of 0
  // added 0.  One that is not is taken again with those edges left out.
  bool odd = false;
#pragma unroll
  for (int k = 0; k < VW; ++k) odd = odd || !(fabsf(acc[k]) < INFINITY);
  if (__any(odd)) {
#pragma unroll
    for (int k = 0; k < VW; ++k) acc[k] = 0.0f;
    gather_rows<TX, VW, MODE, NR, NARROW, MIX, true>(a, X, planes, n_planes, b, e, c, head, grp, on, lane, sw[wave],
                                                     sx[wave], acc);
  }
  if constexpr (MODE != kScalar) {
    float sum[VW];
#pragma unroll
    for (int k = 0; k < VW; ++k) sum[k] = acc[k];
    for (int g = 1; g < a.EPW; ++g)
#pragma unroll
      for (int k = 0; k < VW; ++k) sum[k] += __shfl(acc[k], (gl + g * a.SV) & (kWave - 1));
#pragma unroll
    for (int k = 0; k < VW; ++k) acc[k] = sum[k];
  }
  if (!on || grp != 0) return;
  if (p >= 0) {
    Vec<float, VW>::st(a.part + static_cast<int64_t>(p) * a.width + c, acc);
    return;
  }
#pragma unroll
  for (int k = 0; k < VW; ++k) acc[k] *= a.scale;
  Vec<TO, VW>::st(out + static_cast<int64_t>(row) * a.width + c, acc);
}

// Sums whose pieces one launch joins, (group of rows, 64 columns) a block.
template <typename TO> struct Joins {
  SumArgs a[3];
  TO *out[3];
  int64_t begin[4] = {0, 0, 0, 0};  // first block of each; the end is begin[3]
  int n = 0;
};

// Rows that a block of long_sum_kernel looks through: about 128 groups.
__host__ __device__ inline int join_rows(int n_rows) { return n_rows < 256 ? 1 : n_rows < 8192 ? n_rows >> 7 : 64; }

// Long rows: the pieces' sums added in a fixed order, a wave a quarter of the
// pieces.  Mostly there are none, so what counts is finding that out: one
// round of loads for a group of rows, and one launch for the backward's three
// sums (3,000 rows: 5 us each by windows and apart, 15 by windows together, 5
// us this way).
template <typename TO>
__global__ void __launch_bounds__(kThreads) long_sum_kernel(const Joins<TO> js) {
  __shared__ float red[kWaves][kWave];
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x >> 6;
  for (int64_t block = blockIdx.x; block < js.begin[3]; block += gridDim.x) {
    const int which = block < js.begin[1] ? 0 : block < js.begin[2] ? 1 : 2;
    const SumArgs &a = js.a[which];
    const int columns = (a.width + kWave - 1) / kWave, group = static_cast<int>((block - js.begin[which]) / columns);
    const int c = static_cast<int>((block - js.begin[which]) % columns) * kWave + lane, cc = min(c, a.width - 1);
    const int R = join_rows(a.n_rows), row0 = group * R;
    int b = 0, e = 0;
    if (lane < R && row0 + lane < a.n_rows) row_bounds(a.ptr, row0 + lane, a.E, &b, &e);
    for (uint64_t left = __ballot(e - b > a.T); left; left &= left - 1) {
      const int i = __ffsll(static_cast<unsigned long long>(left)) - 1;
      const int first = __shfl(b, i), n = piece_count(first, __shfl(e, i), a.T);
      const int upto = static_cast<int>(static_cast<int64_t>(n) * (wave + 1) / kWaves);
      float s = 0.0f;
      for (int i0 = static_cast<int>(static_cast<int64_t>(n) * wave / kWaves); i0 < upto; i0 += 8) {
        float v[8];
#pragma unroll
        for (int u = 0; u < 8; ++u)
          v[u] = a.part[static_cast<int64_t>(piece_id(first, a.T, min(i0 + u, n - 1))) * a.width + cc];
#pragma unroll
        for (int u = 0; u < 8; ++u) s += i0 + u < upto ? v[u] : 0.0f;
      }
      __syncthreads();  // the last row's sums are no longer read
      red[wave][lane] = s;
      __syncthreads();
      if (wave != 0 || c >= a.width) continue;
#pragma unroll
      for (int w = 1; w < kWaves; ++w) s += red[w][lane];
      Store<TO>::st(js.out[which] + static_cast<int64_t>(row0 + i) * a.width + c, s * a.scale);
    }
  }
}

// ---------------------------------------------------------------------- host

struct Shape {
  int lmax, K, C, H, D, storage;
  int64_t ldq, ldk, ldv;
  int n_dst, n_src, E;
  float scale;
  int t;         // dropout threshold
  int T, TP;     // edges in a products block's LDS at a time; of a row one block takes
  int64_t pieces;
};

// Edges beyond which a row is cut into pieces, for `units` waves over n_rows
// rows.  Enough units fill the chip by themselves, and a piece costs one that
// mostly finds nothing to do; with fewer, rows of up to twice the mean and 512
// stay whole (488 rows of 765 edges, 16 heads: logits and weights 159 us whole,
// 141 cut); with few, rows are cut into about 2,048 pieces of 64 edges or more
// (one row over 8,064 atoms: logits 20 us at 256, 9 at 64).  A small graph of
// ordinary rows is not cut at all: that saves the launches that join pieces
// (64 atoms, 2,900 edges, forward: 26 us in four launches, 18 in two).
int piece_edges(int64_t units, int n_rows, int E) {
  if (E <= 4096 && E <= static_cast<int64_t>(128) * n_rows) return E > 0 ? E : 1;
  if (units >= 4096) return 4096;
  int64_t T = E / 2048;
  if (units >= 1024) T = std::max(T, std::min<int64_t>(static_cast<int64_t>(E) / n_rows * 2, 512));
  return static_cast<int>(std::min<int64_t>(std::max<int64_t>((T + 63) & ~int64_t(63), 64), 4096));
}

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
  EGNN_REQUIRE(s->ldq <= kMaxStride && s->ldk <= kMaxStride && s->ldv <= kMaxStride,
               "row strides are at most 2^29 elements");
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
  s->TP = piece_edges(static_cast<int64_t>(s->n_dst) * kWaves, s->n_dst, s->E);
  s->pieces = s->E > s->TP ? 2 * ((static_cast<int64_t>(s->E) + s->TP - 1) / s->TP) : 0;
  return EGNN_OK;
}

struct SumPlan {
  int S, SV, EPW, T;
  int64_t pieces;
};

// Slices and piece length of a weighted sum over rows of X of `nv` vectors of
// `bytes` each.
SumPlan sum_plan(int n_rows, int n_x, int E, int nv, int bytes) {
  SumPlan p;
  if (nv <= kWave) {
    // one slice, whatever X is: eight of a line each took 103 us where one takes
    // 81 (rows of 1 KB, 8 MB of them, 1.1 M edges)
    p.S = 1;
    p.SV = nv;
  } else {
    // slices in eights, one XCD each, in whole lookups (four vectors)
    p.S = 8 * ((nv + 8 * kWave - 1) / (8 * kWave));
    while ((p.SV = ((nv + p.S - 1) / p.S + 3) & ~3) > kWave) p.S += 8;
    // Where an XCD's L2 (4 MB) does not hold its slice of X, narrower ones in
    // whole lines (eight vectors) that it does hold: of 48, 32, 24 and 16 the
    // first that fills most lanes (64, 64, 48, 64 of 64) and whose number is
    // one that slot_of spreads evenly.
    if (static_cast<int64_t>(n_x) * p.SV * bytes > kSliceBytes) {
      for (const int SV : {32, 16, 48, 24}) {
        const int used = (nv + SV - 1) / SV, r = used & 7;
        if (SV >= p.SV || static_cast<int64_t>(n_x) * SV * bytes > kSliceBytes || (r & (r - 1)) != 0) continue;
        p.SV = SV;
        p.S = used;
        break;
      }
    }
  }
  p.EPW = kWave / p.SV < 16 ? kWave / p.SV : 16;
  p.T = piece_edges(static_cast<int64_t>(n_rows) * p.S, n_rows, E);
  p.pieces = E > p.T ? 2 * ((static_cast<int64_t>(E) + p.T - 1) / p.T) : 0;
  return p;
}

// Parts of a row's edges in the dot products with v: in eights, so that an
// XCD's part of v fits its L2; one where that leaves too few edges a part to
// pay for reading the row of grad_out again (8), or where rows are short.
// (Rows of 6.4 KB, 181 edges a row, 19 MB of v: 1, 8, 16, 24 parts 374, 153,
// 166, 180 us; 138 edges a row, 52 MB: 879, 532, 477, 529.)
int dot_parts(const Shape &s, int bytes) {
  const int64_t deg = s.E / (s.n_dst > 0 ? s.n_dst : 1);
  const int64_t v = static_cast<int64_t>(s.n_src) * s.K * s.C * bytes;
  const int64_t parts = 8 * ((v + 8 * kPartBytes - 1) / (8 * kPartBytes));
  if (parts * 8 > deg) return deg >= 32 && s.n_dst < 1024 ? 8 : 1;
  // few rows: more parts, down to 8 edges each, until waves fill the chip
  int64_t n = parts;
  while (n * s.n_dst < 8192 && (n + 8) * 8 <= deg && n < 64) n += 8;
  return static_cast<int>(n);
}

size_t align256(size_t n) { return (n + 255) & ~size_t(255); }

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// Elements of the widest load (16 or 8 bytes, or one element) that lies in one
// head and one row and is aligned.
template <typename T> int vec_width(int Ch, int64_t ld, const void *p) {
  for (int V = 16 / sizeof(T); V * sizeof(T) >= 8; V /= 2)
    if (Ch % V == 0 && ld % V == 0 && reinterpret_cast<uintptr_t>(p) % (V * sizeof(T)) == 0) return V;
  return 1;
}

struct Saved {
  float2 *maps;
  int *dst;
};

int64_t plane(const Shape &s) { return (static_cast<int64_t>(s.E) + 63) & ~int64_t(63); }

size_t saved_bytes_of(const Shape &s) {
  const size_t E = s.E, H = s.H;
  return align256(E * 2 * H * 4) + align256(E * 4);
}

Saved carve_saved(const Shape &s, char *p) {
  const size_t E = s.E, H = s.H;
  Saved v;
  v.maps = reinterpret_cast<float2 *>(p);
  p += align256(E * 2 * H * 4);
  v.dst = reinterpret_cast<int *>(p);
  return v;
}

// Pieces of a sum's partial rows: the most any vector width may ask for.
size_t sum_part_bytes(int n_rows, int n_x, int E, int width) {
  size_t most = 0;
  const int sizes[4][2] = {{1, 2}, {1, 4}, {4, 16}, {8, 16}};  // elements and bytes of a vector
  for (const auto &z : sizes) {
    const SumPlan p = sum_plan(n_rows, n_x, E, (width + z[0] - 1) / z[0], z[1]);
    const size_t n = align256(static_cast<size_t>(p.pieces) * width * 4);
    if (n > most) most = n;
  }
  return most;
}

size_t ws_fwd_of(const Shape &s, bool train) {
  return (train ? 0 : saved_bytes_of(s)) + align256(plane(s) * s.H * 4) +
         align256(static_cast<size_t>(s.pieces) * 2 * s.H * 8) + sum_part_bytes(s.n_dst, s.n_src, s.E, s.K * s.C);
}

size_t ws_bwd_of(const Shape &s) {
  const size_t E = s.E, H = s.H, P = plane(s);
  const size_t part = sum_part_bytes(s.n_dst, s.n_src, s.E, 2 * s.H * s.D) +
                      sum_part_bytes(s.n_src, s.n_dst, s.E, 2 * s.H * s.D) +
                      sum_part_bytes(s.n_src, s.n_dst, s.E, s.K * s.C);
  return align256(E * 2 * H * 4) + 2 * align256(E * H * 4) + 2 * align256(P * 2 * H * 4) + align256(P * H * 4) +
         align256(E * 4) + align256(static_cast<size_t>(s.n_dst) * H * 4) +
         align256(static_cast<size_t>(s.pieces) * H * 8) + part;
}

template <typename TX, typename TO, int VW, int NR, bool NARROW, bool MIX>
void launch_sum(unsigned grid, int mode, hipStream_t st, const SumPair<TX, TO> &two) {
  if (mode == kScalar) gather_sum_kernel<TX, TO, VW, kScalar, NR, NARROW, MIX><<<grid, kThreads, 0, st>>>(two);
  else if (mode == kOffset) gather_sum_kernel<TX, TO, VW, kOffset, NR, NARROW, MIX><<<grid, kThreads, 0, st>>>(two);
  else gather_sum_kernel<TX, TO, VW, kLong, NR, NARROW, MIX><<<grid, kThreads, 0, st>>>(two);
}

// What picks the kernel of a sum.
struct SumKind {
  int vw, mode;
  bool mix, narrow, few;  // few: at most 8 planes
  int64_t pieces;
  bool operator==(const SumKind &o) const {
    return vw == o.vw && mode == o.mode && mix == o.mix && narrow == o.narrow && few == o.few;
  }
};

// Completes the arguments of a sum (slices, staging, pieces).
template <typename TX, typename TO> SumKind plan_sum(SumArgs &a, const TX *X, const TO *out) {
  SumKind k;
  // 16-byte vectors of a row; one may hold elements of several heads (mix)
  constexpr int V = 16 / sizeof(TX);
  k.vw = a.width % V == 0 && a.ldx % V == 0 && aligned16(X) && aligned16(out) ? V : 1;
  const SumPlan p = sum_plan(a.n_rows, a.n_x, a.E, a.width / k.vw, k.vw * static_cast<int>(sizeof(TX)));
  a.S = p.S;
  a.SV = p.SV;
  a.EPW = p.EPW;
  a.T = p.T;
  a.planes = a.H;
  if (a.width == a.C && a.S > 1) {
    a.planes = 1;
    for (int i = 0; i < a.S; ++i) {
      const int c0 = i * a.SV * k.vw, c1 = std::min((i + 1) * a.SV * k.vw, a.width);
      if (c0 < c1) a.planes = std::max(a.planes, (c1 - 1) / a.Ch - c0 / a.Ch + 1);
    }
  }
  // whole rounds of the edges in flight
  const int round = p.EPW == 1 ? 8 : 4 * p.EPW, stage = a.planes <= 16 ? kWave : 16;
  if (round > stage) a.EPW = stage / 4;
  a.BE = stage / (a.EPW == 1 ? 8 : 4 * a.EPW) * (a.EPW == 1 ? 8 : 4 * a.EPW);
  k.mode = a.EPW == 1                                                                     ? kScalar
           : static_cast<uint64_t>(a.n_x) * a.ldx * sizeof(TX) < (uint64_t(1) << 32) ? kOffset
                                                                                     : kLong;
  a.units = static_cast<int>(a.n_rows + p.pieces);
  a.unit0 = 0;
  a.blocks = (a.units + kWaves - 1) / kWaves;
  k.mix = k.vw > 1 && a.Ch % V != 0;
  k.narrow = a.planes > 16;
  k.few = a.planes <= 8;  // registers for the next edges' weights: as few as the heads allow
  k.pieces = p.pieces;
  return k;
}

template <typename TX, typename TO>
egnn_status launch_kind(const SumKind &k, unsigned grid, const SumPair<TX, TO> &two, hipStream_t st) {
  constexpr int V = 16 / sizeof(TX);
  if (k.mix && !k.narrow) launch_sum<TX, TO, V, 16, false, true>(grid, k.mode, st, two);
  else if (k.mix) launch_sum<TX, TO, V, 16, true, true>(grid, k.mode, st, two);
  else if (k.vw > 1 && k.few) launch_sum<TX, TO, V, 8, false, false>(grid, k.mode, st, two);
  else if (k.vw > 1 && !k.narrow) launch_sum<TX, TO, V, 16, false, false>(grid, k.mode, st, two);
  else if (k.vw > 1) launch_sum<TX, TO, V, 16, true, false>(grid, k.mode, st, two);
  else if (!k.narrow) launch_sum<TX, TO, 1, 16, false, false>(grid, k.mode, st, two);
  else launch_sum<TX, TO, 1, 16, true, false>(grid, k.mode, st, two);
  EGNN_CHECK_LAUNCH();
  return EGNN_OK;
}

template <typename TX, typename TO> double sum_bytes(const SumArgs &a) {
  return static_cast<double>(a.E) * (4.0 * a.H + 4) + static_cast<double>(a.n_x) * a.width * sizeof(TX) +
         static_cast<double>(a.n_rows) * a.width * sizeof(TO);
}

// A planned sum's pieces are joined once the others of js are launched, too.
template <typename TO> void add_join(Joins<TO> &js, const SumKind &k, const SumArgs &a, TO *out) {
  if (!k.pieces) return;
  js.a[js.n] = a;
  js.out[js.n] = out;
  const int64_t end = js.begin[js.n] + static_cast<int64_t>(ceil_div(a.n_rows, join_rows(a.n_rows))) * ceil_div(a.width, kWave);
  for (int i = ++js.n; i < 4; ++i) js.begin[i] = end;
}

template <typename TO> egnn_status join_pieces(const Joins<TO> &js, hipStream_t st) {
  if (!js.n) return EGNN_OK;
  Timed t(st, "attn_long_sum", 0.0, 0.0);
  long_sum_kernel<TO><<<static_cast<unsigned>(std::min<int64_t>(js.begin[3], kMaxBlocks)), kThreads, 0, st>>>(js);
  EGNN_CHECK_LAUNCH();
  return EGNN_OK;
}

template <typename TX, typename TO>
egnn_status run_sum(SumArgs a, const TX *X, TO *out, const char *name, Joins<TO> &js, hipStream_t st) {
  if (a.n_rows == 0) return EGNN_OK;
  const SumKind k = plan_sum(a, X, out);
  add_join(js, k, a, out);
  const int most = kMaxBlocks / a.S;  // blocks a slice in one launch
  for (; a.unit0 < a.units; a.unit0 += most * kWaves) {
    Timed t(st, name, a.unit0 ? 0.0 : 2.0 * a.E * a.width, a.unit0 ? 0.0 : sum_bytes<TX, TO>(a));
    a.blocks = std::min((a.units - a.unit0 + kWaves - 1) / kWaves, most);
    const unsigned grid = static_cast<unsigned>(a.blocks) * a.S;
    const egnn_status r = launch_kind<TX, TO>(k, grid, SumPair<TX, TO>{{a, a}, {X, X}, {out, out}, grid}, st);
    if (r != EGNN_OK) return r;
  }
  return EGNN_OK;
}

// Two sums that need one kind of kernel share a launch (each has its own part
// of the workspace for its pieces).
template <typename TX, typename TO>
egnn_status run_two_sums(SumArgs a, const TX *Xa, TO *outa, const char *na, SumArgs b, const TX *Xb, TO *outb,
                         const char *nb, const char *both, Joins<TO> &js, hipStream_t st) {
  SumArgs a2 = a, b2 = b;
  if (a.n_rows > 0 && b.n_rows > 0) {
    const SumKind ka = plan_sum(a2, Xa, outa), kb = plan_sum(b2, Xb, outb);
    const int64_t ga = (static_cast<int64_t>(a2.blocks) * a2.S + 7) & ~int64_t(7);
    const int64_t gb = static_cast<int64_t>(b2.blocks) * b2.S;
    // (rows of 1 KB: 3 MB of each, 0.54 M edges, 71 us apart and 61 together;
    // 8 MB of each, 1.1 M edges, 171 and 191: their L2 lines displace each other)
    const int64_t bytes = (static_cast<int64_t>(a.n_x) * a.width + static_cast<int64_t>(b.n_x) * b.width) *
                          static_cast<int64_t>(sizeof(TX));
    if (ka == kb && ga + gb <= kMaxBlocks && bytes <= kPairBytes) {
      add_join(js, ka, a2, outa);
      add_join(js, kb, b2, outb);
      Timed t(st, both, 2.0 * a.E * (a.width + b.width), sum_bytes<TX, TO>(a2) + sum_bytes<TX, TO>(b2));
      return launch_kind<TX, TO>(ka, static_cast<unsigned>(ga + gb),
                                 SumPair<TX, TO>{{a2, b2}, {Xa, Xb}, {outa, outb}, static_cast<unsigned>(ga)}, st);
    }
  }
  const egnn_status r = run_sum<TX, TO>(a, Xa, outa, na, js, st);
  return r != EGNN_OK ? r : run_sum<TX, TO>(b, Xb, outb, nb, js, st);
}

template <typename T, int VW, bool ONE, int NIT = kMaxNit>
void launch_logits(unsigned grid, size_t lds, hipStream_t st, const LogitArgs &a, const T *q, const T *k) {
  if constexpr (NIT > 1)
    if (a.team.nit < NIT) return launch_logits<T, VW, ONE, NIT - 1>(grid, lds, st, a, q, k);
  logits_kernel<T, VW, NIT, ONE><<<grid, kThreads, lds, st>>>(a, q, k);
}

template <typename T, int VW, bool ONE, int NIT = kMaxNit>
void launch_dots(unsigned grid, hipStream_t st, const DotArgs &a, const float *go, const T *v) {
  if constexpr (NIT > 1)
    if (a.team.nit < NIT) return launch_dots<T, VW, ONE, NIT - 1>(grid, st, a, go, v);
  value_dots_kernel<T, VW, NIT, ONE><<<grid, kThreads, 0, st>>>(a, go, v);
}

template <typename T>
egnn_status forward(const Shape &s, const egnn_graph *g, const T *q, const T *k, const T *v, const float *lam,
                    const float *bias, const uint8_t *mask, const uint64_t *rng, uint32_t site, T *out, void *saved,
                    char *ws, hipStream_t st) {
  const bool train = saved != nullptr;
  const Saved sv = carve_saved(s, train ? static_cast<char *>(saved) : ws);
  if (!train) ws += saved_bytes_of(s);
  auto *w = reinterpret_cast<float *>(ws);
  ws += align256(plane(s) * s.H * 4);
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
  a.TP = s.TP;
  a.H = s.H;
  a.D = s.D;
  a.ldq = s.ldq;
  a.ldk = s.ldk;
  a.scale = s.scale;
  a.bias = bias;
  a.mask = mask;
  a.lam = lam;
  a.drop = make_drop(rng, site, s.t);
  a.maps = sv.maps;
  a.keep = train;
  a.w = w;
  a.ldw = plane(s);
  a.dst = sv.dst;
  a.piece_stats = piece_stats;
  if (s.E > 0) {
    constexpr int V = 16 / sizeof(T);
    const int vw = std::min(vec_width<T>(s.D, s.ldq, q), vec_width<T>(s.D, s.ldk, k));
    a.team = make_team(1, 2 * s.H, s.D / vw);
    a.Hpl = log2_ceil(2 * s.H);
    const unsigned grid = static_cast<unsigned>(s.n_dst + s.pieces);
    const size_t lds = static_cast<size_t>(s.T) * (2 * s.H + 2) * 4;
    {
      Timed t(st, "attn_logits", 4.0 * s.E * s.H * s.D,
              static_cast<double>(s.E) * (12.0 * s.H + 8 + (bias ? 8.0 * s.H : 0)) +
                  2.0 * s.H * s.D * sizeof(T) * (static_cast<double>(s.n_dst) + s.n_src));
      const bool one = a.team.esh == 6;
      if (vw == V && one) launch_logits<T, V, true>(grid, lds, st, a, q, k);
      else if (vw == V) launch_logits<T, V, false>(grid, lds, st, a, q, k);
      else if (vw > 1) launch_logits<T, V / 2, false>(grid, lds, st, a, q, k);
      else launch_logits<T, 1, false>(grid, lds, st, a, q, k);
      EGNN_CHECK_LAUNCH();
    }
    if (s.pieces) {
      Timed t(st, "attn_long_weights", 0.0, 0.0);
      long_weights_kernel<<<static_cast<unsigned>(s.pieces), kThreads, static_cast<size_t>(s.T) * (s.H + 1) * 4, st>>>(a);
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
  m.w = w;
  m.ldw = plane(s);
  m.H = s.H;
  m.C = s.C;
  m.Ch = s.C / s.H;
  m.width = s.K * s.C;
  m.scale = 1.0f;
  m.part = reinterpret_cast<float *>(ws);
  Joins<T> js;
  const egnn_status r = run_sum<T, T>(m, v, out, "attn_out", js, st);
  return r != EGNN_OK ? r : join_pieces(js, st);
}

template <typename T>
egnn_status backward(const Shape &s, const egnn_graph *g, const T *q, const T *k, const T *v, const float *lam,
                     const uint64_t *rng, uint32_t site, const void *saved, const float *go, float *gq, float *gk,
                     float *gv, float *glam, float *gbias, char *ws, hipStream_t st) {
  const Saved sv = carve_saved(s, static_cast<char *>(const_cast<void *>(saved)));
  const size_t E = s.E, H = s.H, P = plane(s);
  const auto take = [&ws](size_t bytes) {
    char *p = ws;
    ws += align256(bytes);
    return p;
  };
  auto *dl_rows = reinterpret_cast<float *>(take(E * 2 * H * 4));
  float *dl = gbias ? gbias : dl_rows;
  auto *u = reinterpret_cast<float *>(take(E * H * 4));
  auto *wr = reinterpret_cast<float *>(take(E * H * 4));
  auto *dlp = reinterpret_cast<float *>(take(P * 2 * H * 4));       // planes, by destination
  auto *dlp_src = reinterpret_cast<float *>(take(P * 2 * H * 4));   // planes, by source
  auto *w_src = reinterpret_cast<float *>(take(P * H * 4));
  auto *dst_src = reinterpret_cast<int *>(take(E * 4));
  auto *t1 = reinterpret_cast<float *>(take(static_cast<size_t>(s.n_dst) * H * 4));
  auto *piece_t = reinterpret_cast<float2 *>(take(static_cast<size_t>(s.pieces) * H * 8));
  auto *part = reinterpret_cast<float *>(ws);
  constexpr int V = 16 / sizeof(T);
  const int Ch = s.C / s.H;
  if (s.E > 0) {
    DotArgs a{};
    a.row_ptr = g->row_ptr;
    a.src = g->src;
    a.dst = sv.dst;
    a.n_dst = s.n_dst;
    a.n_src = s.n_src;
    a.E = s.E;
    a.H = s.H;
    a.C = s.C;
    a.K = s.K;
    a.ldv = s.ldv;
    a.u = u;
    const int vw = std::min(vec_width<T>(Ch, s.ldv, v), aligned16(go) ? V : 1);
    a.team = make_team(s.K, s.H, Ch / vw);
    a.parts = dot_parts(s, sizeof(T));
    a.T = piece_edges(static_cast<int64_t>(s.n_dst) * a.parts, s.n_dst, s.E);
    const int64_t pieces = s.E > a.T ? 2 * ((static_cast<int64_t>(s.E) + a.T - 1) / a.T) : 0;
    a.units = static_cast<int>(s.n_dst + pieces);
    const int most = kMaxBlocks / a.parts;
    for (a.unit0 = 0; a.unit0 < a.units; a.unit0 += most * kWaves) {
      Timed t(st, "attn_value_dots", a.unit0 ? 0.0 : 2.0 * s.E * s.K * s.C,
              a.unit0 ? 0.0
                      : static_cast<double>(s.E) * (4.0 * s.H + 4) +
                            static_cast<double>(s.K) * s.C * (4.0 * s.n_dst + sizeof(T) * static_cast<double>(s.n_src)));
      const int left = (a.units - a.unit0 + kWaves - 1) / kWaves;
      a.blocks = left < most ? left : most;
      const unsigned grid = static_cast<unsigned>(a.blocks) * a.parts;
      const bool one = a.team.esh == 6;
      if (vw == V && one) launch_dots<T, V, true>(grid, st, a, go, v);
      else if (vw == V) launch_dots<T, V, false>(grid, st, a, go, v);
      else if (vw > 1 && one) launch_dots<T, V / 2, true>(grid, st, a, go, v);
      else if (vw > 1) launch_dots<T, V / 2, false>(grid, st, a, go, v);
      else launch_dots<T, 1, false>(grid, st, a, go, v);
      EGNN_CHECK_LAUNCH();
    }
  }
  if (s.n_dst > 0) {
    GradArgs a{};
    a.row_ptr = g->row_ptr;
    a.dst = sv.dst;
    a.n_dst = s.n_dst;
    a.E = s.E;
    a.T = s.T;
    a.TP = s.TP;
    a.H = s.H;
    a.Hpl = log2_ceil(s.H);
    a.lam = lam;
    a.drop = make_drop(rng, site, s.t);
    a.maps = sv.maps;
    a.dl = reinterpret_cast<float2 *>(dl);
    a.dlp = dlp;
    a.ldw = plane(s);
    a.wr = wr;
    a.t1 = t1;
    a.u = u;
    a.piece_t = piece_t;
    const size_t lds = static_cast<size_t>(s.T) * ((3 * s.H + 1) * 4 + s.H);
    {
      Timed t(st, "attn_logit_grad", 0.0, static_cast<double>(s.E) * 36.0 * s.H);
      logit_grad_kernel<<<static_cast<unsigned>(s.n_dst + s.pieces), kThreads, lds, st>>>(a);
      EGNN_CHECK_LAUNCH();
    }
    if (s.pieces) {
      Timed t(st, "attn_long_grad", 0.0, 0.0);
      long_grad_kernel<<<static_cast<unsigned>(s.pieces), kThreads, lds, st>>>(a);
      EGNN_CHECK_LAUNCH();
    }
  }
  {
    Timed t(st, "attn_regroup", 0.0, static_cast<double>(s.E) * (24.0 * s.H + 12));
    const unsigned grid = ceil_div(s.E, kThreads) + s.H;
    const auto kernel = s.H % 4 == 0 && aligned16(dl) ? regroup_kernel<true> : regroup_kernel<false>;
    kernel<<<grid, kThreads, 0, st>>>(g->src_perm, g->src_ptr, s.n_src, s.E, s.H, sv.dst, wr, dl, plane(s), dst_src,
                                      w_src, dlp_src, t1, s.n_dst, glam);
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
  m.w = dlp;
  m.ldw = plane(s);
  m.H = 2 * s.H;
  m.C = 2 * s.H * s.D;
  m.Ch = s.D;
  m.width = 2 * s.H * s.D;
  m.scale = s.scale;
  m.part = part;
  const SumArgs to_q = m;
  m.ptr = g->src_ptr;
  m.col = dst_src;
  m.row_of = g->src;
  m.perm = g->src_perm;
  m.n_rows = s.n_src;
  m.n_x = s.n_dst;
  m.ldx = s.ldq;
  m.w = dlp_src;
  part += sum_part_bytes(s.n_dst, s.n_src, s.E, m.width) / 4;
  m.part = part;
  part += sum_part_bytes(s.n_src, s.n_dst, s.E, m.width) / 4;
  Joins<float> js;
  egnn_status r =
      run_two_sums<T, float>(to_q, k, gq, "attn_grad_q", m, q, gk, "attn_grad_k", "attn_grad_qk", js, st);
  if (r != EGNN_OK) return r;
  m.part = part;
  m.ldx = static_cast<int64_t>(s.K) * s.C;
  m.w = w_src;
  m.H = s.H;
  m.C = s.C;
  m.Ch = Ch;
  m.width = s.K * s.C;
  m.scale = 1.0f;
  r = run_sum<float, float>(m, go, gv, "attn_grad_v", js, st);
  return r != EGNN_OK ? r : join_pieces(js, st);
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
