// Dropout of irreps with a mask that is never stored (see egnn.h).
//
//   y = residual + m x,  m in {0, 65536/(65536-t)} per decision
//
// A decision is shared by the 2l+1 components that a rotation mixes (or by all
// components, or by the row), so the operator commutes with rotations.  The
// backward draws the same decisions again from (seed, step, site).
//
// Bound: HBM traffic, one read of each input and one write.  A thread owns one
// group of eight channels (one 16-byte load in bf16, two in fp32), which is
// one generator call, and walks KC consecutive components with it, so the
// rounds' integer products are spread over KC vectors.  Edge embeddings
// (544,000 rows of 25 x 64, bf16, with residual): 960 us, 5.4 TB/s, vector
// units busy 40%; node irreps (8,064 rows of 25 x 128, likewise): 27 us.
#include <cmath>

#include "common.h"
#include "philox.h"
#include "timing.h"

using namespace egnn;

namespace {

constexpr int kThreads = 256;
constexpr int64_t kMaxThreads = int64_t(1) << 30;  // per launch: 32-bit index arithmetic in the kernels

struct DropShape {
  int K, C, L;      // components, channels, lmax
  int share;        // egnn_drop_share
  int KP;           // parts of the component axis (K = KP * KC)
};

template <typename T> struct Eight;
template <> struct Eight<float> {
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
template <> struct Eight<uint16_t> {
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

__device__ inline int degree_of(int k) {  // floor(sqrt(k)) for k < 81
  int l = 0;
  while ((l + 1) * (l + 1) <= k) ++l;
  return l;
}

// Keep factors of the eight channels at c0 of (row, degree l).  C is a
// multiple of 8 here, so the eight decisions are one generator call.
__device__ inline void factors8(const DropShape &s, const Drop &d, const DropKey &key, int64_t row, int l, int c0,
                                float (&m)[8]) {
  if (s.share == EGNN_DROP_ROW) {
    const float f = drop_one(row, d, key);
#pragma unroll
    for (int u = 0; u < 8; ++u) m[u] = f;
    return;
  }
  const int64_t base = s.share == EGNN_DROP_DEGREE ? (row * (s.L + 1) + l) * s.C + c0 : row * s.C + c0;
  const uint4 w = philox4x32(static_cast<uint64_t>(base) >> 3, key);
#pragma unroll
  for (int u = 0; u < 8; ++u) m[u] = drop_draw(w, u) >= d.t ? d.factor : 0.0f;
}

// A dropped element is the residual (or 0) whatever x holds there, so that an
// infinity or NaN in a dropped place does not come through.
__device__ inline float apply(float m, float x, float r) { return m == 0.0f ? r : r + m * x; }

// One thread: eight channels of KC consecutive components of one row.  Lanes
// run over channel groups first, so a group of lanes streams consecutive lines.
template <typename T, int KC, bool RES>
__global__ void __launch_bounds__(kThreads) dropout_vec_kernel(DropShape s, Drop d, int64_t row0, uint32_t n_threads,
                                                               const T *x, const T *res, T *y) {
  const uint32_t i = blockIdx.x * kThreads + threadIdx.x;
  if (i >= n_threads) return;
  const uint32_t CG = static_cast<uint32_t>(s.C) >> 3;
  const uint32_t g = i % CG, q = i / CG;
  const uint32_t kp = q % static_cast<uint32_t>(s.KP);
  const int64_t row = row0 + q / static_cast<uint32_t>(s.KP);
  const int k0 = static_cast<int>(kp) * KC;
  const int64_t at = (row * s.K + k0) * s.C + static_cast<int64_t>(g) * 8;
  float v[KC][8], r[KC][8];
#pragma unroll
  for (int j = 0; j < KC; ++j) Eight<T>::ld(x + at + static_cast<int64_t>(j) * s.C, v[j]);
  if constexpr (RES) {
#pragma unroll
    for (int j = 0; j < KC; ++j) Eight<T>::ld(res + at + static_cast<int64_t>(j) * s.C, r[j]);
  }
  float m[8];
  const bool every = d.t == 0;
  DropKey key{};
  if (every) {
#pragma unroll
    for (int u = 0; u < 8; ++u) m[u] = 1.0f;
  } else {
    key = drop_key(d);
  }
  int l = degree_of(k0);
  bool fresh = true;
#pragma unroll
  for (int j = 0; j < KC; ++j) {
    const int k = k0 + j;
    if (k >= (l + 1) * (l + 1)) {
      ++l;
      fresh = fresh || s.share == EGNN_DROP_DEGREE;
    }
    if (fresh && !every) factors8(s, d, key, row, l, static_cast<int>(g) * 8, m);
    fresh = false;
    float o[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) o[u] = apply(m[u], v[j][u], RES ? r[j][u] : 0.0f);
    Eight<T>::st(y + at + static_cast<int64_t>(j) * s.C, o);
  }
}

// Invariants (one component) with a decision per element: the decisions run
// over the flat array, so groups of eight need no channel count that fits.
template <typename T, bool RES>
__global__ void __launch_bounds__(kThreads) dropout_flat_kernel(Drop d, int64_t group0, uint32_t n_groups, int64_t n,
                                                                const T *x, const T *res, T *y) {
  const uint32_t i = blockIdx.x * kThreads + threadIdx.x;
  if (i >= n_groups) return;
  const int64_t j = group0 + i, at = j * 8;
  float m[8];
  if (d.t == 0) {
#pragma unroll
    for (int u = 0; u < 8; ++u) m[u] = 1.0f;
  } else {
    const uint4 w = philox4x32(static_cast<uint64_t>(j), drop_key(d));
#pragma unroll
    for (int u = 0; u < 8; ++u) m[u] = drop_draw(w, u) >= d.t ? d.factor : 0.0f;
  }
  if (at + 8 <= n) {
    float v[8], r[8], o[8];
    Eight<T>::ld(x + at, v);
    if constexpr (RES) Eight<T>::ld(res + at, r);
#pragma unroll
    for (int u = 0; u < 8; ++u) o[u] = apply(m[u], v[u], RES ? r[u] : 0.0f);
    Eight<T>::st(y + at, o);
  } else {
#pragma unroll
    for (int u = 0; u < 8; ++u)
      if (at + u < n)
        Store<T>::st(y + at + u, apply(m[u], Store<T>::ld(x + at + u), RES ? Store<T>::ld(res + at + u) : 0.0f));
  }
}

// Any channel count and alignment: one thread per (row, part, channel), its
// decision drawn alone and spread over its components.
template <typename T, bool RES>
__global__ void __launch_bounds__(kThreads) dropout_any_kernel(DropShape s, int KC, Drop d, int64_t row0,
                                                               uint32_t n_threads, const T *x, const T *res, T *y) {
  const uint32_t i = blockIdx.x * kThreads + threadIdx.x;
  if (i >= n_threads) return;
  const uint32_t c = i % static_cast<uint32_t>(s.C), q = i / static_cast<uint32_t>(s.C);
  const uint32_t kp = q % static_cast<uint32_t>(s.KP);
  const int64_t row = row0 + q / static_cast<uint32_t>(s.KP);
  float m = 1.0f;
  DropKey key{};
  if (d.t != 0) key = drop_key(d);
  int l = -1;
  const int k0 = static_cast<int>(kp) * KC;
  for (int k = k0; k < k0 + KC; ++k) {
    const int lk = degree_of(k);
    if (d.t != 0 && (l < 0 || (lk != l && s.share == EGNN_DROP_DEGREE))) {
      const int64_t idx = s.share == EGNN_DROP_ROW      ? row
                          : s.share == EGNN_DROP_DEGREE ? (row * (s.L + 1) + lk) * s.C + c
                                                        : row * s.C + c;
      m = drop_one(idx, d, key);
    }
    l = lk;
    const int64_t at = (row * s.K + k) * s.C + c;
    Store<T>::st(y + at, apply(m, Store<T>::ld(x + at), RES ? Store<T>::ld(res + at) : 0.0f));
  }
}

template <typename T, bool RES>
void launch_vec(int KC, unsigned grid, hipStream_t st, const DropShape &s, const Drop &d, int64_t row0, uint32_t n,
                const T *x, const T *res, T *y) {
  switch (KC) {
    case 1: dropout_vec_kernel<T, 1, RES><<<grid, kThreads, 0, st>>>(s, d, row0, n, x, res, y); break;
    case 2: dropout_vec_kernel<T, 2, RES><<<grid, kThreads, 0, st>>>(s, d, row0, n, x, res, y); break;
    case 3: dropout_vec_kernel<T, 3, RES><<<grid, kThreads, 0, st>>>(s, d, row0, n, x, res, y); break;
    case 4: dropout_vec_kernel<T, 4, RES><<<grid, kThreads, 0, st>>>(s, d, row0, n, x, res, y); break;
    case 5: dropout_vec_kernel<T, 5, RES><<<grid, kThreads, 0, st>>>(s, d, row0, n, x, res, y); break;
    case 6: dropout_vec_kernel<T, 6, RES><<<grid, kThreads, 0, st>>>(s, d, row0, n, x, res, y); break;
    default: dropout_vec_kernel<T, 7, RES><<<grid, kThreads, 0, st>>>(s, d, row0, n, x, res, y); break;
  }
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

template <typename T, bool RES>
egnn_status run(const egnn_dropout_desc *e, int64_t n_rows, const Drop &d, const T *x, const T *res, T *y,
                const char *name, hipStream_t st) {
  DropShape s;
  s.L = e->lmax;
  s.K = (e->lmax + 1) * (e->lmax + 1);
  s.C = e->C;
  s.share = e->share;
  // components per thread: K = (lmax+1)^2 divides by lmax + 1; 4 and 3 for the two largest keep registers low
  const int KC = e->lmax <= 6 ? e->lmax + 1 : e->lmax == 7 ? 4 : 3;
  s.KP = s.K / KC;
  const bool al = aligned16(x) && aligned16(y) && (!RES || aligned16(res));
  const int64_t n = n_rows * s.K * s.C;
  Timed t(st, name, static_cast<double>(n) * (RES ? 2 : 1), static_cast<double>(n) * sizeof(T) * (RES ? 3 : 2));
  if (al && s.K == 1 && s.share != EGNN_DROP_ROW) {
    const int64_t groups = (n + 7) / 8;
    for (int64_t g0 = 0; g0 < groups; g0 += kMaxThreads) {
      const uint32_t m = static_cast<uint32_t>(groups - g0 < kMaxThreads ? groups - g0 : kMaxThreads);
      dropout_flat_kernel<T, RES><<<ceil_div(m, kThreads), kThreads, 0, st>>>(d, g0, m, n, x, res, y);
      EGNN_CHECK_LAUNCH();
    }
    return EGNN_OK;
  }
  const bool vec = al && s.C % 8 == 0;
  const int64_t per_row = static_cast<int64_t>(vec ? s.C / 8 : s.C) * s.KP;
  const int64_t rows_max = kMaxThreads / per_row;
  for (int64_t r0 = 0; r0 < n_rows; r0 += rows_max) {
    const int64_t rows = n_rows - r0 < rows_max ? n_rows - r0 : rows_max;
    const uint32_t m = static_cast<uint32_t>(rows * per_row);
    if (vec)
      launch_vec<T, RES>(KC, ceil_div(m, kThreads), st, s, d, r0, m, x, res, y);
    else
      dropout_any_kernel<T, RES><<<ceil_div(m, kThreads), kThreads, 0, st>>>(s, KC, d, r0, m, x, res, y);
    EGNN_CHECK_LAUNCH();
  }
  return EGNN_OK;
}

egnn_status check(const egnn_dropout_desc *e, int64_t n_rows, const uint64_t *rng, const void *x, const void *y,
                  int *t) {
  clear_error();
  EGNN_REQUIRE(e, "dropout description is null");
  EGNN_REQUIRE(e->lmax >= 0 && e->lmax <= 8, "lmax (%d) must lie in 0..8", e->lmax);
  EGNN_REQUIRE(e->C >= 1 && e->C <= 4096, "C (%d) must lie in 1..4096", e->C);
  EGNN_REQUIRE(e->share == EGNN_DROP_CHANNEL || e->share == EGNN_DROP_DEGREE || e->share == EGNN_DROP_ROW,
               "unknown sharing (%d)", e->share);
  EGNN_REQUIRE(e->storage == EGNN_F32 || e->storage == EGNN_BF16, "unknown storage type (%d)", e->storage);
  *t = drop_threshold(e->p);
  EGNN_REQUIRE(*t >= 0, "dropout probability %g must lie in [0, 1) after rounding to 1/65536", e->p);
  EGNN_REQUIRE(n_rows >= 0 && n_rows <= INT32_MAX, "n_rows (%lld) must lie in 0..2^31-1",
               static_cast<long long>(n_rows));
  if (n_rows == 0) return EGNN_OK;
  EGNN_REQUIRE(x && y, "input and output are required");
  EGNN_REQUIRE(rng || *t == 0, "rng state is required when the probability is not zero");
  EGNN_REQUIRE((reinterpret_cast<uintptr_t>(rng) & 7) == 0, "rng state must be 8-byte aligned");
  return EGNN_OK;
}

}  // namespace

extern "C" egnn_status egnn_dropout_fwd(const egnn_dropout_desc *e, int64_t n_rows, const void *x, const void *residual,
                                        const uint64_t *rng, void *y, hipStream_t stream) {
  int t;
  const egnn_status st = check(e, n_rows, rng, x, y, &t);
  if (st != EGNN_OK || n_rows == 0) return st;
  const Drop d = make_drop(rng, e->site, t);
  if (e->storage == EGNN_BF16) {
    const auto *xp = static_cast<const uint16_t *>(x), *rp = static_cast<const uint16_t *>(residual);
    auto *yp = static_cast<uint16_t *>(y);
    return rp ? run<uint16_t, true>(e, n_rows, d, xp, rp, yp, "dropout_fwd", stream)
              : run<uint16_t, false>(e, n_rows, d, xp, rp, yp, "dropout_fwd", stream);
  }
  const auto *xp = static_cast<const float *>(x), *rp = static_cast<const float *>(residual);
  auto *yp = static_cast<float *>(y);
  return rp ? run<float, true>(e, n_rows, d, xp, rp, yp, "dropout_fwd", stream)
            : run<float, false>(e, n_rows, d, xp, rp, yp, "dropout_fwd", stream);
}

extern "C" egnn_status egnn_dropout_bwd(const egnn_dropout_desc *e, int64_t n_rows, const float *grad_y,
                                        const uint64_t *rng, float *grad_x, hipStream_t stream) {
  int t;
  const egnn_status st = check(e, n_rows, rng, grad_y, grad_x, &t);
  if (st != EGNN_OK || n_rows == 0) return st;
  return run<float, false>(e, n_rows, make_drop(rng, e->site, t), grad_y, nullptr, grad_x, "dropout_bwd", stream);
}
