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

// VW neighbouring channels
template <typename T, int VW> struct Span;
template <> struct Span<float, 8> {
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
template <> struct Span<uint16_t, 8> {
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

template <> struct Span<float, 2> {
  __device__ static inline void ld(const float *p, float (&v)[2]) {
    const float2 a = *reinterpret_cast<const float2 *>(p);
    v[0] = a.x; v[1] = a.y;
  }
  __device__ static inline void st(float *p, const float (&v)[2]) {
    *reinterpret_cast<float2 *>(p) = make_float2(v[0], v[1]);
  }
};
template <> struct Span<uint16_t, 2> {
  __device__ static inline void ld(const uint16_t *p, float (&v)[2]) {
    const uint32_t a = *reinterpret_cast<const uint32_t *>(p);
    v[0] = __uint_as_float(a << 16);
    v[1] = __uint_as_float(a & 0xFFFF0000u);
  }
  __device__ static inline void st(uint16_t *p, const float (&v)[2]) {
    *reinterpret_cast<uint32_t *>(p) =
        static_cast<uint32_t>(f32_to_bf16(v[0])) | (static_cast<uint32_t>(f32_to_bf16(v[1])) << 16);
  }
};
template <typename T> struct Span<T, 1> {
  __device__ static inline void ld(const T *p, float (&v)[1]) { v[0] = Store<T>::ld(p); }
  __device__ static inline void st(T *p, const float (&v)[1]) { Store<T>::st(p, v[0]); }
};

__device__ inline int degree_of(int k) {  // floor(sqrt(k)) for k < 81
  int l = 0;
  while ((l + 1) * (l + 1) <= k) ++l;
  return l;
}

// Keep factors of the VW channels at c0 of (row, degree l).  C is a multiple
// of VW, so the decisions lie in one generator call.
template <int VW>
__device__ inline void factors(const DropShape &s, const Drop &d, const DropKey &key, int64_t row, int l, int c0,
                               float (&m)[VW]) {
  if (s.share == EGNN_DROP_ROW) {
    const float f = drop_one(row, d, key);
#pragma unroll
    for (int u = 0; u < VW; ++u) m[u] = f;
    return;
  }
  const int64_t base = s.share == EGNN_DROP_DEGREE ? (row * (s.L + 1) + l) * s.C + c0 : row * s.C + c0;
  const uint4 w = philox4x32(static_cast<uint64_t>(base) >> 3, key);
  const int u0 = VW == 8 ? 0 : static_cast<int>(base & 7);
#pragma unroll
  for (int u = 0; u < VW; ++u) m[u] = drop_draw(w, u0 + u) >= d.t ? d.factor : 0.0f;
}

// A dropped element is the residual (or 0) whatever x holds there, so that an
// infinity or NaN in a dropped place does not come through.
__device__ inline float apply(float m, float x, float r) { return m == 0.0f ? r : r + m * x; }

// One thread: VW channels of KC consecutive components of one row, all of whose
// loads are issued first.  Lanes run over channel groups first, so a group of
// lanes streams consecutive lines.  VW is 8, or 2 or 1 where the channel count
// or the alignment allows no more (50 channels, lmax 4, bf16, 600 MB: 131 us by
// pairs, 5.115 TB/s would take 117; 234 element after element).
template <typename T, int KC, bool RES, int VW>
__global__ void __launch_bounds__(kThreads) dropout_vec_kernel(DropShape s, Drop d, int64_t row0, uint32_t n_threads,
                                                               const T *x, const T *res, T *y) {
  const uint32_t i = blockIdx.x * kThreads + threadIdx.x;
  if (i >= n_threads) return;
  const uint32_t CG = static_cast<uint32_t>(s.C) / VW;
  const uint32_t g = i % CG, q = i / CG;
  const uint32_t kp = q % static_cast<uint32_t>(s.KP);
  const int64_t row = row0 + q / static_cast<uint32_t>(s.KP);
  const int k0 = static_cast<int>(kp) * KC;
  const int64_t at = (row * s.K + k0) * s.C + static_cast<int64_t>(g) * VW;
  float v[KC][VW], r[KC][VW];
#pragma unroll
  for (int j = 0; j < KC; ++j) Span<T, VW>::ld(x + at + static_cast<int64_t>(j) * s.C, v[j]);
  if constexpr (RES) {
#pragma unroll
    for (int j = 0; j < KC; ++j) Span<T, VW>::ld(res + at + static_cast<int64_t>(j) * s.C, r[j]);
  }
  float m[VW];
  const bool every = d.t == 0;
  DropKey key{};
  if (every) {
#pragma unroll
    for (int u = 0; u < VW; ++u) m[u] = 1.0f;
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
    if (fresh && !every) factors<VW>(s, d, key, row, l, static_cast<int>(g) * VW, m);
    fresh = false;
    float o[VW];
#pragma unroll
    for (int u = 0; u < VW; ++u) o[u] = apply(m[u], v[j][u], RES ? r[j][u] : 0.0f);
    Span<T, VW>::st(y + at + static_cast<int64_t>(j) * s.C, o);
  }
}

// Invariants (one component): eight elements of the flat array a thread,
// whatever the channel count.  The decisions run over the same array (one
// generator call), or over its rows (C elements each; one call, or two where
// the eight rows of a call end).  (500,000 rows of 33, bf16, by row: 30 us, 90
// with a thread and a call an element.  Rows of whole eights keep the kernel
// above, whose addresses are simpler: 64 channels, fp32, 73 us against 79.)
template <typename T, bool RES>
__global__ void __launch_bounds__(kThreads) dropout_flat_kernel(Drop d, bool by_row, uint32_t C, int64_t group0,
                                                                uint32_t n_groups, int64_t n, const T *x, const T *res,
                                                                T *y) {
  const uint32_t i = blockIdx.x * kThreads + threadIdx.x;
  if (i >= n_groups) return;
  const int64_t j = group0 + i, at = j * 8;
  float m[8];
  if (d.t == 0) {
#pragma unroll
    for (int u = 0; u < 8; ++u) m[u] = 1.0f;
  } else if (by_row) {
    const DropKey key = drop_key(d);
    uint64_t row = static_cast<uint64_t>(at) / C;
    uint32_t c = static_cast<uint32_t>(static_cast<uint64_t>(at) - row * C);
    uint4 w = philox4x32(row >> 3, key);
    float f = drop_draw(w, static_cast<int>(row & 7)) >= d.t ? d.factor : 0.0f;
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      m[u] = f;
      if (++c == C) {
        c = 0;
        ++row;
        if ((row & 7) == 0) w = philox4x32(row >> 3, key);
        f = drop_draw(w, static_cast<int>(row & 7)) >= d.t ? d.factor : 0.0f;
      }
    }
  } else {
    const uint4 w = philox4x32(static_cast<uint64_t>(j), drop_key(d));
#pragma unroll
    for (int u = 0; u < 8; ++u) m[u] = drop_draw(w, u) >= d.t ? d.factor : 0.0f;
  }
  if (at + 8 <= n) {
    float v[8], r[8], o[8];
    Span<T, 8>::ld(x + at, v);
    if constexpr (RES) Span<T, 8>::ld(res + at, r);
#pragma unroll
    for (int u = 0; u < 8; ++u) o[u] = apply(m[u], v[u], RES ? r[u] : 0.0f);
    Span<T, 8>::st(y + at, o);
  } else {
#pragma unroll
    for (int u = 0; u < 8; ++u)
      if (at + u < n)
        Store<T>::st(y + at + u, apply(m[u], Store<T>::ld(x + at + u), RES ? Store<T>::ld(res + at + u) : 0.0f));
  }
}

template <typename T, bool RES, int VW>
void launch_vec(int KC, unsigned grid, hipStream_t st, const DropShape &s, const Drop &d, int64_t row0, uint32_t n,
                const T *x, const T *res, T *y) {
  switch (KC) {
    case 1: dropout_vec_kernel<T, 1, RES, VW><<<grid, kThreads, 0, st>>>(s, d, row0, n, x, res, y); break;
    case 2: dropout_vec_kernel<T, 2, RES, VW><<<grid, kThreads, 0, st>>>(s, d, row0, n, x, res, y); break;
    case 3: dropout_vec_kernel<T, 3, RES, VW><<<grid, kThreads, 0, st>>>(s, d, row0, n, x, res, y); break;
    case 4: dropout_vec_kernel<T, 4, RES, VW><<<grid, kThreads, 0, st>>>(s, d, row0, n, x, res, y); break;
    case 5: dropout_vec_kernel<T, 5, RES, VW><<<grid, kThreads, 0, st>>>(s, d, row0, n, x, res, y); break;
    case 6: dropout_vec_kernel<T, 6, RES, VW><<<grid, kThreads, 0, st>>>(s, d, row0, n, x, res, y); break;
    default: dropout_vec_kernel<T, 7, RES, VW><<<grid, kThreads, 0, st>>>(s, d, row0, n, x, res, y); break;
  }
}

bool aligned(const void *p, size_t bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }

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
  const auto all_aligned = [&](size_t bytes) {
    return aligned(x, bytes) && aligned(y, bytes) && (!RES || aligned(res, bytes));
  };
  const int64_t n = n_rows * s.K * s.C;
  Timed t(st, name, static_cast<double>(n) * (RES ? 2 : 1), static_cast<double>(n) * sizeof(T) * (RES ? 3 : 2));
  const bool by_row = s.share == EGNN_DROP_ROW;
  if (s.K == 1 && all_aligned(16) && !(by_row && s.C % 8 == 0)) {
    const int64_t groups = (n + 7) / 8;
    for (int64_t g0 = 0; g0 < groups; g0 += kMaxThreads) {
      const uint32_t m = static_cast<uint32_t>(groups - g0 < kMaxThreads ? groups - g0 : kMaxThreads);
      dropout_flat_kernel<T, RES><<<ceil_div(m, kThreads), kThreads, 0, st>>>(d, by_row, s.C, g0, m, n, x, res, y);
      EGNN_CHECK_LAUNCH();
    }
    return EGNN_OK;
  }
  const int VW = s.C % 8 == 0 && all_aligned(16) ? 8 : s.C % 2 == 0 && all_aligned(2 * sizeof(T)) ? 2 : 1;
  const int64_t per_row = static_cast<int64_t>(s.C / VW) * s.KP;
  const int64_t rows_max = kMaxThreads / per_row;
  for (int64_t r0 = 0; r0 < n_rows; r0 += rows_max) {
    const int64_t rows = n_rows - r0 < rows_max ? n_rows - r0 : rows_max;
    const uint32_t m = static_cast<uint32_t>(rows * per_row);
    if (VW == 8) launch_vec<T, RES, 8>(KC, ceil_div(m, kThreads), st, s, d, r0, m, x, res, y);
    else if (VW == 2) launch_vec<T, RES, 2>(KC, ceil_div(m, kThreads), st, s, d, r0, m, x, res, y);
    else launch_vec<T, RES, 1>(KC, ceil_div(m, kThreads), st, s, d, r0, m, x, res, y);
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
