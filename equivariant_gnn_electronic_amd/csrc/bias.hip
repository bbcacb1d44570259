// Learned bias of edges by distance buckets, and the table's gradient (see egnn.h).
//
//   bucket(r) = number of borders <= r;  bias[e][:] = table[bucket(dist_e)][:]
//   grad_table[b][:] = sum of grad_bias[e][:] over the edges of bucket b
//
// Both directions are bound by HBM: the [E][M] array is written (read) once,
// next to 4 bytes of distance an edge.
#include <cmath>

#include "common.h"
#include "timing.h"

using namespace egnn;

namespace {

constexpr int kThreads = 256;
constexpr int kWave = 64;
constexpr int kWaves = kThreads / kWave;
constexpr int kMaxBuckets = 1024;
constexpr int kMaxColumns = 64;
constexpr int kTableLds = 8192;       // floats of a table that is staged in LDS (32 KB)
constexpr int kGradLds = 12544;       // floats of private tables in a block (49 KB: with the borders three blocks a CU)
constexpr int kCUs = 256;
constexpr int kLdsOfCU = 160 * 1024;

// number of borders <= r in an ascending list (NaN: 0); the answer lies in
// 0..n whatever the list holds
__device__ inline int bucket_of(const float *borders, int n, float r) {
  int lo = 0, hi = n;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (borders[mid] <= r) lo = mid + 1;
    else hi = mid;
  }
  return lo;
}

// A wave takes 64 edges: each lane finds one edge's bucket, then the lanes
// write the 64 rows as one contiguous run, VW columns a lane.  (544,000 edges,
// 16 columns, 37 MB: 10.7 us, 3.5 TB/s; a launch alone takes 3.)
template <int VW>
__global__ void __launch_bounds__(kThreads) bias_fwd_kernel(const float *__restrict__ dist, int64_t E,
                                                            const float *__restrict__ borders, int B, int M,
                                                            const float *__restrict__ table, bool staged,
                                                            float *__restrict__ bias) {
  __shared__ float sb[kMaxBuckets];
  __shared__ __align__(16) float stab[kTableLds];
  for (int i = threadIdx.x; i < B - 1; i += kThreads) sb[i] = borders[i];
  if (staged)
    for (int i = threadIdx.x; i < B * M; i += kThreads) stab[i] = table[i];
  __syncthreads();
  const int lane = threadIdx.x & (kWave - 1);
  const int MV = M / VW;
  const uint32_t inv = ((1u << 20) + MV - 1) / MV;  // f / MV = f inv >> 20: f MV < 2^20 as f < 64 MV, MV <= 64
  for (int64_t base = (static_cast<int64_t>(blockIdx.x) * kWaves + (threadIdx.x >> 6)) * kWave; base < E;
       base += static_cast<int64_t>(gridDim.x) * kThreads) {
    const int cnt = static_cast<int>(E - base < kWave ? E - base : kWave);
    const int bk = bucket_of(sb, B - 1, dist[base + (lane < cnt ? lane : cnt - 1)]);
    float *out = bias + base * M;
    for (int f0 = 0; f0 < cnt * MV; f0 += kWave) {
      const int f = f0 + lane;
      const int e = static_cast<int>((static_cast<uint32_t>(f) * inv) >> 20), c = f - e * MV;
      const int at = __shfl(bk, e & (kWave - 1)) * M + c * VW;
      if (f < cnt * MV) {
        if constexpr (VW == 4) {
          const float4 v = staged ? *reinterpret_cast<const float4 *>(stab + at)
                                  : *reinterpret_cast<const float4 *>(table + at);
          reinterpret_cast<float4 *>(out)[f] = v;
        } else {
          out[f] = staged ? stab[at] : table[at];
        }
      }
    }
  }
}

// Partial tables.  A wave takes 64 edges; lane = group * Mt + column adds one
// column of its group's edges into the group's own table in LDS.  Each address
// belongs to one lane, which adds in edge order, so the sums are deterministic.
// Four edges are read, added and written together, so that the chain through
// LDS is one for four.  (3.15 M edges, 16 columns, 64 buckets: LDS float
// atomics 299 us, at 222 cycles an instruction; one edge at a time 97; four 62,
// 3.5 TB/s, what the chains and nine waves a CU of 48 KB tables allow.)
// Copies are summed in a fixed order at the end.
// blockIdx.y picks a tile of Mt columns when a whole table does not fit.
template <int U>
__global__ void __launch_bounds__(kThreads) bias_bwd_kernel(const float *__restrict__ dist, int64_t E,
                                                            const float *__restrict__ borders, int B, int M, int Mt,
                                                            int groups, int copies,
                                                            const float *__restrict__ grad, float *__restrict__ part) {
  constexpr int Q = U < 4 ? U : 4;       // edges read, added and written together
  extern __shared__ float lds[];
  float *sb = lds;                       // [B]
  float *tab = lds + ((B + 3) & ~3);     // [copies][B][Mt]
  const int waves = copies / groups;     // waves that add (the launch has copies = waves * groups)
  for (int i = threadIdx.x; i < B - 1; i += blockDim.x) sb[i] = borders[i];
  for (int i = threadIdx.x; i < copies * B * Mt; i += blockDim.x) tab[i] = 0.0f;
  __syncthreads();
  const int lane = threadIdx.x & (kWave - 1), wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c0 = blockIdx.y * Mt;
  const int mt = M - c0 < Mt ? M - c0 : Mt;
  const int grp = lane / Mt, c = lane - grp * Mt;
  const bool on = grp < groups && c < mt;
  float *mine = tab + ((wave * groups + (grp < groups ? grp : 0)) * B) * Mt + (c < Mt ? c : 0);
  const int ge = grp < groups ? grp : 0;
  const int64_t step = static_cast<int64_t>(gridDim.x) * waves * kWave;
  const uint32_t own = static_cast<uint32_t>(ge * M + (c < mt ? c : 0));
  // a round is U edges of every group; the next round's loads are under way
  // while one is added (addresses past the end are clamped, their values not
  // used; before it the wave's part of an address is scalar work: 75 us to 67)
  const auto load = [&](int64_t base, int i0, float (&v)[U]) {
    if (base + i0 + groups * U <= E) {
      const float *g = grad + (base + i0) * M + c0;
#pragma unroll
      for (int u = 0; u < U; ++u) v[u] = (g + u * groups * M)[own];
      return;
    }
    const int64_t left = E - base - 1;
    const float *g = grad + base * M + c0 + (c < mt ? c : 0);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int e = i0 + u * groups + ge;
      v[u] = g[static_cast<int64_t>(e < left ? e : static_cast<int>(left)) * M];
    }
  };
  int64_t base = (static_cast<int64_t>(blockIdx.x) * waves + wave) * kWave;
  if (base < E) {
    float v[U];
    float r = dist[base + lane < E ? base + lane : E - 1];
    load(base, 0, v);
    while (base < E) {
      const int cnt = static_cast<int>(E - base < kWave ? E - base : kWave);
      const int64_t after = base + step;
      const int bk = bucket_of(sb, B - 1, r) * Mt;
      if (after < E) r = dist[after + lane < E ? after + lane : E - 1];
      for (int i0 = 0; i0 < cnt; i0 += groups * U) {
        float cur[U];
#pragma unroll
        for (int u = 0; u < U; ++u) cur[u] = v[u];
        const bool more = i0 + groups * U < cnt;
        if (more || after < E) load(more ? base : after, more ? i0 + groups * U : 0, v);
        if (i0 + groups * U > cnt) {
#pragma unroll
          for (int u = 0; u < U; ++u) cur[u] = i0 + u * groups + ge < cnt ? cur[u] : 0.0f;
        }
#pragma unroll
        for (int u = 0; u < U; u += Q) {
          int at[Q];
          float t[Q];
#pragma unroll
          for (int k = 0; k < Q; ++k)  // of edge i0 + (u + k) groups + ge, counted modulo 64
            at[k] = __builtin_amdgcn_ds_bpermute((i0 + (u + k) * groups) * 4 + ge * 4, bk);
          if (on) {
#pragma unroll
            for (int k = 0; k < Q; ++k) t[k] = mine[at[k]];
            // an edge of the same bucket as an earlier one of the round's adds to that one's sum
#pragma unroll
            for (int k = 0; k < Q; ++k) {
#pragma unroll
              for (int j = 0; j < k; ++j) t[k] = at[j] == at[k] ? t[j] : t[k];
              t[k] += cur[u + k];
            }
#pragma unroll
            for (int k = 0; k < Q; ++k) mine[at[k]] = t[k];
          }
        }
      }
      base = after;
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < B * mt; i += blockDim.x) {
    const int b = i / mt, cc = i - b * mt;
    double s = 0.0;  // thousands of short sums are joined: in 64 bits that adds no error to theirs
    for (int k = 0; k < copies; ++k) s += tab[(k * B + b) * Mt + cc];
    part[(static_cast<int64_t>(blockIdx.x) * B + b) * M + c0 + cc] = static_cast<float>(s);
  }
}

// grad_table[i] = sum over the partial tables: 32 threads an entry, in a fixed order
__global__ void __launch_bounds__(kThreads) bias_sum_kernel(const float *__restrict__ part, int n_part, int n,
                                                            float *__restrict__ out) {
  __shared__ double red[32][9];
  const int col = threadIdx.x & 7, r = threadIdx.x >> 3;
  const int i = blockIdx.x * 8 + col;
  const float *p = part + (i < n ? i : n - 1);
  double s = 0.0;
  for (int p0 = r; p0 < n_part; p0 += 32 * 8) {
    float v[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) v[u] = p[static_cast<int64_t>(p0 + 32 * u < n_part ? p0 + 32 * u : p0) * n];
#pragma unroll
    for (int u = 0; u < 8; ++u) s += p0 + 32 * u < n_part ? v[u] : 0.0f;
  }
  red[r][col] = s;
  __syncthreads();
  if (r == 0 && i < n) {
#pragma unroll
    for (int k = 1; k < 32; ++k) s += red[k][col];
    out[i] = static_cast<float>(s);
  }
}

struct GradPlan {
  int Mt, groups, waves, blocks;
};

// Edges of a group in one round.  A wave's 64 edges are covered by whole rounds
// of groups * U places, of which those past the last edge are work for nothing,
// and a round costs about as much as one more edge a group.  (3.15 M edges, 64
// buckets, 16 for any number of columns against this: 1 column 68 and 31 us, 2
// columns 65 and 33, 6 columns 81 and 62, 8 columns 64 and 44.)
int edges_a_round(int groups) {
  int best = 1;
  int least = INT32_MAX;
  for (const int U : {16, 8, 4, 2, 1}) {
    const int rounds = (kWave + groups * U - 1) / (groups * U);
    const int cost = rounds * (U + 1);
    if (cost < least) {
      least = cost;
      best = U;
    }
  }
  return best;
}

// Columns per tile, edge groups per wave and waves per block so that the
// block's private tables fit LDS.
GradPlan grad_plan(int B, int M, int64_t E) {
  GradPlan p;
  int Mt = M;
  while (Mt > 1 && B * Mt > kGradLds) Mt = (Mt + 1) / 2;
  p.Mt = Mt;
  const int fit = kGradLds / (B * Mt);  // private tables that fit
  p.groups = kWave / Mt;
  if (p.groups > fit) p.groups = fit;
  p.waves = fit / p.groups;
  if (p.waves > kWaves) p.waves = kWaves;
  // a partial table for each block that the CUs hold at once, so that all of them
  // run together (6 columns, 64 buckets: 62 us where 768 blocks of 60 KB do not
  // fit at once, 46; 16 columns, 500 buckets: 417 with three blocks a CU, 345)
  const int at_once = kLdsOfCU / (4 * (B + 3 + p.waves * p.groups * B * Mt) + 1024);
  const int64_t most = kCUs * (at_once > 8 ? 8 : at_once), want = (E + p.waves * kWave - 1) / (p.waves * kWave);
  p.blocks = static_cast<int>(want < 1 ? 1 : want > most ? most : want);
  return p;
}

egnn_status check(const egnn_bias_desc *d, const egnn_graph *g) {
  clear_error();
  EGNN_REQUIRE(d, "bias description is null");
  EGNN_REQUIRE(d->n_buckets >= 1 && d->n_buckets <= kMaxBuckets, "n_buckets (%d) must lie in 1..%d", d->n_buckets,
               kMaxBuckets);
  EGNN_REQUIRE(d->n_columns >= 1 && d->n_columns <= kMaxColumns, "n_columns (%d) must lie in 1..%d", d->n_columns,
               kMaxColumns);
  EGNN_REQUIRE(g, "graph is null");
  EGNN_REQUIRE(g->n_edges >= 0 && g->n_edges <= INT32_MAX, "n_edges (%lld) must lie in 0..2^31-1",
               static_cast<long long>(g->n_edges));
  EGNN_REQUIRE(g->n_edges == 0 || g->dist, "the graph's dist array is required");
  return EGNN_OK;
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

}  // namespace

extern "C" egnn_status egnn_distance_borders(int32_t n_buckets, int32_t n_linear, double r_linear, double r_max,
                                             float *borders) {
  clear_error();
  EGNN_REQUIRE(n_buckets >= 1 && n_buckets <= kMaxBuckets, "n_buckets (%d) must lie in 1..%d", n_buckets, kMaxBuckets);
  EGNN_REQUIRE(n_linear >= 1 && n_linear <= n_buckets, "n_linear (%d) must lie in 1..n_buckets", n_linear);
  EGNN_REQUIRE(std::isfinite(r_linear) && r_linear > 0.0, "r_linear must be positive");
  EGNN_REQUIRE(n_linear == n_buckets || (std::isfinite(r_max) && r_max > r_linear), "r_max must exceed r_linear");
  EGNN_REQUIRE(borders || n_buckets == 1, "borders is null");
  // n_linear buckets of equal width up to r_linear, then equal ratios up to
  // r_max, whose last bucket also takes everything beyond
  for (int i = 0; i < n_buckets - 1; ++i)
    borders[i] = static_cast<float>(
        i < n_linear ? r_linear * (i + 1) / n_linear
                     : r_linear * std::pow(r_max / r_linear, static_cast<double>(i + 1 - n_linear) / (n_buckets - n_linear)));
  return EGNN_OK;
}

extern "C" egnn_status egnn_distance_bias_fwd(const egnn_bias_desc *d, const egnn_graph *g, const float *borders,
                                              const float *table, float *bias, hipStream_t stream) {
  const egnn_status st = check(d, g);
  if (st != EGNN_OK) return st;
  const int64_t E = g->n_edges;
  if (E == 0) return EGNN_OK;
  const int B = d->n_buckets, M = d->n_columns;
  EGNN_REQUIRE((borders || B == 1) && table && bias, "borders, table and bias are required");
  Timed t(stream, "distance_bias_fwd", 0.0, 4.0 * (static_cast<double>(E) * (M + 1) + B * M));
  const bool staged = B * M <= kTableLds;
  const unsigned want = ceil_div(E, kThreads), grid = want < 2048 ? want : 2048;  // eight blocks a CU
  if (M % 4 == 0 && aligned16(table) && aligned16(bias))
    bias_fwd_kernel<4><<<grid, kThreads, 0, stream>>>(g->dist, E, borders, B, M, table, staged, bias);
  else
    bias_fwd_kernel<1><<<grid, kThreads, 0, stream>>>(g->dist, E, borders, B, M, table, staged, bias);
  EGNN_CHECK_LAUNCH();
  return EGNN_OK;
}

extern "C" egnn_status egnn_distance_bias_workspace(const egnn_bias_desc *d, const egnn_graph *g, size_t *bytes) {
  const egnn_status st = check(d, g);
  if (st != EGNN_OK) return st;
  EGNN_REQUIRE(bytes, "bytes is null");
  const GradPlan p = grad_plan(d->n_buckets, d->n_columns, g->n_edges);
  *bytes = static_cast<size_t>(p.blocks) * d->n_buckets * d->n_columns * sizeof(float);
  return EGNN_OK;
}

extern "C" egnn_status egnn_distance_bias_bwd(const egnn_bias_desc *d, const egnn_graph *g, const float *borders,
                                              const float *grad_bias, float *grad_table, void *ws, size_t ws_bytes,
                                              hipStream_t stream) {
  const egnn_status st = check(d, g);
  if (st != EGNN_OK) return st;
  const int64_t E = g->n_edges;
  const int B = d->n_buckets, M = d->n_columns;
  EGNN_REQUIRE((borders || B == 1) && grad_table, "borders and grad_table are required");
  EGNN_REQUIRE(E == 0 || grad_bias, "grad_bias is required");
  size_t need = 0;
  egnn_distance_bias_workspace(d, g, &need);
  if (!ws || ws_bytes < need) {
    set_error("workspace of %zu bytes, needs %zu", ws ? ws_bytes : size_t(0), need);
    return EGNN_E_WORKSPACE;
  }
  EGNN_REQUIRE((reinterpret_cast<uintptr_t>(ws) & 15) == 0, "workspace must be 16-byte aligned");
  auto *part = static_cast<float *>(ws);
  const GradPlan p = grad_plan(B, M, E);
  const int copies = p.waves * p.groups;
  const size_t lds = (((B + 3) & ~3) + static_cast<size_t>(copies) * B * p.Mt) * sizeof(float);
  {
    Timed t(stream, "distance_bias_bwd", static_cast<double>(E) * M, 4.0 * static_cast<double>(E) * (M + 1));
    const dim3 grid(p.blocks, (M + p.Mt - 1) / p.Mt);
    const int U = edges_a_round(p.groups);
    const auto kernel = U == 16  ? bias_bwd_kernel<16>
                        : U == 8 ? bias_bwd_kernel<8>
                        : U == 4 ? bias_bwd_kernel<4>
                        : U == 2 ? bias_bwd_kernel<2>
                                 : bias_bwd_kernel<1>;
    kernel<<<grid, p.waves * kWave, lds, stream>>>(g->dist, E, borders, B, M, p.Mt, p.groups, copies, grad_bias, part);
    EGNN_CHECK_LAUNCH();
  }
  Timed t(stream, "distance_bias_sum", static_cast<double>(p.blocks) * B * M, 4.0 * (p.blocks + 1.0) * B * M);
  bias_sum_kernel<<<ceil_div(B * M, 8), kThreads, 0, stream>>>(part, p.blocks, B * M, grad_table);
  EGNN_CHECK_LAUNCH();
  return EGNN_OK;
}
