// balance.cu -- the router's balance loss with per-expert counts, and the
// gradient of the router's logits.
//
// Over the n tokens that the mask leaves (all without one), k slots each, with
// p = softmax(logits) over all E experts and c_e slots that chose expert e:
//   loss = coef E sum_e f_e P_e,   f_e = c_e / (n k),   P_e = mean_t p[t, e]
//   d logits[t, e] = dloss coef E / n  p (f_e - sum_j f_j p[t, j])   (balance)
// and, from the gradient dw of the routing weights w of the chosen slots,
//   w = softmax over the chosen:  + w_j (dw_j - sum_i w_i dw_i) at their IDs
//   w = p at the chosen:          + w_j dw_j at their IDs - p sum_i w_i dw_i.
//
// Bound by memory: the forward reads the logits once, the gradient reads them
// again (keeping p would take a write and a read more) and writes as much.
// A group of L lanes holds a row in registers, 4 NV columns a lane, so that
// maximum, sum and the weighted sum take no second read.  The same lanes see the
// same columns in every row, so the forward's column sums stay in registers too;
// it issues the next row's loads before it works on the present one.  The
// gradient's f_e are in shared memory, which leaves room for half as many rows
// again.  Column sums are fp32, of 256 rows of a group and then of a CTA's groups, and
// two-sums of fp32 across CTAs, in a fixed order: results do not depend on the order of
// execution.
// Measured (65,536 x 896, top-16): forward 43 us (5.5 TB/s) and 7 for the join,
// gradient 76 to 81 (6 TB/s).
#include "../../include/situ_moe.h"
#include "gemm_groups.cuh"

#include <cooperative_groups.h>

#include <type_traits>

namespace situ {

namespace {

constexpr int kFwdThreads = 512;     // one CTA per SM, so that there are few partial sums
constexpr int kBackThreads = 256;    // three CTAs per SM
// One more of either where rows are short (up to 256 columns: a chain of reductions
// each) and many: 65,536 x 130, top-6, 30 + 33 us without and 24 + 30 with them;
// 8,192 x 256 11 + 9 and 12 + 10.
constexpr int fwd_ctas(int nv) { return nv <= 2 ? 2 : 1; }
constexpr int back_ctas(int nv) { return nv <= 2 ? 4 : 3; }
constexpr int kManyRows = 16, kManyBackRows = 8;   // of a group
constexpr int kMaxExperts = SITU_MAX_LOCAL_EXPERTS;
constexpr int kFinalCtas = 8;        // of the joining kernel's one cluster
constexpr int kFinalThreads = 512;
constexpr int kMostSms = 256;        // that grids are sized for
constexpr int kFold = 256;           // rows of a group whose column sums stay in registers

struct BalanceParams {
  const float* logits;
  long ld;
  const int32_t* ids;
  const uint8_t* mask;
  int T, E, k;
  float coef;
  float* loss;
  int32_t *counts, *tokens;
  float2* stats;
  // partial sums: [grid][pitch] each, pitch = E rounded up to 4, then a token count per CTA
  int pitch;
  float* part_p;
  int32_t *part_c, *part_n;
};

struct RouterBackParams {
  const float* logits;
  long ld;
  const int32_t* ids;
  const uint8_t* mask;
  int T, E, k, renorm;
  float coef;
  const int32_t *counts, *tokens;
  const float2* stats;
  const float *dloss, *w, *dw;
  float* out;
  long ldo;
};

// The rows' groups: L lanes of a warp, or four whole warps (L = 128).
template <int L>
struct Group {
  int id, lane;          // group in the CTA, lane in the group
  __device__ __forceinline__ Group() : id(threadIdx.x / L), lane(threadIdx.x % L) {}
  __device__ __forceinline__ void sync() const {
    if (L > kWarp) asm volatile("bar.sync %0, %1;" ::"r"(id + 1), "n"(L) : "memory");
    else __syncwarp();
  }
  // op over the group, the same bits in every lane; red: 8 floats of the
  // group, free again after two further calls
  template <class Op>
  __device__ __forceinline__ float reduce(float v, float* red, int& turn, Op op) const {
#pragma unroll
    for (int d = (L < kWarp ? L : kWarp) / 2; d >= 1; d >>= 1) v = op(v, __shfl_xor_sync(0xffffffffu, v, d));
    if (L > kWarp) {
      float* r = red + 4 * turn;
      turn ^= 1;
      if ((lane & 31) == 0) r[lane >> 5] = v;
      sync();
      v = op(op(r[0], r[1]), op(r[2], r[3]));
    }
    return v;
  }
};

// Column i of a lane's j-th four: neighbours where rows are read 16 bytes a lane
// (VEC), else a lane's width apart, so that a load's lanes are neighbours (35,954 x
// 729, both passes: 81 us with fours, 77 so).
template <int L, bool VEC>
__device__ __forceinline__ int column(int lane, int j, int i) {
  return VEC ? 4 * (lane + L * j) + i : lane + L * (4 * j + i);
}
template <int L, bool VEC>
__device__ __forceinline__ float4 columns(const float* row, int lane, int j) {
  return VEC ? *reinterpret_cast<const float4*>(row + 4 * (lane + L * j))
             : make_float4(row[lane + L * 4 * j], row[lane + L * (4 * j + 1)], row[lane + L * (4 * j + 2)],
                           row[lane + L * (4 * j + 3)]);
}

// A lane's columns of a row, `none` past its end.
template <int L, int NV, bool VEC>
__device__ __forceinline__ void load_row(float (&v)[4 * NV], const float* row, int lane, int E, float none) {
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    if (VEC) {
      const int c = column<L, VEC>(lane, j, 0);
      const float4 x = c < E ? __ldg(reinterpret_cast<const float4*>(row + c)) : make_float4(none, none, none, none);
      v[4 * j] = x.x;
      v[4 * j + 1] = x.y;
      v[4 * j + 2] = x.z;
      v[4 * j + 3] = x.w;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int c = column<L, VEC>(lane, j, i);
        v[4 * j + i] = c < E ? __ldg(row + c) : none;
      }
    }
  }
}

__device__ __forceinline__ float fmax_op(float a, float b) { return fmaxf(a, b); }
__device__ __forceinline__ float add_op(float a, float b) { return a + b; }

template <int L, int NV, bool VEC>
__global__ void __launch_bounds__(kFwdThreads, fwd_ctas(NV))
balance_kernel(BalanceParams p) {
  constexpr int kGroups = kFwdThreads / L, V = 4 * NV;
  extern __shared__ float smem[];              // column sums [E], counts [E]
  __shared__ float red[kGroups][8];
  __shared__ int tokens_s;
  __shared__ double loss_s[kFwdThreads / kWarp];
  float* sum_p = smem;
  int* hist = reinterpret_cast<int*>(smem + p.E);
  for (int e = threadIdx.x; e < p.E; e += kFwdThreads) {
    sum_p[e] = 0.f;
    hist[e] = 0;
  }
  if (threadIdx.x == 0) tokens_s = 0;
  __syncthreads();
  const Group<L> g;
  int turn = 0, mine = 0;
  float acc[V], cur[V];
#pragma unroll
  for (int i = 0; i < V; ++i) acc[i] = 0.f;
  const long step = (long)gridDim.x * kGroups;
  // whole warps take part in the shuffles: a group past the end repeats the last row
  const long first = (long)blockIdx.x * kGroups + g.id;
  const long rounds = (p.T - (long)blockIdx.x * kGroups + step - 1) / step;
  load_row<L, NV, VEC>(cur, p.logits + (size_t)min(first, (long)p.T - 1) * p.ld, g.lane, p.E, -INFINITY);
  for (long from = 0; from < rounds; from += kFold) {
    for (long i = from; i < min(rounds, from + kFold); ++i) {
      const long t = first + i * step;
      const bool have = t < p.T, keep = have && (!p.mask || p.mask[t] != 0);
      const int id = keep && g.lane < p.k ? __ldg(p.ids + (size_t)t * p.k + g.lane) : -1;
      float v[V];
      float m = -INFINITY;
#pragma unroll
      for (int c = 0; c < V; ++c) {
        v[c] = cur[c];
        m = fmaxf(m, v[c]);
      }
      load_row<L, NV, VEC>(cur, p.logits + (size_t)min(t + step, (long)p.T - 1) * p.ld, g.lane, p.E, -INFINITY);
      m = g.reduce(m, red[g.id], turn, fmax_op);
      if (m == -INFINITY) m = 0.f;               // a row of -inf: p = 0
      float s = 0.f;
#pragma unroll
      for (int c = 0; c < V; ++c) {
        v[c] = exp2_approx((v[c] - m) * kLog2e);   // 2 ulps, next to the 2^-24 |l - m| of any fp32 softmax
        s += v[c];
      }
      s = g.reduce(s, red[g.id], turn, add_op);
      const float inv = s == 0.f ? 0.f : 1.f / s;
      if (have && g.lane == 0) p.stats[t] = make_float2(m, inv);
      if (keep) {
#pragma unroll
        for (int c = 0; c < V; ++c) acc[c] = fmaf(v[c], inv, acc[c]);
        mine += g.lane == 0;
      }
      if (id >= 0 && id < p.E) atomicAdd(hist + id, 1);
    }
    // the groups' column sums, in the groups' order
    if (L < kWarp) {
#pragma unroll
      for (int c = 0; c < V; ++c) acc[c] += __shfl_xor_sync(0xffffffffu, acc[c], 16);
    }
    constexpr int kTurns = L < kWarp ? kFwdThreads / kWarp : kGroups;
    for (int w = 0; w < kTurns; ++w) {
      if (L < kWarp ? (int)threadIdx.x / kWarp == w && (threadIdx.x & 31) < L : g.id == w) {
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int c = column<L, VEC>(g.lane, j, i);
            if (c < p.E) sum_p[c] += acc[4 * j + i];
          }
      }
      __syncthreads();
    }
#pragma unroll
    for (int c = 0; c < V; ++c) acc[c] = 0.f;
  }
  griddep_launch_dependents();
  if (mine) atomicAdd(&tokens_s, mine);
  __syncthreads();
  if (gridDim.x > 1) {
    const size_t at = (size_t)blockIdx.x * p.pitch;
    for (int e = threadIdx.x; e < p.pitch; e += kFwdThreads) {
      p.part_p[at + e] = e < p.E ? sum_p[e] : 0.f;
      p.part_c[at + e] = e < p.E ? hist[e] : 0;
    }
    if (threadIdx.x == 0) p.part_n[blockIdx.x] = tokens_s;
    return;
  }
  // the only CTA: the whole result
  double l = 0.0;
  for (int e = threadIdx.x; e < p.E; e += kFwdThreads) {
    p.counts[e] = hist[e];
    l += (double)hist[e] * (double)sum_p[e];
  }
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
  if ((threadIdx.x & 31) == 0) loss_s[threadIdx.x >> 5] = l;
  __syncthreads();
  if (threadIdx.x == 0) {
    double a = 0.0;
    for (int w = 0; w < kFwdThreads / kWarp; ++w) a += loss_s[w];
    const double n = tokens_s;
    *p.tokens = tokens_s;
    *p.loss = n > 0 ? (float)((double)p.coef * p.E * a / (n * n * p.k)) : 0.f;
  }
}

// An fp32 sum and what its additions lost (Knuth's two-sum): 48 bits at the
// price of six fp32 additions, of which this GPU does 64 times as many as fp64
// ones (with these the join of 304 parts of 896 took 25 us).
struct Sum {
  float s = 0.f, lost = 0.f;
  __device__ __forceinline__ void add(float a) {
    const float t = __fadd_rn(s, a), z = __fadd_rn(t, -s);
    lost = __fadd_rn(lost, __fadd_rn(__fadd_rn(s, -__fadd_rn(t, -z)), __fadd_rn(a, -z)));
    s = t;
  }
};

// Joins `parts` CTAs' sums: one cluster of CTAS, a share of the columns per CTA,
// four columns a thread, their parts in up to 32 slices; the loss's terms meet in
// CTA 0.  One CTA where that is no more than 256 KB to read, up to kJoinPitch columns.
constexpr int kJoinPitch = 4 * kFinalThreads;
template <int CTAS>
__global__ void __cluster_dims__(CTAS, 1, 1) __launch_bounds__(kFinalThreads)
balance_join_kernel(BalanceParams p, int parts) {
  namespace cg = cooperative_groups;
  __shared__ float2 slice_p[4][kFinalThreads];
  __shared__ int slice_c[4][kFinalThreads];
  __shared__ double warp_l[kFinalThreads / kWarp];
  __shared__ double cta_l[CTAS];
  __shared__ int tokens_s;
  if (CTAS > 1) cluster_arrive();                      // CTA 0 has begun before its shared memory is written
  if (threadIdx.x == 0) tokens_s = 0;
  griddep_wait();
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = CTAS > 1 ? (int)cluster.block_rank() : 0;
  const int quads = p.pitch / 4, cols = (quads + CTAS - 1) / CTAS, c0 = rank * cols, width = max(0, min(cols, quads - c0));
  const int slices = min(32, kFinalThreads / cols);      // at least one: cols <= kFinalThreads
  const int c = threadIdx.x % cols, s = threadIdx.x / cols;
  Sum a[4];
  int n[4] = {0, 0, 0, 0};
  if (c < width && s < slices) {
    const float4* pp = reinterpret_cast<const float4*>(p.part_p) + c0 + c;
    const int4* pc = reinterpret_cast<const int4*>(p.part_c) + c0 + c;
#pragma unroll 8
    for (int i = s; i < parts; i += slices) {
      const float4 v = __ldcg(pp + (size_t)i * quads);
      const int4 k = __ldcg(pc + (size_t)i * quads);
      a[0].add(v.x);
      a[1].add(v.y);
      a[2].add(v.z);
      a[3].add(v.w);
      n[0] += k.x;
      n[1] += k.y;
      n[2] += k.z;
      n[3] += k.w;
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    slice_p[j][threadIdx.x] = make_float2(a[j].s, a[j].lost);
    slice_c[j][threadIdx.x] = n[j];
  }
  __syncthreads();
  double l = 0.0;
  for (int o = threadIdx.x; o < 4 * width; o += kFinalThreads) {   // a column a thread
    const int q = o >> 2, j = o & 3, e = 4 * (c0 + q) + j;
    Sum t;
    float lost = 0.f;
    int k = 0;
    for (int i = 0; i < slices; ++i) {
      const float2 v = slice_p[j][i * cols + q];
      t.add(v.x);
      lost += v.y;
      k += slice_c[j][i * cols + q];
    }
    if (e < p.E) {
      p.counts[e] = k;
      l += (double)k * ((double)t.s + (double)(t.lost + lost));
    }
  }
  if (rank == 0 && (int)threadIdx.x < parts) atomicAdd(&tokens_s, __ldcg(p.part_n + threadIdx.x));
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
  if ((threadIdx.x & 31) == 0) warp_l[threadIdx.x >> 5] = l;
  __syncthreads();
  if (CTAS > 1) cluster_wait();
  if (threadIdx.x == 0) {
    double t = 0.0;
    for (int w = 0; w < kFinalThreads / kWarp; ++w) t += warp_l[w];
    *(CTAS > 1 ? cluster.map_shared_rank(&cta_l[rank], 0) : &cta_l[0]) = t;
  }
  if (CTAS > 1) cluster.sync();
  if (rank == 0 && threadIdx.x == 0) {
    double t = 0.0;
    for (int i = 0; i < CTAS; ++i) t += cta_l[i];
    const double tok = tokens_s;
    *p.tokens = tokens_s;
    *p.loss = tok > 0 ? (float)((double)p.coef * p.E * t / (tok * tok * p.k)) : 0.f;
  }
}
static_assert(kMaxExperts / 4 / kFinalCtas <= kFinalThreads && kJoinPitch / 4 <= kFinalThreads &&
                  fwd_ctas(1) * kMostSms <= kFinalThreads,
              "a thread per four columns, per part");

template <int L, int NV, bool VEC>
__global__ void __launch_bounds__(kBackThreads, back_ctas(NV))
router_back_kernel(RouterBackParams p) {
  constexpr int kGroups = kBackThreads / L, V = 4 * NV, kPitch = 4 * L * NV;
  extern __shared__ float4 smem4[];            // a row of the chosen slots' terms per group, zeros between rows
  __shared__ float red[kGroups][8];
  const Group<L> g;
  float* mine = reinterpret_cast<float*>(smem4) + g.id * kPitch;
  for (int c = g.lane; c < kPitch; c += L) mine[c] = 0.f;
  g.sync();
  // F_e = dloss coef E / n f_e of every column: in shared memory, the lanes' own in
  // registers would leave room for half the rows
  float* F_s = reinterpret_cast<float*>(smem4) + kGroups * kPitch;
  {
    const int n = p.tokens ? *p.tokens : 0;
    const float gl = p.dloss && n > 0 ? (float)((double)*p.dloss * p.coef * p.E / ((double)n * n * p.k)) : 0.f;
    for (int c = threadIdx.x; c < kPitch; c += kBackThreads) F_s[c] = p.dloss && c < p.E ? (float)p.counts[c] * gl : 0.f;
  }
  __syncthreads();
  auto F4 = [&](int j) { return columns<L, VEC>(F_s, g.lane, j); };
  int turn = 0;
  const long step = (long)gridDim.x * kGroups;
  const long first = (long)blockIdx.x * kGroups + g.id;
  const long rounds = (p.T - (long)blockIdx.x * kGroups + step - 1) / step;
  for (long i = 0; i < rounds; ++i) {
    const long t = first + i * step;
    float v[V];
    load_row<L, NV, VEC>(v, p.logits + (size_t)min(t, (long)p.T - 1) * p.ld, g.lane, p.E, -INFINITY);
    const bool have = t < p.T;
    const bool slot = have && p.dw && g.lane < p.k;
    const float2 st = have ? __ldg(p.stats + t) : make_float2(0.f, 0.f);
    int id = -1;
    float w = 0.f, dw = 0.f;
    if (slot) {
      const size_t at = (size_t)t * p.k + g.lane;
      id = __ldg(p.ids + at);
      if (id < 0 || id >= p.E) id = -1;
      else {
        w = __ldg(p.w + at);
        dw = __ldg(p.dw + at);
      }
    }
    const bool keep = have && (!p.mask || p.mask[t] != 0);
    if (!keep && dw == 0.f) w = 0.f;            // a padding token's weight may be NaN
    float dot = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const float4 F = F4(j);
#pragma unroll
      for (int c = 4 * j; c < 4 * j + 4; ++c) v[c] = exp2_approx((v[c] - st.x) * kLog2e) * st.y;
      dot = fmaf(F.x, v[4 * j], fmaf(F.y, v[4 * j + 1], fmaf(F.z, v[4 * j + 2], fmaf(F.w, v[4 * j + 3], dot))));
    }
    dot = g.reduce(dot, red[g.id], turn, add_op);
    float wd = 0.f;
    if (p.dw) {
      wd = g.reduce(w * dw, red[g.id], turn, add_op);
      float add = p.renorm ? w * (dw - wd) : w * dw;
      // an ID that a row names twice: its first lane takes the terms of all
      if (L < kWarp || g.lane < kWarp) {
        const int wl = threadIdx.x & 31;
        const unsigned same = __match_any_sync(0xffffffffu, id >= 0 ? id + (L < kWarp ? (wl & 16) << 16 : 0) : -1 - wl);
        bool lead = id >= 0;
        if (__any_sync(0xffffffffu, (same & (same - 1)) != 0)) {
          const float own = add;
          lead = lead && __ffs(same) - 1 == wl;
          add = 0.f;
          for (int q = 0; q < kWarp; ++q) {
            const float o = __shfl_sync(0xffffffffu, own, q);
            if (same >> q & 1) add += o;
          }
        }
        if (lead) mine[id] = add;
      }
      g.sync();
    }
    const float all = p.renorm ? 0.f : wd;
    const float sub = keep ? dot + all : all;   // p (F - dot) - p all
    if (!keep && all == 0.f) {                  // a padding token, whatever its logits hold
#pragma unroll
      for (int c = 0; c < V; ++c) v[c] = 0.f;
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float4 x = p.dw ? columns<L, VEC>(mine, g.lane, j) : make_float4(0.f, 0.f, 0.f, 0.f);
      const float4 F = keep ? F4(j) : make_float4(0.f, 0.f, 0.f, 0.f);
      x.x = fmaf(v[4 * j], F.x - sub, x.x);
      x.y = fmaf(v[4 * j + 1], F.y - sub, x.y);
      x.z = fmaf(v[4 * j + 2], F.z - sub, x.z);
      x.w = fmaf(v[4 * j + 3], F.w - sub, x.w);
      if (!have) continue;
      const int c = column<L, VEC>(g.lane, j, 0);
      float* o = p.out + (size_t)t * p.ldo + c;
      if (VEC) {
        if (c < p.E) *reinterpret_cast<float4*>(o) = x;
      } else {
        if (c < p.E) o[0] = x.x;
        if (c + L < p.E) o[L] = x.y;
        if (c + 2 * L < p.E) o[2 * L] = x.z;
        if (c + 3 * L < p.E) o[3 * L] = x.w;
      }
    }
    if (p.dw) {
      g.sync();
      if (id >= 0) mine[id] = 0.f;
      g.sync();
    }
  }
}

// The lanes of a row and the 16-byte pieces of a lane: two rows a warp up to
// 128 experts, a warp per row up to 1,024, four warps beyond.
template <class F>
cudaError_t with_shape(int E, bool vec, F&& f) {
  auto call = [&](auto l, auto nv) {
    return vec ? f(l, nv, std::integral_constant<bool, true>{}) : f(l, nv, std::integral_constant<bool, false>{});
  };
#define SITU_SHAPE(L, NV) return call(std::integral_constant<int, L>{}, std::integral_constant<int, NV>{})
  if (E <= 64) SITU_SHAPE(16, 1);
  if (E <= 128) SITU_SHAPE(16, 2);
  if (E <= 1024) {
    const int nv = (E + 127) / 128;
    if (nv <= 2) SITU_SHAPE(32, 2);
    if (nv <= 4) SITU_SHAPE(32, 4);
    if (nv <= 6) SITU_SHAPE(32, 6);
    if (nv == 7) SITU_SHAPE(32, 7);
    SITU_SHAPE(32, 8);
  }
  if (E <= 2048) SITU_SHAPE(128, 4);
  SITU_SHAPE(128, 8);
#undef SITU_SHAPE
}

// of the current device; without one, those that the sizes are asked for
int sms() {
  const int n = gg::sm_count();
  return n < 1 ? 152 : n < kMostSms ? n : kMostSms;
}
// CTAs for T rows: `ctas` to an SM, `more` where E is short and a group would take more than `many` rows
int grid_of(int T, int E, int threads, int ctas, int more, int many) {
  const int groups = threads / (E <= 128 ? 16 : E <= 1024 ? 32 : 128);
  const long rows = (T + groups - 1) / groups;
  const long n = sms(), most = n * (E <= 256 && rows > many * ctas * n ? more : ctas);
  return (int)(rows < 1 ? 1 : rows > most ? most : rows);
}
// One CTA does the whole forward up to this many rows per group: a second
// launch costs about 3 us, as do four rows in turn.
int forward_grid(int T, int E) {
  const int g = grid_of(T, E, kFwdThreads, fwd_ctas(8), fwd_ctas(1), kManyRows);
  return g <= 4 ? 1 : g;
}

bool bad(const void* q, uintptr_t mask) { return (reinterpret_cast<uintptr_t>(q) & mask) != 0; }

}  // namespace
}  // namespace situ

extern "C" size_t situ_moe_balance_loss_workspace_size(int32_t T, int32_t num_experts_total) {
  using namespace situ;
  if (T < 0 || T > SITU_GEMM_MAX_ROWS || num_experts_total < 1 || num_experts_total > kMaxExperts) return 0;
  if (forward_grid(T, num_experts_total) == 1) return 0;   // one CTA writes the result itself
  const size_t grid = (size_t)forward_grid(T, num_experts_total), pitch = (size_t)(num_experts_total + 3) / 4 * 4;
  return (grid * (2 * pitch + 1) * 4 + 15) / 16 * 16;
}

extern "C" situ_status situ_moe_balance_loss(const situ_balance_args* a, void* workspace, size_t workspace_bytes,
                                             void* stream) {
  using namespace situ;
  if (!a) return SITU_ERR_NULL_ARG;
  const int E = a->num_experts_total;
  if (a->T < 0 || a->T > SITU_GEMM_MAX_ROWS || E < 1 || E > kMaxExperts || a->top_k < 1 || a->top_k > SITU_MAX_TOP_K ||
      a->top_k > E || a->ld < E || a->ld > (int64_t)1 << 39)
    return SITU_ERR_BAD_SHAPE;
  const size_t need = situ_moe_balance_loss_workspace_size(a->T, E);
  if (!a->loss || !a->counts || !a->tokens || (need > 0 && !workspace)) return SITU_ERR_NULL_ARG;
  if (a->T > 0 && (!a->router_logits || !a->topk_ids || !a->row_stats)) return SITU_ERR_NULL_ARG;
  if (bad(a->router_logits, 3) || bad(a->topk_ids, 3) || bad(a->loss, 3) || bad(a->counts, 3) || bad(a->tokens, 3) ||
      bad(a->row_stats, 7) || bad(workspace, 15))
    return SITU_ERR_MISALIGNED;
  if (workspace_bytes < need) return SITU_ERR_WORKSPACE_TOO_SMALL;
  cudaStream_t st = (cudaStream_t)stream;
  const int grid = forward_grid(a->T, E);
  BalanceParams p;
  p.logits = a->router_logits;
  p.ld = (long)a->ld;
  p.ids = a->topk_ids;
  p.mask = a->mask;
  p.T = a->T;
  p.E = E;
  p.k = a->top_k;
  p.coef = a->coef;
  p.loss = a->loss;
  p.counts = a->counts;
  p.tokens = a->tokens;
  p.stats = reinterpret_cast<float2*>(a->row_stats);
  p.part_p = static_cast<float*>(workspace);
  p.pitch = (E + 3) / 4 * 4;
  p.part_c = reinterpret_cast<int32_t*>(p.part_p + (size_t)grid * p.pitch);
  p.part_n = p.part_c + (size_t)grid * p.pitch;
  auto join = [&](int parts) {
    return (size_t)parts * p.pitch * 8 <= 256 * 1024 && p.pitch <= kJoinPitch
               ? launch_pdl(balance_join_kernel<1>, dim3(1), dim3(kFinalThreads), 0, st, p, parts)
               : launch_pdl(balance_join_kernel<kFinalCtas>, dim3(kFinalCtas), dim3(kFinalThreads), 0, st, p, parts);
  };
  if (a->T == 0) return join(0) == cudaSuccess ? SITU_OK : SITU_ERR_CUDA;
  const bool vec = E % 4 == 0 && a->ld % 4 == 0 && !bad(a->router_logits, 15);
  cudaError_t e = with_shape(E, vec, [&](auto l, auto nv, auto v) {
    balance_kernel<l.value, nv.value, v.value><<<grid, kFwdThreads, (size_t)E * 8, st>>>(p);
    return cudaGetLastError();
  });
  if (e == cudaSuccess && grid > 1)
    e = join(grid);
  return e == cudaSuccess ? SITU_OK : SITU_ERR_CUDA;
}

extern "C" situ_status situ_moe_router_backward(const situ_router_backward_args* a, void* stream) {
  using namespace situ;
  if (!a) return SITU_ERR_NULL_ARG;
  const int E = a->num_experts_total;
  if (a->T < 0 || a->T > SITU_GEMM_MAX_ROWS || E < 1 || E > kMaxExperts || a->top_k < 1 || a->top_k > SITU_MAX_TOP_K ||
      a->top_k > E || a->ld < E || a->ldo < E || a->ld > (int64_t)1 << 39 || a->ldo > (int64_t)1 << 39)
    return SITU_ERR_BAD_SHAPE;
  if (a->renormalize != 0 && a->renormalize != 1) return SITU_ERR_UNSUPPORTED;
  if (a->T == 0) return SITU_OK;
  if (!a->router_logits || !a->row_stats || !a->dlogits || (a->dloss && (!a->counts || !a->tokens)) ||
      (a->dweights && (!a->topk_weights || !a->topk_ids)))
    return SITU_ERR_NULL_ARG;
  if (bad(a->router_logits, 3) || bad(a->topk_ids, 3) || bad(a->counts, 3) || bad(a->tokens, 3) || bad(a->dloss, 3) ||
      bad(a->topk_weights, 3) || bad(a->dweights, 3) || bad(a->dlogits, 3) || bad(a->row_stats, 7))
    return SITU_ERR_MISALIGNED;
  RouterBackParams p;
  p.logits = a->router_logits;
  p.ld = (long)a->ld;
  p.ids = a->topk_ids;
  p.mask = a->mask;
  p.T = a->T;
  p.E = E;
  p.k = a->top_k;
  p.renorm = a->renormalize;
  p.coef = a->coef;
  p.counts = a->counts;
  p.tokens = a->dloss ? a->tokens : nullptr;
  p.stats = reinterpret_cast<const float2*>(a->row_stats);
  p.dloss = a->dloss;
  p.w = a->topk_weights;
  p.dw = a->dweights;
  p.out = a->dlogits;
  p.ldo = (long)a->ldo;
  const bool vec = E % 4 == 0 && a->ld % 4 == 0 && a->ldo % 4 == 0 && !bad(a->router_logits, 15) && !bad(a->dlogits, 15);
  const cudaError_t e = with_shape(E, vec, [&](auto l, auto nv, auto v) {
    constexpr int kSmem = (kBackThreads / l.value + 1) * 4 * l.value * nv.value * 4;   // a row of each group, and F
    auto* k = router_back_kernel<l.value, nv.value, v.value>;
    if (kSmem > 44 * 1024) {   // 48 KB with the static part
      const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
      if (e != cudaSuccess) return e;
    }
    k<<<grid_of(p.T, E, kBackThreads, back_ctas(8), back_ctas(1), kManyBackRows), kBackThreads, kSmem, (cudaStream_t)stream>>>(p);
    return cudaGetLastError();
  });
  return e == cudaSuccess ? SITU_OK : SITU_ERR_CUDA;
}
