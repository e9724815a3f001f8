// lora.cu -- low-rank adapters of many requests beside a shared projection,
// and their gradients.
//
// Row i of x [S, K] takes adapter e = ids[i] (or the one whose rows
// [offsets[e], offsets[e + 1]) hold i), or none:
//   u[i] = x[i] A[e]^T            A [n, r, K]
//   y[i] = base[i] + s[e] u[i] B[e]^T     B [n, N, r]
// and from dy: v = s dy B, dx = dx0 + v A, dA[e] = v^T x, dB[e] = dy^T (s u)
// over e's rows.  r is small (8 to 128), so all of it is bound by the bytes of
// x, base and y and of the adapters in use: 2 r (K + N) operations a row
// against 2 K + 4 N bytes, 16 to 100 a byte.
//
// Few rows (a decode step): lora_row_kernel, a cluster of eight CTAs per row.
// Each CTA takes an eighth of u's sums and, after they have met in shared
// memory, an eighth of y's columns; its part of B is on its way into the L2
// meanwhile.  One launch, fp32 multiply-adds.
//
// More rows: two kernels on tiles of 64 rows.  shrink_kernel streams x and
// the adapter once into partial sums of u (split over K where there are few
// tiles); expand_kernel joins them and adds s u B^T to base.  Neighbouring rows
// of one request share an adapter, so a tile has one or a few: it goes through
// its distinct adapters and keeps, of each one's sums, its own rows.  Any order
// of rows works without sorting or copying them, and a row's result holds
// nothing of another adapter's weights, infinities or NaN among them.  At 16
// rows per warp's MMA, with the weights in shared memory by cp.async, mma.sync
// keeps up with the bytes: tcgen05 would need 128 rows of one adapter to a tile
// and operands copied to where it reads them.
//
// u enters the second product in 16 bits.  For 16-bit results it is rounded
// once (half an ulp of u, as y itself is); for fp32 results it goes as a sum of
// 16-bit terms, three in bf16 and two in f16, which hold 24 and 22 of its bits.
// f16 rows are brought to [2^14, 2^15) by a power of two first, taken out of the
// sums again, so that a u beyond f16 neither overflows nor vanishes.
#include "../../include/situ_moe.h"
#include "gemm_groups.cuh"

#include <cooperative_groups.h>

namespace situ {

using namespace gg;

namespace {

constexpr int kTile = 128;         // rows of a tile
constexpr int kChunk = 64;         // contraction elements of a stage (shrink)
constexpr int kStages = 4;         // of shrink
constexpr int kMaxStages = 3;      // of expand
constexpr int kCols = 128;         // columns of a step (expand)
constexpr int kMaxRank = 128;
constexpr int kCluster = 8;        // CTAs of a row
constexpr int kRowThreads = 256;

struct LoraParams {
  const int32_t *ids, *offsets;
  int S, C, r, n;                  // C: the other extent (contraction or columns)
  int r16;                         // r rounded up to 16
  int splits, chunks;              // shrink: parts of the contraction, stages in all
  float* part;                     // [splits][S][r]
  const float* scale;              // [n] or null
  const void* base;
  long ld_base;
  void* out;
  long ldo;
  void* u16;                       // [S, r] scaled, of the operands' type, or null
  int groups;                      // expand: column groups of a tile
  int stages, w_stage, u_bytes;    // shared memory: stages of w (expand), bytes of one, of u
  int* err;
};

// 16-bit terms that u is taken in
__host__ __device__ constexpr int terms_of(int dt, bool f32) { return !f32 ? 1 : dt == SITU_DT_BF16 ? 3 : 2; }

struct RowParams {
  const void *x, *a, *b, *base;
  void *out, *u16;
  long ldx, ld_base, ldo;
  const int32_t *ids, *offsets;
  const float* scale;
  int S, K, N, r, n;
};

__device__ __forceinline__ int adapter_of(const int32_t* ids, const int32_t* offsets, int n, int row) {
  if (ids) {
    const int e = __ldg(ids + row);
    return e >= 0 && e < n ? e : -1;
  }
  int lo = 0, hi = n + 1;          // the first entry beyond row lies in [lo, hi]
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(offsets + mid) > row) hi = mid;
    else lo = mid + 1;
  }
  return lo <= n ? lo - 1 : -1;
}

template <int DT>
__device__ __forceinline__ uint32_t pack16(float a, float b) {
  return DT == SITU_DT_BF16 ? f32x2_to_bf16x2(a, b) : pack_f16x2(a, b);
}
template <int DT>
__device__ __forceinline__ float lo16(uint32_t w) {
  return DT == SITU_DT_BF16 ? bf16_lo(w) : f16_to_f32(w & 0xFFFFu);
}
template <int DT>
__device__ __forceinline__ float hi16(uint32_t w) {
  return DT == SITU_DT_BF16 ? bf16_hi(w) : f16_to_f32(w >> 16);
}
template <int DT>
__device__ __forceinline__ float dot8(const uint4& a, const uint4& b, float acc) {
  const uint32_t u[4] = {a.x, a.y, a.z, a.w}, v[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    acc = fmaf(lo16<DT>(u[i]), lo16<DT>(v[i]), acc);
    acc = fmaf(hi16<DT>(u[i]), hi16<DT>(v[i]), acc);
  }
  return acc;
}

// --------------------------------------------------------------------------
// a row per cluster
// --------------------------------------------------------------------------

__device__ __forceinline__ void prefetch_l2(const void* p, long bytes) {
  if (bytes > 0) asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"((uint32_t)bytes) : "memory");
}

template <int DT, bool F32>
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kRowThreads)
lora_row_kernel(RowParams p) {
  namespace cg = cooperative_groups;
  constexpr int kWarps = kRowThreads / 32;
  __shared__ float part[kMaxRank / kCluster * kWarps];
  __shared__ float u_s[kMaxRank];
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank(), row = blockIdx.x / kCluster;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int e = adapter_of(p.ids, p.offsets, p.n, row);      // of the whole cluster
  const int n8 = p.N / 8, c0 = (int)((long)n8 * rank / kCluster) * 8, c1 = (int)((long)n8 * (rank + 1) / kCluster) * 8;
  const uint16_t* b = static_cast<const uint16_t*>(p.b) + ((size_t)max(e, 0) * p.N + c0) * p.r;
  const int dots = p.r / kCluster, per = dots < kWarps ? kWarps / dots : 1;
  cluster_arrive();                  // shared memory of a CTA that has not begun may not be written
  if (e >= 0) {
    if (threadIdx.x == 0) prefetch_l2(b, (long)(c1 - c0) * p.r * 2);
    if (threadIdx.x == 32 && p.base)
      prefetch_l2(static_cast<const uint8_t*>(p.base) + ((size_t)row * p.ld_base + c0) * (F32 ? 4 : 2),
                  (long)(c1 - c0) * (F32 ? 4 : 2));
    // this CTA's sums of u, r / 8 of them, each over `per` warps
    const uint4* x = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.x) + (size_t)row * p.ldx);
    const int pieces = p.K / 8, s = warp % per;
    for (int d = warp / per; d < dots; d += kWarps / per) {
      const uint4* a = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.a) +
                                                      ((size_t)e * p.r + rank * dots + d) * p.K);
      float acc[4] = {0.f, 0.f, 0.f, 0.f};
      int i = lane + 32 * s;
      for (; i + 96 * per < pieces; i += 128 * per) {
        uint4 xv[4], av[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          xv[j] = __ldg(x + i + 32 * per * j);
          av[j] = __ldg(a + i + 32 * per * j);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[j] = dot8<DT>(xv[j], av[j], acc[j]);
      }
      for (; i < pieces; i += 32 * per) acc[0] = dot8<DT>(__ldg(x + i), __ldg(a + i), acc[0]);
      float t = (acc[0] + acc[1]) + (acc[2] + acc[3]);
#pragma unroll
      for (int o = 16; o >= 1; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
      if (lane == 0) part[d * per + s] = t;
    }
    __syncthreads();
  }
  cluster_wait();
  if (e >= 0) {
    const float f = p.scale ? __ldg(p.scale + e) : 1.f;
    // to every CTA of the cluster
    for (int i = threadIdx.x; i < dots * kCluster; i += kRowThreads) {
      const int d = i / kCluster;
      float t = 0.f;
      for (int j = 0; j < per; ++j) t += part[d * per + j];
      *cluster.map_shared_rank(&u_s[rank * dots + d], i % kCluster) = t * f;
    }
  }
  cluster.sync();
  if (p.u16 && rank == 0 && (int)threadIdx.x < p.r)
    static_cast<uint16_t*>(p.u16)[(size_t)row * p.r + threadIdx.x] =
        e >= 0 ? (uint16_t)pack16<DT>(u_s[threadIdx.x], 0.f) : (uint16_t)0;
  const float* base32 = static_cast<const float*>(p.base);
  const uint16_t* base16 = static_cast<const uint16_t*>(p.base);
  for (int c = threadIdx.x; c < c1 - c0; c += kRowThreads) {
    float t = 0.f;
    if (e >= 0) {
      const uint4* w = reinterpret_cast<const uint4*>(b + (size_t)c * p.r);
#pragma unroll 2
      for (int j = 0; j < p.r / 8; ++j) {
        const uint4 v = __ldg(w + j);
        const float* q = u_s + 8 * j;
        t = fmaf(lo16<DT>(v.x), q[0], t);
        t = fmaf(hi16<DT>(v.x), q[1], t);
        t = fmaf(lo16<DT>(v.y), q[2], t);
        t = fmaf(hi16<DT>(v.y), q[3], t);
        t = fmaf(lo16<DT>(v.z), q[4], t);
        t = fmaf(hi16<DT>(v.z), q[5], t);
        t = fmaf(lo16<DT>(v.w), q[6], t);
        t = fmaf(hi16<DT>(v.w), q[7], t);
      }
    }
    const size_t at = (size_t)row * p.ldo + c0 + c, from = (size_t)row * p.ld_base + c0 + c;
    if (F32) {
      const float y = p.base ? base32[from] : 0.f;
      static_cast<float*>(p.out)[at] = e >= 0 ? y + t : y;
    } else {
      const uint16_t y = p.base ? base16[from] : (uint16_t)0;
      static_cast<uint16_t*>(p.out)[at] = e >= 0 ? (uint16_t)pack16<DT>(lo16<DT>(y) + t, 0.f) : y;
    }
  }
}

// --------------------------------------------------------------------------
// tiles of 128 rows
// --------------------------------------------------------------------------

// A tile's adapters: each row's (kNone: none, kNoRow: past the end), and the
// distinct ones in the order of their first rows.
constexpr int kNone = -1, kNoRow = -2;
struct Adapters {
  alignas(16) int of[kTile];   // row -> adapter
  int at[kTile];       // row -> its place in `list`, or kNone / kNoRow
  int list[kTile];
  uint32_t lead[kTile / 32];
  int count;
};
// by all threads of the block, kTile or more
__device__ __forceinline__ void find_adapters(Adapters& t, const LoraParams& p, int row0) {
  const int i = threadIdx.x;
  const bool mine = i < kTile;
  int e = kNoRow;
  if (mine) {
    e = row0 + i < p.S ? adapter_of(p.ids, p.offsets, p.n, row0 + i) : kNoRow;
    t.of[i] = e;
  }
  __syncthreads();
  const int e0 = t.of[0];
  if (__syncthreads_and(!mine || e == e0 || e == kNoRow)) {
    if (mine) t.at[i] = e >= 0 ? 0 : e;
    if (i == 0) {
      t.list[0] = e0;
      t.count = e0 >= 0 ? 1 : 0;
    }
    __syncthreads();
    return;
  }
  int first = i;       // the first row of this one's adapter
  if (mine && e >= 0) {
    const int4* of = reinterpret_cast<const int4*>(t.of);
    for (int j = 0; 4 * j < i; ++j) {
      const int4 v = of[j];
      const int f = v.x == e ? 0 : v.y == e ? 1 : v.z == e ? 2 : v.w == e ? 3 : 4;
      if (f < 4) {
        first = min(i, 4 * j + f);
        break;
      }
    }
  }
  if (mine) {
    __syncwarp();
    const uint32_t lead = __ballot_sync(0xffffffffu, e >= 0 && first == i);
    if ((i & 31) == 0) t.lead[i >> 5] = lead;
  }
  __syncthreads();
  if (mine) {
    int place = __popc(t.lead[first >> 5] & ((1u << (first & 31)) - 1u));
    for (int w = 0; w < first >> 5; ++w) place += __popc(t.lead[w]);
    t.at[i] = e >= 0 ? place : e;
    if (e >= 0 && first == i) t.list[place] = e;
    if (i == 0) t.count = __popc(t.lead[0]) + __popc(t.lead[1]) + __popc(t.lead[2]) + __popc(t.lead[3]);
  }
  __syncthreads();
}

// A ring whose length the launch chooses.
struct Turns {
  int n, s = 0, used = 0;
  uint32_t ph = 0;
  __device__ __forceinline__ explicit Turns(int stages) : n(stages) {}
  __device__ __forceinline__ bool again() const { return used == n; }   // the stage has been used before
  __device__ __forceinline__ void next() {
    if (used < n) ++used;
    if (++s == n) {
      s = 0;
      ph ^= 1;
    }
  }
  // wait(stage, parity) for the last use of each stage
  template <class Wait>
  __device__ __forceinline__ bool last(Wait&& wait) const {
    bool ok = true;
    for (int j = 0; j < used; ++j) ok = wait(j, j < s ? ph : ph ^ 1) && ok;
    return ok;
  }
};

constexpr int kXBytes = kTile * 128;          // 64 elements of 128 rows
constexpr int kTmemCols = 256;                // of a CTA: two CTAs per SM
constexpr int kShrinkThreads = 192;           // copies, MMAs, four epilogue warps
constexpr int kExpandThreads = 320;           // copies, MMAs, eight epilogue warps
constexpr int kEpiThreads = 256;
constexpr int kStagePitch = 36;               // floats of a row of a warp's 32 x 32 sums in shared memory

// D[128, N] of 16-bit operands in fp32; trans_b: B's N elements contiguous
__device__ __forceinline__ uint32_t idesc_of(bool bf16, bool trans_b, int N) {
  return (1u << 4) | (bf16 ? (1u << 7) | (1u << 10) : 0u) | (trans_b ? 1u << 16 : 0u) | ((uint32_t)(N >> 3) << 17) |
         ((uint32_t)(128 >> 4) << 24);
}

// part[split][i][j] = sum over the split's k of x[i, k] W[e(i)][j][k] (TRANS:
// W[e][k][j]): the tile's rows on the MMA's M side, an adapter's r on its N
// side, in TMEM columns of its own.  As many adapters as the columns hold share
// a pass over x.
template <int DT, bool TRANS>
__global__ void __launch_bounds__(kShrinkThreads)
shrink_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_w, const LoraParams p) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ Adapters ad;
  __shared__ uint64_t bars[4 * kStages + 3];
  __shared__ uint32_t holder[2];
  const uint32_t sbase = (saddr(smem_raw) + 1023) & ~1023u;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int row0 = blockIdx.x * kTile, split = blockIdx.y;
  const uint32_t bar0 = saddr(bars);
  auto xfull = [&](int s) { return bar0 + 8 * s; };
  auto xempty = [&](int s) { return bar0 + 8 * (kStages + s); };
  auto wfull = [&](int s) { return bar0 + 8 * (2 * kStages + s); };
  auto wempty = [&](int s) { return bar0 + 8 * (3 * kStages + s); };
  const uint32_t acc_full = bar0 + 8 * 4 * kStages, acc_empty = acc_full + 8, drain = acc_full + 16;
  if (tid == 0) {
    holder[1] = (uint32_t)*reinterpret_cast<volatile int*>(p.err);   // an earlier launch gave up a wait: no work then
    prefetch_map(&map_x);
    prefetch_map(&map_w);
    for (int s = 0; s < 4 * kStages; ++s) mbar_init(bar0 + 8 * s, 1);
    mbar_init(acc_full, 1);
    mbar_init(acc_empty, 4);
    mbar_init(drain, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) tmem_alloc<1>(saddr(holder), kTmemCols);
  find_adapters(ad, p, row0);
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = holder[0];
  const int nd = holder[1] != 0 ? 0 : ad.count, per = kTmemCols / p.r16;
  const int k0 = (int)((long)p.chunks * split / p.splits), k1 = (int)((long)p.chunks * (split + 1) / p.splits);
  const uint32_t wbase = sbase + kStages * kXBytes;
  const int wboxes = (p.r + 63) / 64;

  if (warp == 0) {
    // ---------------- copies ----------------
    const bool leader = elect_one();
    Turns x(kStages), w(kStages);
    bool ok = true;
    for (int d0 = 0; d0 < nd && ok; d0 += per) {
      const int d1 = min(nd, d0 + per);
      for (int k = k0; k < k1 && ok; ++k) {
        if (x.again() && !warp_wait(xempty(x.s), x.ph ^ 1, p.err, 81)) {
          ok = false;
          break;
        }
        if (leader) {
          mbar_expect_tx(xfull(x.s), kXBytes);
          copy_2d<1>(sbase + x.s * kXBytes, &map_x, k * kChunk, row0, xfull(x.s));
        }
        __syncwarp();
        x.next();
        for (int d = d0; d < d1; ++d, w.next()) {
          if (w.again() && !warp_wait(wempty(w.s), w.ph ^ 1, p.err, 82)) {
            ok = false;
            break;
          }
          if (leader) {
            const uint32_t to = wbase + w.s * p.w_stage;
            mbar_expect_tx(wfull(w.s), TRANS ? wboxes * 8192 : p.r16 * 128);
            if (!TRANS) copy_3d<1>(to, &map_w, k * kChunk, 0, ad.list[d], wfull(w.s));
            else
              for (int c = 0; c < wboxes; ++c) copy_3d<1>(to + 8192 * c, &map_w, 64 * c, k * kChunk, ad.list[d], wfull(w.s));
          }
          __syncwarp();
        }
      }
    }
    leave(
        ok,
        [&] {
          const bool a = x.last([&](int j, uint32_t ph) { return warp_wait(xempty(j), ph, p.err, 83); });
          return w.last([&](int j, uint32_t ph) { return warp_wait(wempty(j), ph, p.err, 84); }) && a;
        },
        [&] {
          x.last([&](int j, uint32_t ph) { return drain_wait(xfull(j), ph); });
          w.last([&](int j, uint32_t ph) { return drain_wait(wfull(j), ph); });
        });
  } else if (warp == 1) {
    // ---------------- MMAs ----------------
    const bool leader = elect_one();
    const uint32_t idesc = idesc_of(DT == SITU_DT_BF16, TRANS, p.r16);
    Turns x(kStages), w(kStages);
    bool ok = true;
    int pass = 0;
    for (int d0 = 0; d0 < nd && ok; d0 += per, ++pass) {
      const int d1 = min(nd, d0 + per);
      if (pass > 0 && !warp_wait(acc_empty, (pass - 1) & 1, p.err, 85)) {
        ok = false;
        break;
      }
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      for (int k = k0; k < k1 && ok; ++k, x.next()) {
        if (!warp_wait(xfull(x.s), x.ph, p.err, 86)) {
          ok = false;
          break;
        }
        const int steps = min(kChunk / 16, (p.C - k * kChunk + 15) >> 4);
        for (int d = d0; d < d1; ++d, w.next()) {
          if (!warp_wait(wfull(w.s), w.ph, p.err, 87)) {
            ok = false;
            break;
          }
          asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
          if (leader) {
            const uint32_t wa = wbase + w.s * p.w_stage;
            const uint64_t xd = sdesc(sbase + x.s * kXBytes), wd = TRANS ? sdesc_mn(wa, 8192) : sdesc(wa);
            for (int i = 0; i < steps; ++i)
              mma_f16<1>(tmem + (d - d0) * p.r16, xd + 2 * i, wd + (TRANS ? 128 : 2) * i, idesc, ((k - k0) | i) != 0);
            mma_commit(wempty(w.s));
            if (d + 1 == d1) mma_commit(xempty(x.s));
          }
          __syncwarp();
        }
      }
      if (ok) {
        if (leader) mma_commit(acc_full);
        __syncwarp();
      }
    }
    leave(
        ok, [&] { return w.last([&](int j, uint32_t ph) { return warp_wait(wempty(j), ph, p.err, 88); }); },
        [&] {
          if (leader) mma_commit(drain);
          __syncwarp();
          drain_wait(drain, 0);
        });
  } else {
    // ---------------- sums to memory, a row per lane ----------------
    const int q = warp & 3, at = ad.at[32 * q + lane], row = row0 + 32 * q + lane;
    float* out = p.part + ((size_t)split * p.S + row) * p.r;
    bool ok = true;
    int pass = 0;
    for (int d0 = 0; d0 < nd && ok; d0 += per, ++pass) {
      const int d1 = min(nd, d0 + per);
      ok = warp_wait(acc_full, pass & 1, p.err, 89);
      if (!ok) break;
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      for (int d = d0; d < d1; ++d) {
        if (!__any_sync(0xffffffffu, at == d)) continue;
        for (int j = 0; j < p.r16; j += 16) {
          uint32_t v[16];
          tmem_ld16_nowait(tmem + ((uint32_t)(32 * q) << 16) + (d - d0) * p.r16 + j, v);
          tmem_ld_wait<16>(v);
          if (at == d) {
#pragma unroll
            for (int i = 0; i < 16; i += 4)
              if (j + i < p.r)
                *reinterpret_cast<uint4*>(out + j + i) = make_uint4(v[i], v[i + 1], v[i + 2], v[i + 3]);
          }
        }
      }
      asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
      mbar_arrive_if(acc_empty, lane == 0);
    }
  }
  griddep_launch_dependents();
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    tmem_free<1>(tmem, kTmemCols);
  }
}

// out[i][c] = base[i][c] + s[e] sum_j u[i][j] W[e][c][j] (TRANS: W[e][j][c]),
// u the sum of its parts: the tile's rows on the MMA's M side, 128 columns on
// its N side, u in shared memory for all the CTA's columns (its 16-bit terms
// one after the other along the contraction).  The sums go through shared memory
// into the order in which 16 bytes a lane of base and out are coalesced.
template <int DT, bool TRANS, bool F32>
__global__ void __launch_bounds__(kExpandThreads)
expand_kernel(const __grid_constant__ CUtensorMap map_w, const LoraParams p) {
  constexpr int kTerms = terms_of(DT, F32);
  extern __shared__ uint8_t smem_raw[];
  __shared__ Adapters ad;
  __shared__ float back[kTile];      // f16: the power of two that a row's u was divided by
  __shared__ uint64_t bars[2 * kMaxStages + 6];
  __shared__ uint32_t holder[2];
  uint8_t* smem = smem_raw + (((saddr(smem_raw) + 1023) & ~1023u) - saddr(smem_raw));
  const uint32_t sbase = saddr(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int row0 = blockIdx.x * kTile;
  const uint32_t bar0 = saddr(bars);
  auto full = [&](int s) { return bar0 + 8 * s; };
  auto empty = [&](int s) { return bar0 + 8 * (kMaxStages + s); };
  auto acc_full = [&](int b) { return bar0 + 8 * (2 * kMaxStages + b); };
  auto acc_empty = [&](int b) { return bar0 + 8 * (2 * kMaxStages + 2 + b); };
  const uint32_t u_full = bar0 + 8 * (2 * kMaxStages + 4), drain = u_full + 8;
  if (tid == 0) {
    prefetch_map(&map_w);
    for (int s = 0; s < 2 * kMaxStages; ++s) mbar_init(bar0 + 8 * s, 1);
    for (int b = 0; b < 2; ++b) {
      mbar_init(acc_full(b), 1);
      mbar_init(acc_empty(b), kEpiThreads / 32);
    }
    mbar_init(u_full, kEpiThreads / 32);
    mbar_init(drain, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) tmem_alloc<1>(saddr(holder), kTmemCols);
  find_adapters(ad, p, row0);
  griddep_wait();                    // the parts, and the status, are the predecessor's
  if (tid == 0) holder[1] = (uint32_t)*reinterpret_cast<volatile int*>(p.err);
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = holder[0];
  const bool dead = holder[1] != 0;
  const int nd = dead ? 0 : ad.count;
  const int blocks = (p.C + kCols - 1) / kCols;
  const int b0 = (int)((long)blocks * blockIdx.y / p.groups), b1 = (int)((long)blocks * (blockIdx.y + 1) / p.groups);
  const uint32_t ubase = sbase, wbase = sbase + p.u_bytes;
  const int rboxes = (p.r + 63) / 64, steps = p.r16 / 16;

  if (warp == 0) {
    // ---------------- copies ----------------
    const bool leader = elect_one();
    Turns w(p.stages);
    bool ok = true;
    const int rrows = min(64, p.r16);                   // TRANS: contraction rows of a box
    for (int b = b0; b < b1 && ok; ++b)
      for (int d = 0; d < nd; ++d, w.next()) {
        if (w.again() && !warp_wait(empty(w.s), w.ph ^ 1, p.err, 91)) {
          ok = false;
          break;
        }
        if (leader) {
          const uint32_t to = wbase + w.s * p.w_stage;
          const int c0 = b * kCols, e = ad.list[d];
          if (!TRANS) {
            mbar_expect_tx(full(w.s), rboxes * kXBytes);
            for (int i = 0; i < rboxes; ++i) copy_3d<1>(to + i * kXBytes, &map_w, 64 * i, c0, e, full(w.s));
          } else {
            mbar_expect_tx(full(w.s), rboxes * 2 * rrows * 128);
            for (int i = 0; i < rboxes; ++i)
              for (int h = 0; h < 2; ++h)
                copy_3d<1>(to + (2 * i + h) * rrows * 128, &map_w, c0 + 64 * h, 64 * i, e, full(w.s));
          }
        }
        __syncwarp();
      }
    leave(
        ok, [&] { return w.last([&](int j, uint32_t ph) { return warp_wait(empty(j), ph, p.err, 92); }); },
        [&] { w.last([&](int j, uint32_t ph) { return drain_wait(full(j), ph); }); });
  } else if (warp == 1) {
    // ---------------- MMAs ----------------
    const bool leader = elect_one();
    const uint32_t idesc = idesc_of(DT == SITU_DT_BF16, TRANS, kCols);
    const uint32_t rrows = (uint32_t)min(64, p.r16);
    Turns w(p.stages), acc(2);
    bool ok = nd == 0 || b0 == b1 || warp_wait(u_full, 0, p.err, 93);
    for (int b = b0; b < b1 && ok; ++b)
      for (int d = 0; d < nd; ++d, w.next(), acc.next()) {
        if ((acc.again() && !warp_wait(acc_empty(acc.s), acc.ph ^ 1, p.err, 94)) || !warp_wait(full(w.s), w.ph, p.err, 95)) {
          ok = false;
          break;
        }
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        if (leader) {
          const uint32_t wa = wbase + w.s * p.w_stage;
          for (int t = kTerms - 1; t >= 0; --t)         // the smallest term first
            for (int i = 0; i < steps; ++i) {
              const int k = t * steps + i;              // sixteens along u's terms
              const uint64_t ud = sdesc(ubase + (k >> 2) * kXBytes) + 2 * (k & 3);
              const uint64_t wd = TRANS ? sdesc_mn(wa + (i >> 2) * 2 * rrows * 128, rrows * 128) + 128 * (i & 3)
                                        : sdesc(wa + (i >> 2) * kXBytes) + 2 * (i & 3);
              mma_f16<1>(tmem + acc.s * kCols, ud, wd, idesc, t != kTerms - 1 || i != 0);
            }
          mma_commit(empty(w.s));
          mma_commit(acc_full(acc.s));
        }
        __syncwarp();
      }
    leave(
        ok, [&] { return w.last([&](int j, uint32_t ph) { return warp_wait(empty(j), ph, p.err, 96); }); },
        [&] {
          if (leader) mma_commit(drain);
          __syncwarp();
          drain_wait(drain, 0);
        });
  } else if (!dead) {
    const int et = tid - 64;
    {
      // u of the tile: two threads to a row, eight elements of each sixteen each
      const int i = et >> 1, row = row0 + i, e = ad.of[i];
      const float f = e >= 0 && p.scale ? __ldg(p.scale + e) : 1.f;
      const bool write = p.u16 && blockIdx.y == 0 && e != kNoRow;
      auto sum8 = [&](int j, float (&u)[8]) {
#pragma unroll
        for (int k = 0; k < 8; ++k) u[k] = 0.f;
        if (e < 0 || j >= p.r) return;
        for (int s = 0; s < p.splits; ++s) {
          const float4* src = reinterpret_cast<const float4*>(p.part + ((size_t)s * p.S + row) * p.r + j);
          const float4 v = __ldcg(src), w = __ldcg(src + 1);
          u[0] += v.x;
          u[1] += v.y;
          u[2] += v.z;
          u[3] += v.w;
          u[4] += w.x;
          u[5] += w.y;
          u[6] += w.z;
          u[7] += w.w;
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) u[k] *= f;
      };
      float to = 1.f;
      if (DT == SITU_DT_F16) {
        float m = 0.f;
        for (int j = 8 * (et & 1); j < p.r16; j += 16) {
          float u[8];
          sum8(j, u);
#pragma unroll
          for (int k = 0; k < 8; ++k) m = fmaxf(m, fabsf(u[k]));
        }
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
        const int k = (int)(__float_as_uint(m) >> 23) - 127;          // m in [2^k, 2^(k + 1))
        const int ex = m > 0.f && m < INFINITY ? max(-100, min(120, k - 14)) : 0;
        to = exp2i(-ex);
        if ((et & 1) == 0) back[i] = exp2i(ex);
      }
      for (int j = 8 * (et & 1); j < p.r16; j += 16) {
        float u[8];
        sum8(j, u);
        if (write && j < p.r)
          *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.u16) + (size_t)row * p.r + j) =
              make_uint4(pack16<DT>(u[0], u[1]), pack16<DT>(u[2], u[3]), pack16<DT>(u[4], u[5]), pack16<DT>(u[6], u[7]));
#pragma unroll
        for (int t = 0; t < kTerms; ++t) {
          uint32_t v[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float a = u[2 * k] * (t == 0 ? to : 1.f), b = u[2 * k + 1] * (t == 0 ? to : 1.f);
            v[k] = pack16<DT>(a, b);
            // what the term leaves; an infinity leaves nothing
            u[2 * k] = fabsf(a) < INFINITY ? a - lo16<DT>(v[k]) : 0.f;
            u[2 * k + 1] = fabsf(b) < INFINITY ? b - hi16<DT>(v[k]) : 0.f;
          }
          const int k = t * p.r16 + j;                  // along u's terms: 128-byte swizzled rows of 64
          *reinterpret_cast<uint4*>(smem + (k >> 6) * kXBytes + i * 128 + ((((k & 63) >> 3) ^ (i & 7)) << 4)) =
              make_uint4(v[0], v[1], v[2], v[3]);
        }
      }
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    asm volatile("bar.sync 1, 256;" ::: "memory");      // back[] and, before the barrier below, every lane's u
    mbar_arrive_if(u_full, lane == 0);

    // ---------------- sums to memory ----------------
    const int q = warp & 3, h = (warp - 2) >> 2;        // this warp's 32 rows, and 64 of the 128 columns
    constexpr int kEl = F32 ? 4 : 2, kLanes = F32 ? 8 : 4, kRows = 32 / kLanes, kIts = kLanes;   // lanes per row of 32 columns
    const uint8_t* base = static_cast<const uint8_t*>(p.base);
    uint8_t* out = static_cast<uint8_t*>(p.out);
    float* stage = reinterpret_cast<float*>(smem + p.u_bytes + p.stages * p.w_stage) + (warp - 2) * 32 * kStagePitch;
    const int my_at = ad.at[32 * q + lane];
    const float my_back = DT == SITU_DT_F16 ? back[32 * q + lane] : 1.f;
    const int r_in = lane / kLanes, c_in = lane % kLanes * (16 / kEl);
    auto place = [&](int it, int col, long ld) {        // of 16 bytes: bytes from the array's start
      return ((size_t)(row0 + 32 * q + it * kRows + r_in) * (size_t)ld + col + c_in) * kEl;
    };
    // rows without an adapter take base as it is
    if (p.base != p.out && __any_sync(0xffffffffu, my_at == kNone)) {
      for (int b = b0; b < b1; ++b)
        for (int c = 0; c < 64; c += 32) {
          const int col = b * kCols + 64 * h + c;
#pragma unroll
          for (int it = 0; it < kIts; ++it)
            if (ad.at[32 * q + it * kRows + r_in] == kNone && col + c_in < p.C)
              *reinterpret_cast<uint4*>(out + place(it, col, p.ldo)) =
                  base ? *reinterpret_cast<const uint4*>(base + place(it, col, p.ld_base)) : make_uint4(0, 0, 0, 0);
        }
    }
    Turns acc(2);
    bool ok = true;
    for (int b = b0; b < b1 && ok; ++b)
      for (int d = 0; d < nd; ++d, acc.next()) {
        const bool work = __any_sync(0xffffffffu, my_at == d);
        uint4 y[2][kIts];
        if (work) {
          // base on its way while the sums are made
#pragma unroll
          for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int it = 0; it < kIts; ++it) {
              const int col = b * kCols + 64 * h + 32 * c;
              y[c][it] = base && ad.at[32 * q + it * kRows + r_in] == d && col + c_in < p.C
                             ? *reinterpret_cast<const uint4*>(base + place(it, col, p.ld_base))
                             : make_uint4(0, 0, 0, 0);
            }
        }
        if (!warp_wait(acc_full(acc.s), acc.ph, p.err, 97)) {
          ok = false;
          break;
        }
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        if (work) {
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int col = b * kCols + 64 * h + 32 * c;
            uint32_t v[32];
            tmem_ld32_nowait(tmem + ((uint32_t)(32 * q) << 16) + acc.s * kCols + 64 * h + 32 * c, v);
            tmem_ld_wait<32>(v);
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 32; i += 4)
              *reinterpret_cast<float4*>(stage + lane * kStagePitch + i) =
                  make_float4(__uint_as_float(v[i]) * my_back, __uint_as_float(v[i + 1]) * my_back,
                              __uint_as_float(v[i + 2]) * my_back, __uint_as_float(v[i + 3]) * my_back);
            __syncwarp();
#pragma unroll
            for (int it = 0; it < kIts; ++it) {
              const int r = it * kRows + r_in;
              if (ad.at[32 * q + r] != d || col + c_in >= p.C) continue;
              const float* src = stage + r * kStagePitch + c_in;
              const float4 a = *reinterpret_cast<const float4*>(src);
              uint4 o = y[c][it];
              if (F32) {
                o.x = __float_as_uint(__uint_as_float(o.x) + a.x);
                o.y = __float_as_uint(__uint_as_float(o.y) + a.y);
                o.z = __float_as_uint(__uint_as_float(o.z) + a.z);
                o.w = __float_as_uint(__uint_as_float(o.w) + a.w);
              } else {
                const float4 e = *reinterpret_cast<const float4*>(src + 4);
                o.x = pack16<DT>(lo16<DT>(o.x) + a.x, hi16<DT>(o.x) + a.y);
                o.y = pack16<DT>(lo16<DT>(o.y) + a.z, hi16<DT>(o.y) + a.w);
                o.z = pack16<DT>(lo16<DT>(o.z) + e.x, hi16<DT>(o.z) + e.y);
                o.w = pack16<DT>(lo16<DT>(o.w) + e.z, hi16<DT>(o.w) + e.w);
              }
              *reinterpret_cast<uint4*>(out + place(it, col, p.ldo)) = o;
            }
          }
        }
        asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
        mbar_arrive_if(acc_empty(acc.s), lane == 0);
      }
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    tmem_free<1>(tmem, kTmemCols);
  }
}

// --------------------------------------------------------------------------
// launches
// --------------------------------------------------------------------------

// Parts of the contraction: two CTAs per SM, parts of at least two stages.  For
// fp32 results a part is 1,024 elements at most: the tensor cores truncate when
// they add (6e-9 of a sum of one sign per element), the parts meet in fp32.
int splits_of(int S, int C, bool f32) {
  const int tiles = (S + kTile - 1) / kTile, chunks = (C + kChunk - 1) / kChunk;
  int s = 2 * 152 / tiles;
  if (s > chunks / 2) s = chunks / 2;
  if (f32 && s < (chunks + 15) / 16) s = (chunks + 15) / 16;
  return s < 1 ? 1 : s;
}

template <int DT, bool TRANS, bool F32>
cudaError_t launch_pair(const CUtensorMap& mx, const CUtensorMap& mw, const LoraParams& s, const CUtensorMap& mo, LoraParams x,
                        cudaStream_t st) {
  auto* shrink = shrink_kernel<DT, TRANS>;
  auto* expand = expand_kernel<DT, TRANS, F32>;
  const unsigned tiles = (unsigned)((s.S + kTile - 1) / kTile);
  const int shrink_smem = 1024 + kStages * (kXBytes + s.w_stage);
  x.u_bytes = (terms_of(DT, F32) * x.r16 + 63) / 64 * kXBytes;
  const int rest = 1024 + x.u_bytes + kEpiThreads / 32 * 32 * kStagePitch * 4;
  x.stages = rest + 3 * x.w_stage <= 108 * 1024 || rest + 2 * x.w_stage > 108 * 1024 ? 3 : 2;   // two CTAs per SM where that does it
  if (rest + x.stages * x.w_stage > 224 * 1024) x.stages = 2;
  const int expand_smem = rest + x.stages * x.w_stage;
  // in every call, so that a context created anew has them too
  cudaError_t e = cudaFuncSetAttribute(shrink, cudaFuncAttributeMaxDynamicSharedMemorySize, 160 * 1024);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(expand, cudaFuncAttributeMaxDynamicSharedMemorySize, 224 * 1024);
  if (e != cudaSuccess) return e;
  shrink<<<dim3(tiles, (unsigned)s.splits), kShrinkThreads, shrink_smem, st>>>(mx, mw, s);
  e = cudaGetLastError();
  return e != cudaSuccess ? e : launch_pdl(expand, dim3(tiles, (unsigned)x.groups), dim3(kExpandThreads), expand_smem, st, mo, x);
}

// x [S, C] times the adapters' w [n, r, C] (TRANS: [n, C, r]), and that times
// the other factor [n, C', r] (TRANS: [n, r, C']), onto out.
template <bool TRANS>
situ_status launch_tiles(int dtype, bool f32, const void* rows, int64_t ld_rows, const void* w, const void* other, LoraParams s,
                         LoraParams x, cudaStream_t st) {
  const uint64_t S = (uint64_t)s.S, C = (uint64_t)s.C, O = (uint64_t)x.C, r = (uint64_t)s.r, n = (uint64_t)s.n;
  s.r16 = x.r16 = (s.r + 15) / 16 * 16;
  s.chunks = (s.C + kChunk - 1) / kChunk;
  s.splits = x.splits = splits_of(s.S, s.C, f32);
  const int boxes = (s.r + 63) / 64;
  s.w_stage = boxes * 8192;
  const int rrows = s.r16 < 64 ? s.r16 : 64;
  x.w_stage = TRANS ? boxes * 2 * rrows * 128 : boxes * kXBytes;
  const int tiles = (s.S + kTile - 1) / kTile, blocks = (x.C + kCols - 1) / kCols;
  // column groups: about four CTAs per SM, of two blocks or more (u is read and laid out by each)
  const int groups = (4 * 152 + tiles - 1) / tiles, most = blocks > 2 ? blocks / 2 : 1;
  x.groups = groups < most ? groups : most;
  const CUtensorMapDataType dt = dtype == SITU_DT_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  CUtensorMap mx, mw, mo;
  const uint64_t dx[2] = {C, S}, sx[1] = {(uint64_t)ld_rows * 2};
  const uint32_t bx[2] = {64, kTile};
  bool ok = make_map_nd(&mx, dt, rows, 2, dx, sx, bx);
  if (TRANS) {
    const uint64_t dw[3] = {r, C, n}, sw[2] = {r * 2, r * C * 2}, dof[3] = {O, r, n}, so[2] = {O * 2, r * O * 2};
    const uint32_t bw[3] = {64, kChunk, 1}, bo[3] = {64, (uint32_t)rrows, 1};
    ok = ok && make_map_nd(&mw, dt, w, 3, dw, sw, bw) && make_map_nd(&mo, dt, other, 3, dof, so, bo);
  } else {
    const uint64_t dw[3] = {C, r, n}, sw[2] = {C * 2, r * C * 2}, dof[3] = {r, O, n}, so[2] = {r * 2, r * O * 2};
    const uint32_t bw[3] = {64, (uint32_t)s.r16, 1}, bo[3] = {64, kCols, 1};
    ok = ok && make_map_nd(&mw, dt, w, 3, dw, sw, bw) && make_map_nd(&mo, dt, other, 3, dof, so, bo);
  }
  if (!ok) return SITU_ERR_CUDA;
  constexpr int kB = SITU_DT_BF16, kF = SITU_DT_F16;
  const cudaError_t e = dtype == kB ? (f32 ? launch_pair<kB, TRANS, true>(mx, mw, s, mo, x, st)
                                           : launch_pair<kB, TRANS, false>(mx, mw, s, mo, x, st))
                                    : (f32 ? launch_pair<kF, TRANS, true>(mx, mw, s, mo, x, st)
                                           : launch_pair<kF, TRANS, false>(mx, mw, s, mo, x, st));
  return e == cudaSuccess ? SITU_OK : SITU_ERR_CUDA;
}

// A cluster per row, or tiles.
bool by_rows(int S) { return S <= 64; }

// for either type of result
size_t part_bytes(int S, int C, int r) { return S == 0 ? 0 : (size_t)splits_of(S, C, true) * S * r * 4; }

bool bad(const void* q, uintptr_t mask) { return (reinterpret_cast<uintptr_t>(q) & mask) != 0; }
bool bad_ld(int64_t ld, int64_t cols, int64_t unit) { return ld < cols || ld % unit != 0 || ld > (int64_t)1 << 39; }
bool bad_extent(int C) { return C < 8 || C % 8 != 0 || C > SITU_GEMM_MAX_DIM; }
bool bad_sizes(int S, int K, int N, int r, int n) {
  return S < 0 || S > SITU_GEMM_MAX_ROWS || bad_extent(K) || bad_extent(N) || r < 8 || r % 8 != 0 || r > kMaxRank || n < 1 ||
         n > SITU_LORA_MAX_ADAPTERS;
}

}  // namespace
}  // namespace situ

extern "C" size_t situ_moe_lora_workspace_size(int32_t S, int32_t K, int32_t N, int32_t r) {
  using namespace situ;
  if (bad_sizes(S, K, N, r, 1)) return 0;
  return S == 0 || by_rows(S) ? 16 : part_bytes(S, K, r);
}

extern "C" situ_status situ_moe_lora(const situ_lora_args* a, void* workspace, size_t workspace_bytes, void* stream) {
  using namespace situ;
  if (!a) return SITU_ERR_NULL_ARG;
  if ((a->dtype != SITU_DT_BF16 && a->dtype != SITU_DT_F16) || (a->out_dtype != a->dtype && a->out_dtype != SITU_DT_F32))
    return SITU_ERR_UNSUPPORTED;
  const int f32 = a->out_dtype == SITU_DT_F32;
  if (bad_sizes(a->S, a->K, a->N, a->r, a->n) || bad_ld(a->ldx, a->K, 8) || bad_ld(a->ldo, a->N, f32 ? 4 : 8) ||
      (a->base && bad_ld(a->ld_base, a->N, f32 ? 4 : 8)))
    return SITU_ERR_BAD_SHAPE;
  if (a->S == 0) return SITU_OK;
  if (!a->x || !a->a || !a->b || !a->out || !a->ids == !a->offsets) return SITU_ERR_NULL_ARG;
  if (bad(a->x, 15) || bad(a->a, 15) || bad(a->b, 15) || bad(a->base, 15) || bad(a->out, 15) || bad(a->u, 15) ||
      bad(a->ids, 3) || bad(a->offsets, 3) || bad(a->scale, 3))
    return SITU_ERR_MISALIGNED;
  cudaStream_t st = (cudaStream_t)stream;
  if (by_rows(a->S)) {
    RowParams p;
    p.x = a->x;
    p.a = a->a;
    p.b = a->b;
    p.base = a->base;
    p.out = a->out;
    p.u16 = a->u;
    p.ldx = (long)a->ldx;
    p.ld_base = (long)a->ld_base;
    p.ldo = (long)a->ldo;
    p.ids = a->ids;
    p.offsets = a->offsets;
    p.scale = a->scale;
    p.S = a->S;
    p.K = a->K;
    p.N = a->N;
    p.r = a->r;
    p.n = a->n;
    auto launch = [&](auto k) { k<<<(unsigned)a->S * kCluster, kRowThreads, 0, st>>>(p); };
    if (a->dtype == SITU_DT_BF16)
      f32 ? launch(lora_row_kernel<SITU_DT_BF16, true>) : launch(lora_row_kernel<SITU_DT_BF16, false>);
    else
      f32 ? launch(lora_row_kernel<SITU_DT_F16, true>) : launch(lora_row_kernel<SITU_DT_F16, false>);
    return cudaGetLastError() == cudaSuccess ? SITU_OK : SITU_ERR_CUDA;
  }
  if (!workspace || !a->device_status) return SITU_ERR_NULL_ARG;
  if (bad(workspace, 15) || bad(a->device_status, 3)) return SITU_ERR_MISALIGNED;
  if (workspace_bytes < part_bytes(a->S, a->K, a->r)) return SITU_ERR_WORKSPACE_TOO_SMALL;
  LoraParams s = {};
  s.ids = a->ids;
  s.offsets = a->offsets;
  s.S = a->S;
  s.r = a->r;
  s.n = a->n;
  s.part = static_cast<float*>(workspace);
  s.scale = a->scale;
  s.err = a->device_status;
  LoraParams x = s;
  s.C = a->K;
  x.C = a->N;
  x.base = a->base;
  x.ld_base = (long)a->ld_base;
  x.out = a->out;
  x.ldo = (long)a->ldo;
  x.u16 = a->u;
  return launch_tiles<false>(a->dtype, f32 != 0, a->x, a->ldx, a->a, a->b, s, x, st);
}

extern "C" size_t situ_moe_lora_backward_workspace_size(int32_t S, int32_t K, int32_t N, int32_t r) {
  using namespace situ;
  if (bad_sizes(S, K, N, r, 1)) return 0;
  return part_bytes(S, N, r) + ((size_t)S * r * 2 + 15) / 16 * 16 + 16;
}

extern "C" situ_status situ_moe_lora_backward(const situ_lora_backward_args* a, void* workspace, size_t workspace_bytes,
                                              void* stream) {
  using namespace situ;
  if (!a) return SITU_ERR_NULL_ARG;
  if ((a->dtype != SITU_DT_BF16 && a->dtype != SITU_DT_F16) || (a->dx_dtype != a->dtype && a->dx_dtype != SITU_DT_F32))
    return SITU_ERR_UNSUPPORTED;
  const int f32 = a->dx_dtype == SITU_DT_F32;
  if (bad_sizes(a->S, a->K, a->N, a->r, a->n) || a->n > SITU_GEMM_MAX_GROUPS || bad_ld(a->ld_dy, a->N, 8) ||
      bad_ld(a->ldx, a->K, 8) || bad_ld(a->ld_dx, a->K, f32 ? 4 : 8) || (a->dx0 && bad_ld(a->ld_dx0, a->K, f32 ? 4 : 8)))
    return SITU_ERR_BAD_SHAPE;
  if (!a->da || !a->db || !a->offsets || !a->device_status || !workspace) return SITU_ERR_NULL_ARG;
  if (a->S > 0 && (!a->dy || !a->x || !a->a || !a->b || !a->u || !a->dx)) return SITU_ERR_NULL_ARG;
  const void* ptrs[] = {a->dy, a->x, a->a, a->b, a->u, a->dx0, a->dx, a->da, a->db, workspace};
  for (const void* q : ptrs)
    if (bad(q, 15)) return SITU_ERR_MISALIGNED;
  if (bad(a->offsets, 3) || bad(a->scale, 3) || bad(a->device_status, 3)) return SITU_ERR_MISALIGNED;
  if (workspace_bytes < situ_moe_lora_backward_workspace_size(a->S, a->K, a->N, a->r)) return SITU_ERR_WORKSPACE_TOO_SMALL;
  uint8_t* v = static_cast<uint8_t*>(workspace) + part_bytes(a->S, a->N, a->r);
  if (a->S > 0) {
    LoraParams s = {};
    s.offsets = a->offsets;
    s.S = a->S;
    s.r = a->r;
    s.n = a->n;
    s.part = static_cast<float*>(workspace);
    s.scale = a->scale;
    s.err = a->device_status;
    LoraParams x = s;
    s.C = a->N;
    x.C = a->K;
    x.base = a->dx0;
    x.ld_base = (long)a->ld_dx0;
    x.out = a->dx;
    x.ldo = (long)a->ld_dx;
    x.u16 = v;
    const situ_status t =
        launch_tiles<true>(a->dtype, f32 != 0, a->dy, a->ld_dy, a->b, a->a, s, x, (cudaStream_t)stream);
    if (t != SITU_OK) return t;
  }
  // over an adapter's rows: dA = v^T x, dB = dy^T u
  situ_grouped_gemm_args g = {};
  g.direction = SITU_GROUPED_WGRAD;
  g.dtype = g.out_dtype = a->dtype;
  g.S = a->S;
  g.E = a->n;
  g.offsets = a->offsets;
  g.device_status = a->device_status;
  g.a = v;
  g.lda = g.N = a->r;
  g.b = a->x;
  g.ldb = a->ldx;
  g.K = a->K;
  g.out = a->da;
  g.ldo = a->K;
  const situ_status st = situ_moe_grouped_gemm(&g, stream);
  if (st != SITU_OK) return st;
  g.a = a->dy;
  g.lda = a->ld_dy;
  g.N = a->N;
  g.b = a->u;
  g.ldb = g.K = a->r;
  g.out = a->db;
  g.ldo = a->r;
  return situ_moe_grouped_gemm(&g, stream);
}
