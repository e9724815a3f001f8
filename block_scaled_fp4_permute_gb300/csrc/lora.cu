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
#include "situ_internal.h"

#include <cooperative_groups.h>

namespace situ {

namespace {

constexpr int kTile = 64;          // rows of a tile, 16 per warp
constexpr int kTileThreads = 128;
constexpr int kChunk = 64;         // contraction elements of a stage (shrink)
constexpr int kStages = 4;
constexpr int kCols = 128;         // columns of a step (expand)
constexpr int kMaxRank = 128;
constexpr int kCluster = 8;        // CTAs of a row
constexpr int kRowThreads = 256;

struct LoraParams {
  const void* x;                   // shrink's rows
  long ldx;
  const void* w;                   // this kernel's adapter factor
  const int32_t *ids, *offsets;
  int S, C, r, n;                  // C: the other extent (contraction or columns)
  int splits, chunks;              // shrink: parts of the contraction, stages in all
  float* part;                     // [splits][S][r]
  const float* scale;              // [n] or null
  const void* base;
  long ld_base;
  void* out;
  long ldo;
  void* u16;                       // [S, r] scaled, of the operands' type, or null
  int groups;                      // expand: column groups of a tile
};

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
// tiles of 64 rows
// --------------------------------------------------------------------------

__device__ __forceinline__ uint32_t smem_at(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
// 16 bytes to shared memory, zeros where `have` is false
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool have) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(have ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void* src, bool have) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(have ? 4 : 0) : "memory");
}
__device__ __forceinline__ void commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void wait_copies() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
template <bool TRANS>
__device__ __forceinline__ void ldmatrix4(uint32_t (&d)[4], uint32_t at) {
  if (TRANS)
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(d[0]), "=r"(d[1]), "=r"(d[2]), "=r"(d[3]) : "r"(at) : "memory");
  else
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(d[0]), "=r"(d[1]), "=r"(d[2]), "=r"(d[3]) : "r"(at) : "memory");
}
template <int DT>
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if (DT == SITU_DT_BF16)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// A tile's adapters: each row's (kNone: none, kNoRow: past the end), and the
// distinct ones in the order of their first rows.
constexpr int kNone = -1, kNoRow = -2;
struct Adapters {
  int of[kTile];       // row -> adapter
  int at[kTile];       // row -> its place in `list`, or kNone / kNoRow
  int list[kTile];
  int count;
};
__device__ __forceinline__ void find_adapters(Adapters& t, const LoraParams& p, int row0) {
  const int i = threadIdx.x;
  if (i < kTile) t.of[i] = row0 + i < p.S ? adapter_of(p.ids, p.offsets, p.n, row0 + i) : kNoRow;
  __syncthreads();
  const bool same = __syncthreads_and(i >= kTile || t.of[i] == t.of[0] || t.of[i] == kNoRow);
  if (same) {
    if (i < kTile) t.at[i] = t.of[i] >= 0 ? 0 : t.of[i];
    if (i == 0) {
      t.list[0] = t.of[0];
      t.count = t.of[0] >= 0 ? 1 : 0;
    }
  } else if (i < 32) {
    // the first row of each adapter, by the first warp: rows i and i + 32
    int first[2];
    unsigned lead[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int e = t.of[i + 32 * h];
      first[h] = i + 32 * h;
      for (int j = 0; j < i + 32 * h; ++j)
        if (t.of[j] == e) {
          first[h] = j;
          break;
        }
      lead[h] = __ballot_sync(0xffffffffu, e >= 0 && first[h] == i + 32 * h);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int e = t.of[i + 32 * h], f = first[h];
      const int place = f < 32 ? __popc(lead[0] & ((1u << f) - 1u))
                               : __popc(lead[0]) + __popc(lead[1] & ((1u << (f - 32)) - 1u));
      t.at[i + 32 * h] = e >= 0 ? place : e;
      if (e >= 0 && f == i + 32 * h) t.list[place] = e;
    }
    if (i == 0) t.count = __popc(lead[0]) + __popc(lead[1]);
  }
  __syncthreads();
}
// Which of a tile's adapters the warp's 16 rows take (bit d: list[d]).
__device__ __forceinline__ uint64_t adapters_of_warp(const Adapters& t) {
  const int lane = threadIdx.x & 31, a = t.at[(threadIdx.x >> 5) * 16 + (lane & 15)];
  const uint32_t lo = __reduce_or_sync(0xffffffffu, a >= 0 && a < 32 ? 1u << a : 0u);
  const uint32_t hi = __reduce_or_sync(0xffffffffu, a >= 32 ? 1u << (a - 32) : 0u);
  return (uint64_t)hi << 32 | lo;
}

constexpr int kXPitch = kChunk + 8;   // elements: 144 bytes, ldmatrix without conflicts

template <int RP, bool TRANS>
struct ShrinkCfg {
  static constexpr int kWPitch = TRANS ? RP + 8 : kXPitch;
  static constexpr int kWRows = TRANS ? kChunk : RP;
  static constexpr int kXBytes = kTile * kXPitch * 2, kWBytes = kWRows * kWPitch * 2;
  static constexpr int kSmem = kStages * (kXBytes + kWBytes);
};

// part[split][i][j] = sum over the split's k of x[i, k] W[e(i)][j][k] (TRANS: W[e][k][j]).
template <int DT, int RP, bool TRANS>
__global__ void __launch_bounds__(kTileThreads)
shrink_kernel(LoraParams p) {
  using Cfg = ShrinkCfg<RP, TRANS>;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ Adapters ad;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int row0 = blockIdx.x * kTile, split = blockIdx.y;
  find_adapters(ad, p, row0);
  const int nd = ad.count;
  const int k0 = (int)((long)p.chunks * split / p.splits), k1 = (int)((long)p.chunks * (split + 1) / p.splits);
  const int total = nd * (k1 - k0), pairs = (p.r + 15) / 16;
  const uint32_t xs = smem_at(smem), ws = xs + kStages * Cfg::kXBytes;
  const uint16_t* x = static_cast<const uint16_t*>(p.x);
  const uint16_t* w = static_cast<const uint16_t*>(p.w);
  // the step that is copied next: chunk and place in the list
  int lk = k0, ld = 0;
  auto load = [&](int stage) {
    const int c0 = lk * kChunk;
    if (ld == 0) {                   // a chunk of x serves all the adapters
      const uint32_t at = xs + (lk - k0) % kStages * Cfg::kXBytes;
#pragma unroll
      for (int i = 0; i < kTile * kChunk / 8 / kTileThreads; ++i) {
        const int piece = tid + i * kTileThreads, r = piece / (kChunk / 8), c = piece % (kChunk / 8) * 8;
        const bool have = row0 + r < p.S && c0 + c < p.C;
        copy16(at + (r * kXPitch + c) * 2, have ? x + (size_t)(row0 + r) * p.ldx + c0 + c : x, have);
      }
    }
    const uint16_t* we = w + (size_t)ad.list[ld] * p.r * p.C;
    const uint32_t at = ws + stage * Cfg::kWBytes;
    if (!TRANS) {
      for (int piece = tid; piece < pairs * 16 * (kChunk / 8); piece += kTileThreads) {
        const int r = piece / (kChunk / 8), c = piece % (kChunk / 8) * 8;
        const bool have = r < p.r && c0 + c < p.C;
        copy16(at + (r * Cfg::kWPitch + c) * 2, have ? we + (size_t)r * p.C + c0 + c : we, have);
      }
    } else {
      const int per = pairs * 2;
      for (int piece = tid; piece < kChunk * per; piece += kTileThreads) {
        const int c = piece / per, r = piece % per * 8;
        const bool have = r < p.r && c0 + c < p.C;
        copy16(at + (c * Cfg::kWPitch + r) * 2, have ? we + (size_t)(c0 + c) * p.r + r : we, have);
      }
    }
    if (++ld == nd) {
      ld = 0;
      ++lk;
    }
  };
  float acc[RP / 8][4];
#pragma unroll
  for (int t = 0; t < RP / 8; ++t)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[t][i] = 0.f;
  const uint64_t mine = adapters_of_warp(ad);
  const int at0 = ad.at[warp * 16 + (lane >> 2)], at1 = ad.at[warp * 16 + (lane >> 2) + 8];
  const bool one = (mine & (mine - 1)) == 0;
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) {
    if (s < total) load(s);
    commit();
  }
  int k = k0, d = 0;
  for (int i = 0; i < total; ++i) {
    wait_copies<kStages - 2>();
    __syncthreads();
    if (i + kStages - 1 < total) load((i + kStages - 1) % kStages);
    commit();
    if (mine >> d & 1) {
      const uint32_t xa = xs + (k - k0) % kStages * Cfg::kXBytes +
                          ((warp * 16 + (lane & 15)) * kXPitch + (lane >> 4) * 8) * 2;
      const uint32_t wa = ws + i % kStages * Cfg::kWBytes;
      float t[RP / 8][4];
#pragma unroll
      for (int j = 0; j < RP / 8; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) t[j][q] = acc[j][q];
#pragma unroll
      for (int ks = 0; ks < kChunk / 16; ++ks) {
        uint32_t a[4];
        ldmatrix4<false>(a, xa + ks * 32);
#pragma unroll
        for (int j = 0; j < RP / 16; ++j) {
          if (j >= pairs) break;
          uint32_t b[4];
          if (!TRANS)
            ldmatrix4<false>(b, wa + ((j * 16 + (lane >> 4) * 8 + (lane & 7)) * Cfg::kWPitch + ks * 16 + ((lane >> 3) & 1) * 8) * 2);
          else
            ldmatrix4<true>(b, wa + ((ks * 16 + ((lane >> 3) & 1) * 8 + (lane & 7)) * Cfg::kWPitch + j * 16 + (lane >> 4) * 8) * 2);
          mma<DT>(t[2 * j], a, b[0], b[1]);
          mma<DT>(t[2 * j + 1], a, b[2], b[3]);
        }
      }
      // of several adapters' sums each row keeps its own
#pragma unroll
      for (int j = 0; j < RP / 8; ++j) {
        if (one || at0 == d) {
          acc[j][0] = t[j][0];
          acc[j][1] = t[j][1];
        }
        if (one || at1 == d) {
          acc[j][2] = t[j][2];
          acc[j][3] = t[j][3];
        }
      }
    }
    if (++d == nd) {
      d = 0;
      ++k;
    }
  }
  wait_copies<0>();
  griddep_launch_dependents();
  // rows of no adapter give zeros
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int at = h ? at1 : at0, row = row0 + warp * 16 + (lane >> 2) + 8 * h;
    if (at == kNoRow) continue;
    float* o = p.part + ((size_t)split * p.S + row) * p.r + (lane & 3) * 2;
#pragma unroll
    for (int j = 0; j < RP / 8; ++j)
      if (8 * j < p.r)
        *reinterpret_cast<float2*>(o + 8 * j) =
            at >= 0 ? make_float2(acc[j][2 * h], acc[j][2 * h + 1]) : make_float2(0.f, 0.f);
  }
}

template <int DT, int RP, bool TRANS, bool F32>
struct ExpandCfg {
  static constexpr int kTerms = !F32 ? 1 : DT == SITU_DT_BF16 ? 3 : 2;
  static constexpr int kUPitch = RP + 8;
  static constexpr int kUBytes = kTile * kUPitch * 2;                // of a term
  static constexpr int kWPitch = TRANS ? kCols + 8 : RP + 8;
  static constexpr int kWBytes = (TRANS ? RP : kCols) * kWPitch * 2;
  static constexpr int kSmem = kTerms * kUBytes + 2 * kWBytes;
};

// Where a column goes in shared memory: 8q + 2t + i of each 32 to 8t + 2q + i.
__device__ __forceinline__ int dealt(int c) { return (c & ~30) + (c & 6) * 4 + (c & 24) / 4; }

// out[i][c] = base[i][c] + s[e] sum_j u[i][j] W[e][c][j] (TRANS: W[e][j][c]),
// u the sum of its parts.
//
// The MMA's columns are dealt out so that a thread's sums of four of its
// 8-column tiles are eight neighbours of a row: 16-byte loads of base and
// stores of out straight from registers.
template <int DT, int RP, bool TRANS, bool F32>
__global__ void __launch_bounds__(kTileThreads)
expand_kernel(LoraParams p) {
  using Cfg = ExpandCfg<DT, RP, TRANS, F32>;
  constexpr int kTerms = Cfg::kTerms;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ Adapters ad;
  __shared__ float back[kTile];      // f16: the power of two that a row's u was divided by
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int row0 = blockIdx.x * kTile;
  find_adapters(ad, p, row0);
  const int nd = ad.count, pairs = (p.r + 15) / 16;
  const int blocks = (p.C + kCols - 1) / kCols;
  const int b0 = (int)((long)blocks * blockIdx.y / p.groups), b1 = (int)((long)blocks * (blockIdx.y + 1) / p.groups);
  const int total = nd * (b1 - b0);
  const uint32_t us = smem_at(smem), ws = us + kTerms * Cfg::kUBytes;
  const uint16_t* w = static_cast<const uint16_t*>(p.w);
  int lb = b0, ld = 0;
  auto load = [&](int stage) {
    const uint16_t* we = w + (size_t)ad.list[ld] * p.r * p.C;
    const int c0 = lb * kCols;
    const uint32_t at = ws + stage * Cfg::kWBytes;
    if (!TRANS) {
      const int per = pairs * 2;
      for (int piece = tid; piece < kCols * per; piece += kTileThreads) {
        const int c = piece / per, r = piece % per * 8;
        const bool have = r < p.r && c0 + c < p.C;
        copy16(at + (dealt(c) * Cfg::kWPitch + r) * 2, have ? we + (size_t)(c0 + c) * p.r + r : we, have);
      }
    } else {
      for (int piece = tid; piece < pairs * 16 * (kCols / 2); piece += kTileThreads) {
        const int r = piece / (kCols / 2), c = piece % (kCols / 2) * 2;
        const bool have = r < p.r && c0 + c < p.C;
        copy4(at + (r * Cfg::kWPitch + dealt(c)) * 2, have ? we + (size_t)r * p.C + c0 + c : we, have);
      }
    }
    if (++ld == nd) {
      ld = 0;
      ++lb;
    }
  };
  if (total > 0) load(0);
  commit();
  griddep_wait();                    // the parts are the predecessor's output
  {
    // two threads to a row, half of its u each
    const int i = tid >> 1, half = RP / 2, j0 = (tid & 1) * half, row = row0 + i;
    const int e = ad.of[i];
    float u[RP / 2];
#pragma unroll
    for (int j = 0; j < half; ++j) u[j] = 0.f;
    if (e >= 0) {
      for (int s = 0; s < p.splits; ++s) {
        const float* src = p.part + ((size_t)s * p.S + row) * p.r + j0;
#pragma unroll
        for (int j = 0; j < half; j += 4) {
          if (j0 + j >= p.r) break;
          const float4 v = __ldcg(reinterpret_cast<const float4*>(src + j));
          u[j] += v.x;
          u[j + 1] += v.y;
          u[j + 2] += v.z;
          u[j + 3] += v.w;
        }
      }
      const float f = p.scale ? __ldg(p.scale + e) : 1.f;
#pragma unroll
      for (int j = 0; j < half; ++j) u[j] *= f;
    }
    if (p.u16 && blockIdx.y == 0 && e != kNoRow) {
      uint32_t* o = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.u16) + (size_t)row * p.r + j0);
#pragma unroll
      for (int j = 0; j < half; j += 2)
        if (j0 + j < p.r) o[j / 2] = pack16<DT>(u[j], u[j + 1]);
    }
    if (DT == SITU_DT_F16) {
      float m = 0.f;
#pragma unroll
      for (int j = 0; j < half; ++j) m = fmaxf(m, fabsf(u[j]));
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
      const int k = (int)(__float_as_uint(m) >> 23) - 127;            // m in [2^k, 2^(k + 1))
      const int ex = m > 0.f && m < INFINITY ? max(-100, min(120, k - 14)) : 0;
      const float to = exp2i(-ex);
#pragma unroll
      for (int j = 0; j < half; ++j) u[j] *= to;
      if ((tid & 1) == 0) back[i] = exp2i(ex);
    }
#pragma unroll
    for (int t = 0; t < kTerms; ++t) {
#pragma unroll
      for (int j = 0; j < half; j += 2) {
        const uint32_t v = pack16<DT>(u[j], u[j + 1]);
        *reinterpret_cast<uint32_t*>(smem + t * Cfg::kUBytes + (i * Cfg::kUPitch + j0 + j) * 2) = v;
        if (t + 1 < kTerms) {        // what the term leaves; an infinity leaves nothing
          u[j] = fabsf(u[j]) < INFINITY ? u[j] - lo16<DT>(v) : 0.f;
          u[j + 1] = fabsf(u[j + 1]) < INFINITY ? u[j + 1] - hi16<DT>(v) : 0.f;
        }
      }
    }
  }
  const uint64_t mine = adapters_of_warp(ad);
  const int g = lane >> 2, q = lane & 3;
  int at[2];
  size_t from[2], to[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int i = warp * 16 + g + 8 * h;
    at[h] = ad.at[i];
    from[h] = (size_t)(row0 + i) * p.ld_base;
    to[h] = (size_t)(row0 + i) * p.ldo;
  }
  __syncthreads();
  const float f0 = DT == SITU_DT_F16 ? back[warp * 16 + g] : 1.f, f1 = DT == SITU_DT_F16 ? back[warp * 16 + g + 8] : 1.f;
  constexpr int kEl = F32 ? 4 : 2, kVec = F32 ? 2 : 1;   // bytes of an element; 16-byte pieces of eight
  const uint8_t* base = static_cast<const uint8_t*>(p.base);
  uint8_t* out = static_cast<uint8_t*>(p.out);
  // rows without an adapter take base as it is
  if (p.base != p.out && (at[0] == kNone || at[1] == kNone)) {
    for (int b = b0; b < b1; ++b)
#pragma unroll
      for (int s = 0; s < kCols / 32; ++s) {
        const int c = b * kCols + 32 * s + 8 * q;
        if (c >= p.C) break;
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (at[h] == kNone)
#pragma unroll
            for (int v = 0; v < kVec; ++v)
              *reinterpret_cast<uint4*>(out + (to[h] + c) * kEl + 16 * v) =
                  base ? *reinterpret_cast<const uint4*>(base + (from[h] + c) * kEl + 16 * v) : make_uint4(0, 0, 0, 0);
      }
  }
  int b = b0, d = 0;
  for (int i = 0; i < total; ++i) {
    const bool work = mine >> d & 1;
    // base on its way while the weights arrive
    uint4 y[kCols / 32][2][kVec];
    if (work && base) {
#pragma unroll
      for (int s = 0; s < kCols / 32; ++s) {
        const int c = b * kCols + 32 * s + 8 * q;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int v = 0; v < kVec; ++v)
            y[s][h][v] = at[h] == d && c < p.C ? *reinterpret_cast<const uint4*>(base + (from[h] + c) * kEl + 16 * v)
                                               : make_uint4(0, 0, 0, 0);
      }
    } else {
#pragma unroll
      for (int s = 0; s < kCols / 32; ++s)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int v = 0; v < kVec; ++v) y[s][h][v] = make_uint4(0, 0, 0, 0);
    }
    wait_copies<0>();
    __syncthreads();
    if (i + 1 < total) load((i + 1) & 1);
    commit();
    if (work) {
      const uint32_t wa = ws + (i & 1) * Cfg::kWBytes;
      float acc[kCols / 8][4];
#pragma unroll
      for (int t = 0; t < kCols / 8; ++t)
#pragma unroll
        for (int v = 0; v < 4; ++v) acc[t][v] = 0.f;
#pragma unroll 1
      for (int ks = 0; ks < pairs; ++ks) {
        uint32_t a[kTerms][4];
#pragma unroll
        for (int t = 0; t < kTerms; ++t)
          ldmatrix4<false>(a[t], us + t * Cfg::kUBytes + ((warp * 16 + (lane & 15)) * Cfg::kUPitch + ks * 16 + (lane >> 4) * 8) * 2);
#pragma unroll
        for (int j = 0; j < kCols / 16; ++j) {      // tiles 2j and 2j + 1
          uint32_t f[4];
          if (!TRANS) {
            ldmatrix4<false>(f, wa + ((j * 16 + (lane >> 4) * 8 + (lane & 7)) * Cfg::kWPitch + ks * 16 + ((lane >> 3) & 1) * 8) * 2);
          } else {
            ldmatrix4<true>(f, wa + ((ks * 16 + ((lane >> 3) & 1) * 8 + (lane & 7)) * Cfg::kWPitch + j * 16 + (lane >> 4) * 8) * 2);
          }
#pragma unroll
          for (int t = kTerms - 1; t >= 0; --t) {   // the smallest first
            mma<DT>(acc[2 * j], a[t], f[0], f[1]);
            mma<DT>(acc[2 * j + 1], a[t], f[2], f[3]);
          }
        }
      }
#pragma unroll
      for (int s = 0; s < kCols / 32; ++s) {
        const int c = b * kCols + 32 * s + 8 * q;
        if (c >= p.C) break;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (at[h] != d) continue;
          const float f = h ? f1 : f0;
          uint4 o[kVec];
          uint32_t* ow = reinterpret_cast<uint32_t*>(o);
          const uint32_t* yw = reinterpret_cast<const uint32_t*>(y[s][h]);
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            const float e0 = acc[4 * s + t][2 * h] * f, e1 = acc[4 * s + t][2 * h + 1] * f;
            if (F32) {
              ow[2 * t] = __float_as_uint(__uint_as_float(yw[2 * t]) + e0);
              ow[2 * t + 1] = __float_as_uint(__uint_as_float(yw[2 * t + 1]) + e1);
            } else {
              ow[t] = pack16<DT>(lo16<DT>(yw[t]) + e0, hi16<DT>(yw[t]) + e1);
            }
          }
#pragma unroll
          for (int v = 0; v < kVec; ++v) *reinterpret_cast<uint4*>(out + (to[h] + c) * kEl + 16 * v) = o[v];
        }
      }
    }
    if (++d == nd) {
      d = 0;
      ++b;
    }
  }
  wait_copies<0>();
}

// --------------------------------------------------------------------------
// launches
// --------------------------------------------------------------------------

// Tiles of rows times parts of the contraction: about three CTAs per SM, parts
// of at least two stages, and partial sums (4 r splits bytes a row) of an
// eighth of the row's bytes at most.
int splits_of(int S, int C, int r) {
  const int tiles = (S + kTile - 1) / kTile, chunks = (C + kChunk - 1) / kChunk;
  int s = (3 * 152 + tiles - 1) / tiles;
  const int most = S > 2 * kTile ? C / (16 * r) : 32;
  s = s < most ? s : most;
  s = s < chunks / 2 ? s : chunks / 2;
  return s < 1 ? 1 : s;
}

// Raises a kernel's shared memory limit: in every call, so that a context
// created anew has it too.
template <class K>
cudaError_t allow_smem(K* kernel, int bytes) {
  if (bytes <= 44 * 1024) return cudaSuccess;   // 48 KB with the static part
  return cudaFuncSetAttribute(reinterpret_cast<const void*>(kernel), cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

template <int DT, int RP, bool TRANS>
cudaError_t launch_shrink(const LoraParams& p, cudaStream_t st) {
  auto* k = shrink_kernel<DT, RP, TRANS>;
  constexpr int smem = ShrinkCfg<RP, TRANS>::kSmem;
  const cudaError_t e = allow_smem(k, smem);
  if (e != cudaSuccess) return e;
  k<<<dim3((unsigned)((p.S + kTile - 1) / kTile), (unsigned)p.splits), kTileThreads, smem, st>>>(p);
  return cudaGetLastError();
}
template <int DT, int RP, bool TRANS, bool F32>
cudaError_t launch_expand(const LoraParams& p, cudaStream_t st) {
  auto* k = expand_kernel<DT, RP, TRANS, F32>;
  constexpr int smem = ExpandCfg<DT, RP, TRANS, F32>::kSmem;
  const cudaError_t e = allow_smem(k, smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(k, dim3((unsigned)((p.S + kTile - 1) / kTile), (unsigned)p.groups), dim3(kTileThreads), smem, st, p);
}

template <int RP, bool TRANS>
cudaError_t launch_pair(int dtype, int out_f32, const LoraParams& s, const LoraParams& x, cudaStream_t st) {
  constexpr int kB = SITU_DT_BF16, kF = SITU_DT_F16;
  cudaError_t e = dtype == kB ? launch_shrink<kB, RP, TRANS>(s, st) : launch_shrink<kF, RP, TRANS>(s, st);
  if (e != cudaSuccess) return e;
  if (out_f32) return dtype == kB ? launch_expand<kB, RP, TRANS, true>(x, st) : launch_expand<kF, RP, TRANS, true>(x, st);
  return dtype == kB ? launch_expand<kB, RP, TRANS, false>(x, st) : launch_expand<kF, RP, TRANS, false>(x, st);
}
template <bool TRANS>
cudaError_t launch_tiles(int dtype, int out_f32, LoraParams s, LoraParams x, cudaStream_t st) {
  s.chunks = (s.C + kChunk - 1) / kChunk;
  s.splits = x.splits = splits_of(s.S, s.C, s.r);
  const int tiles = (s.S + kTile - 1) / kTile, blocks = (x.C + kCols - 1) / kCols;
  const int groups = (8 * 152 + tiles - 1) / tiles;        // about eight CTAs per SM
  x.groups = groups < blocks ? groups : blocks;
  if (s.r <= 16) return launch_pair<16, TRANS>(dtype, out_f32, s, x, st);
  if (s.r <= 32) return launch_pair<32, TRANS>(dtype, out_f32, s, x, st);
  if (s.r <= 64) return launch_pair<64, TRANS>(dtype, out_f32, s, x, st);
  return launch_pair<128, TRANS>(dtype, out_f32, s, x, st);
}

// A cluster per row, or tiles.
bool by_rows(int S) { return S <= 64; }

size_t part_bytes(int S, int C, int r) { return ((size_t)splits_of(S, C, r) * S * r * 4 + 15) / 16 * 16; }

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
  if (!workspace) return SITU_ERR_NULL_ARG;
  if (bad(workspace, 15)) return SITU_ERR_MISALIGNED;
  if (workspace_bytes < part_bytes(a->S, a->K, a->r)) return SITU_ERR_WORKSPACE_TOO_SMALL;
  LoraParams s = {};
  s.ids = a->ids;
  s.offsets = a->offsets;
  s.S = a->S;
  s.r = a->r;
  s.n = a->n;
  s.part = static_cast<float*>(workspace);
  s.scale = a->scale;
  LoraParams x = s;
  s.x = a->x;
  s.ldx = (long)a->ldx;
  s.w = a->a;
  s.C = a->K;
  x.w = a->b;
  x.C = a->N;
  x.base = a->base;
  x.ld_base = (long)a->ld_base;
  x.out = a->out;
  x.ldo = (long)a->ldo;
  x.u16 = a->u;
  return launch_tiles<false>(a->dtype, f32, s, x, st) == cudaSuccess ? SITU_OK : SITU_ERR_CUDA;
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
    LoraParams x = s;
    s.x = a->dy;
    s.ldx = (long)a->ld_dy;
    s.w = a->b;
    s.C = a->N;
    x.w = a->a;
    x.C = a->K;
    x.base = a->dx0;
    x.ld_base = (long)a->ld_dx0;
    x.out = a->dx;
    x.ldo = (long)a->ld_dx;
    x.u16 = v;
    if (launch_tiles<true>(a->dtype, f32, s, x, (cudaStream_t)stream) != cudaSuccess) return SITU_ERR_CUDA;
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
