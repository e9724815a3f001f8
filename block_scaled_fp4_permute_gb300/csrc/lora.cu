// lora.cu -- low-rank adapters of many requests beside a shared projection, and
// the gradient of their input.
//
// Row i of x [S, K] takes adapter e = ids[i] (or the one whose rows
// [offsets[e], offsets[e + 1]) hold i), or none:
//   u[i] = s[e] x[i] A[e]^T          A [n, r, K]
//   y[i] = base[i] + u[i] B[e]^T     B [n, N, r]
// and from dy: v = s dy B, dx = dx0 + v A (lora_grads.cu has dA and dB).  r is
// small (8 to 128), so all of it is bound by the bytes of x, base and y and of the
// adapters in use: 2 r (K + N) operations a row against 2 K + 4 N bytes.
//
// Few rows (a decode step): lora_row_kernel, a cluster of eight CTAs per row.
// Each CTA takes an eighth of u's sums and, after they have met in shared
// memory, an eighth of y's columns; its part of B is on its way into the L2
// meanwhile.  One launch, fp32 multiply-adds: 64 rows at rank 16 beside 3584 x 6144
// in 6.4 us.
//
// More rows: two kernels on tcgen05.  shrink_kernel streams x and the adapter once
// into partial sums of u; expand_kernel joins them and adds u B^T to base.
// Neighbouring rows of one request share an adapter, so a tile has one or a few:
// it goes through its distinct adapters and keeps, of each one's sums, its own
// rows.  A row's result then holds nothing of another adapter's weights, infinities
// and NaN among them, and rows need no order.  Where they have none and the
// adapters are many, they are sorted first and copied row by row.
// (mma.sync gave 266 multiply-adds a clock and SM, a thirtieth of tcgen05's: it held
// a shrink at rank 32 at 28 us where the bytes take 9.)
// Measured (bf16, 16,384 rows, 3584 -> 6144, rank 64, four adapters): 104 us forwards
// for 519 MB (5.0 TB/s), 162 backwards with the gradients for 753 MB.  The shrink's
// CTAs end 29 us after its start (32 where a tile has rows of two adapters) and
// the expand streams 403 MB in 55; the rest is what begins and ends: first loads,
// u's parts and the first sums.
//
// u enters the second product in 16 bits.  For 16-bit results it is rounded
// once (half an ulp of u, as y itself is); for fp32 results it goes as a sum of
// 16-bit terms, three in bf16 and two in f16, which hold 24 and 22 of its bits.
// f16 rows are brought to [2^14, 2^15) by a power of two first, taken out of the
// sums again, so that a u beyond f16 neither overflows nor vanishes.
#include "lora_common.cuh"

#include <cooperative_groups.h>

namespace situ {

using namespace lora;

namespace {

constexpr int kTile = 128;         // rows of a tile
constexpr int kChunk = 64;         // contraction elements of a stage (shrink)
constexpr int kXBytes = kTile * 128;   // a box: 128 bytes of 128 rows
constexpr int kMaxStages = 16;     // of a ring
constexpr int kShrinkSmem = 217 * 1024, kExpandSmem = 220 * 1024;   // 227 KB with the static parts
constexpr int kCluster = 8;        // CTAs of a row
constexpr int kRowThreads = 256;

// f16, backwards (lora_common.cuh): u as the forward pass kept it, and what makes it anew
// where that has lost it.
struct FarParams {
  const uint16_t *u, *x, *a;
  long ldx;
  int K;
  float *u32, *row_most;
  uint32_t* most;                  // null: not this case
};

struct LoraParams {
  const int32_t *ids, *offsets;
  int S, C, r, n;                  // C: the other extent (contraction or columns)
  int r16;                         // r rounded up to 16
  int chunks;                      // of the contraction
  int run;                         // shrink: chunks of a sum in tensor memory
  long shrink_ctas, least;         // CTAs that the shrink's chunks are dealt out over, chunks of each at least
  float* part;                     // [parts of a tile][S][r]
  const float* scale;              // [n] or null
  const float* times;              // [1] or null: what u counts times besides
  const void* base;
  long ld_base;
  void* out;
  long ldo;
  void* u16;                       // [S, 2, r] scaled, in two terms of the operands' type, or null; f16 backwards: fp32 [S, r]
  FarParams far;                   // backwards, f16
  int stages, w_stage;             // shared memory: stages of w, bytes of one
  int x_stages;                    // shrink: of x
  int y_stages, u_stages, u_bytes; // expand: items of base, tiles of u, bytes of one
  // Rows sorted by adapter, where *mixed (null: never): their numbers, how many
  // have an adapter, and of each row its place among them (-1: none).
  const int32_t *mixed, *perm, *kept, *place;
  int* err;
};

// 16-bit terms that u is taken in
__host__ __device__ constexpr int terms_of(int dt, bool f32) { return !f32 ? 1 : dt == SITU_DT_BF16 ? 3 : 2; }

// columns of an item of expand
__host__ __device__ constexpr int cols_of(bool f32) { return f32 ? 64 : 128; }

struct RowParams {
  const void *x, *a, *b, *base;
  void *out, *u16;
  long ldx, ld_base, ldo;
  const int32_t *ids, *offsets;
  const float* scale;
  int S, K, N, r, n;
};

// The same for a whole warp, a row to each lane: up to 31 adapters' offsets in one
// load where a search takes a load after the other.  Rows from S on have none.
__device__ __forceinline__ int adapter_of_lane(const int32_t* ids, const int32_t* offsets, int n, int row, int S) {
  if (ids || n >= 32) return row < S ? adapter_of(ids, offsets, n, row) : -1;
  const int lane = threadIdx.x & 31, o = lane <= n ? __ldcg(offsets + lane) : 0;
  int first = n + 1;               // entry beyond row
  for (int j = n; j >= 0; --j)
    if (__shfl_sync(0xffffffffu, o, j) > row) first = j;
  return row < S && first <= n ? first - 1 : -1;
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
  if (p.u16 && rank == 0 && (int)threadIdx.x < p.r) {
    uint32_t hi = 0, lo = 0;
    if (e >= 0) two_terms<DT>(u_s[threadIdx.x], 0.f, hi, lo);
    uint16_t* o = static_cast<uint16_t*>(p.u16) + (size_t)row * 2 * p.r + threadIdx.x;
    o[0] = (uint16_t)hi;
    o[p.r] = (uint16_t)lo;
  }
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
// tiles
// --------------------------------------------------------------------------

// The adapters of a tile of R rows: each row's (-1: none), and the distinct ones
// in the order of their first rows.
template <int R>
struct Adapters {
  alignas(16) int of[R];   // row -> adapter
  int at[R];               // row -> its place in `list`, or -1
  int list[R];
  int halves[R];           // of each in `list`: whether rows of the first 128 take it (1), and of the others (2)
  uint32_t lead[R / 32], same[R / 32];
  int count;
};
constexpr int kEpi = 256;   // epilogue threads of either kernel
// of T threads at a named barrier; whether all of them came with ok
template <int T>
__device__ __forceinline__ void sync_some() {
  asm volatile("bar.sync 1, %0;" ::"n"(T) : "memory");
}
template <int T>
__device__ __forceinline__ bool all_of(bool ok) {
  uint32_t r;
  asm volatile("{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n barrier.cta.red.and.pred q, 1, %2, p;\n selp.u32 %0, 1, 0, q;\n}"
               : "=r"(r)
               : "r"((uint32_t)ok), "n"(T)
               : "memory");
  return r != 0;
}
// The rows to go through: `count` of them, the i-th is number row(i), S where there
// is none.
struct Rows {
  const int32_t* perm;   // null: as they are
  int S, count;
  __device__ __forceinline__ explicit Rows(const LoraParams& p)
      : perm(p.mixed && __ldcg(p.mixed) ? p.perm : nullptr), S(p.S), count(perm ? __ldcg(p.kept) : p.S) {}
  __device__ __forceinline__ int row(int i) const { return i >= count ? S : perm ? __ldcg(perm + i) : i; }
};
// of row i of a tile, for its thread (whole warps)
__device__ __forceinline__ int tile_adapter(const LoraParams& p, const Rows& rows, int row0, int i) {
  return adapter_of_lane(p.ids, p.offsets, p.n, row0 + i < rows.count ? rows.row(row0 + i) : p.S, p.S);
}
// By R threads, of which this is number i and has e = tile_adapter.  Where one of
// them comes without ok (it gave up waiting for the place) nothing is written.
template <int R>
__device__ __forceinline__ bool find_adapters(Adapters<R>& t, const Rows& rows, int row0, int i, int e, bool ok) {
  if (!all_of<R>(ok)) return false;
  const int lane = i & 31, w = i >> 5;
  t.of[i] = e;
  t.halves[i] = 0;
  sync_some<R>();
  const int e0 = t.of[0];
  const bool same = __all_sync(0xffffffffu, e == e0 || row0 + i >= rows.count);
  if (lane == 0) t.same[w] = same;
  sync_some<R>();
  uint32_t all = 1;
#pragma unroll
  for (int v = 0; v < R / 32; ++v) all &= t.same[v];
  if (all) {
    t.at[i] = e >= 0 ? 0 : -1;
    if (i == 0) {
      t.list[0] = e0;
      t.halves[0] = rows.count - row0 > 128 ? 3 : 1;
      t.count = e0 >= 0 ? 1 : 0;
    }
    sync_some<R>();
    return true;
  }
  // the first row of this one's adapter: in its warp, then in those before it, an
  // adapter at a time
  const int l0 = __ffs(__match_any_sync(0xffffffffu, e)) - 1;
  int first = 32 * w + l0;
  uint32_t lead = __ballot_sync(0xffffffffu, e >= 0 && l0 == lane);
  for (uint32_t rest = lead; rest; rest &= rest - 1) {
    const int l = __ffs(rest) - 1, its = __shfl_sync(0xffffffffu, e, l);
    for (int v = 0; v < w; ++v) {
      const uint32_t found = __ballot_sync(0xffffffffu, t.of[32 * v + lane] == its);
      if (found) {
        if (e == its) first = 32 * v + __ffs(found) - 1;
        lead &= ~(1u << l);
        break;
      }
    }
  }
  if (lane == 0) t.lead[w] = lead;
  sync_some<R>();
  int place = __popc(t.lead[first >> 5] & ((1u << (first & 31)) - 1u));
  for (int v = 0; v < first >> 5; ++v) place += __popc(t.lead[v]);
  t.at[i] = e >= 0 ? place : -1;
  if (e >= 0 && first == i) t.list[place] = e;
  if (e >= 0) atomicOr(&t.halves[place], 1 << (i >> 7));
  if (i == 0) {
    int n = 0;
#pragma unroll
    for (int v = 0; v < R / 32; ++v) n += __popc(t.lead[v]);
    t.count = n;
  }
  sync_some<R>();
  return true;
}

// f16, backwards: a row of u anew from x and a, to fp32, by a warp; its largest finite
// magnitude.
__device__ __noinline__ float u_anew(const uint4* x, const uint4* a, int pieces, int r, float f, float* out) {
  const int lane = threadIdx.x & 31;
  float m = 0.f;
#pragma unroll 1
  for (int c = 0; c < r; c += 8) {
    const uint4* w = a + (size_t)c * pieces;
    float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int d = lane; d < pieces; d += 32) {
      const uint4 v = __ldg(x + d);
#pragma unroll
      for (int t = 0; t < 8; ++t) acc[t] = dot8<SITU_DT_F16>(v, __ldg(w + (size_t)t * pieces + d), acc[t]);
    }
#pragma unroll
    for (int t = 0; t < 8; ++t) {
#pragma unroll
      for (int o = 16; o >= 1; o >>= 1) acc[t] += __shfl_xor_sync(0xffffffffu, acc[t], o);
      acc[t] *= f;
      m = finite_max(m, acc[t]);
    }
    if (lane == 0) put8(out + c, acc);
  }
  return m;
}
__device__ __forceinline__ bool zeros(const uint4* x, int pieces) {
  bool any = false;
  for (int d = threadIdx.x & 31; d < pieces; d += 32) {
    const uint4 v = __ldg(x + d);
    any = any || ((v.x | v.y | v.z | v.w) & 0x7FFF7FFFu) != 0;
  }
  return !__any_sync(0xffffffffu, any);
}
// f16, backwards: each row's largest finite magnitude of u, from the kept terms.  Where
// those have lost it (an infinity, or nothing from kLeast on, beside which f16's steps
// are no longer small) u is made anew, which the sign of the largest says.  By a warp,
// while the first sums are on their way (16,384 rows at rank 64 backwards 152 us, with all
// rows made anew 870).
constexpr float kLeast = 1.f / 256;      // a step's half is 2^-17 of it
__device__ __forceinline__ void look_at_u(const LoraParams& p, long unit) {
  const RowLanes k(p.r, unit);
  uint2 hi[kRowTurns];
#pragma unroll
  for (int i = 0; i < kRowTurns; ++i) {
    const long row = k.row(i, p.S);
    hi[i] = row < p.S ? __ldg(reinterpret_cast<const uint2*>(p.far.u + (size_t)row * 2 * p.r + k.j)) : make_uint2(0, 0);
  }
  uint32_t lost = 0;                                      // bit i: this lane's row of turn i has been lost
#pragma unroll
  for (int i = 0; i < kRowTurns; ++i) {
    constexpr int kF16 = SITU_DT_F16;
    const float v[4] = {lo16<kF16>(hi[i].x), hi16<kF16>(hi[i].x), lo16<kF16>(hi[i].y), hi16<kF16>(hi[i].y)};
    float m = 0.f;
    bool finite = true;
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      m = finite_max(m, v[t]);
      finite = finite && fabsf(v[t]) < INFINITY;
    }
    m = k.largest(m);
    const long row = k.row(i, p.S);
    if (row < p.S && (!finite || m < kLeast)) lost |= 1u << i;
    if (row < p.S && k.j == 0) p.far.row_most[row] = m;
  }
  if (!__any_sync(0xffffffffu, lost != 0)) return;
  for (uint32_t rest = lost; rest; rest &= rest - 1) {    // rows without an adapter are zeros
    const int i = __ffs(rest) - 1;
    if (adapter_of(nullptr, p.offsets, p.n, (int)k.row(i, p.S)) < 0) lost &= ~(1u << i);
  }
  __syncwarp();
#pragma unroll 1
  for (int i = 0; i < kRowTurns; ++i) {
    const uint32_t lanes = __ballot_sync(0xffffffffu, lost >> i & 1);
#pragma unroll 1
    for (int a = 0; a < k.per; ++a) {                     // a row after the other, by all lanes
      const uint32_t of = (k.q == 32 ? 0xffffffffu : (1u << k.q) - 1) << (a * k.q);
      if (!(lanes & of)) continue;
      const long row = k.row0 + (long)i * k.per + a;
      const int e = adapter_of(nullptr, p.offsets, p.n, (int)row), pieces = p.far.K / 8;
      const uint4* x = reinterpret_cast<const uint4*>(p.far.x + (size_t)row * p.far.ldx);
      if (zeros(x, pieces)) continue;                     // kept as they are
      const float m = u_anew(x, reinterpret_cast<const uint4*>(p.far.a) + (size_t)e * p.r * pieces, pieces, p.r,
                             p.scale ? __ldg(p.scale + e) : 1.f, p.far.u32 + (size_t)row * p.r);
      __syncwarp();
      if ((threadIdx.x & 31) == 0) p.far.row_most[row] = -m;
    }
  }
}

constexpr int kTmemCols = 512;                // of an SM
constexpr int kShrinkRows = 256;              // of a tile of the shrink: two MMAs share an adapter's weights
constexpr int kShrinkThreads = 64 + kEpi;     // copies, MMAs; eight epilogue warps
constexpr int kExpandThreads = 128 + kEpi + kTile;   // copies of base and out, MMAs, copies of weights; eight epilogue warps; u

// A CTA's items of one tile, `per` items to a tile, and the next tile's.
struct Segment {
  long i, end;
  int per, tile, from, to;
  __device__ __forceinline__ Segment(long i0, long i1, int per_tile) : i(i0), end(i1), per(per_tile) { set(); }
  __device__ __forceinline__ bool more() const { return i < end; }
  __device__ __forceinline__ void next() {
    i += to - from;
    set();
  }
  __device__ __forceinline__ void set() {
    tile = (int)(i / per);
    from = (int)(i - (long)tile * per);
    to = (int)min((long)per, from + (end - i));
  }
};

__device__ __forceinline__ void store_2d(const CUtensorMap* map, uint32_t src, int x, int y) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(x), "r"(y), "r"(src)
               : "memory");
}
__device__ __forceinline__ void store_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void store_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}

// part[.][i][j] = sum over a range of k of x[i, k] W[e(i)][j][k] (TRANS:
// W[e][k][j]): the tile's rows on the MMA's M side (two MMAs of 128: with one the
// weights were a third of what the SMs take in), an adapter's r on its N side, in TMEM columns of its own.  As many
// adapters as half of the columns hold share a pass over x; the other half takes
// the next sums meanwhile.  The chunks of all tiles are dealt out evenly over the
// CTAs, one per SM; what a CTA has of a tile is that tile's next part.  For fp32
// results p.run chunks (1,024 elements) make a sum: the tensor cores truncate when
// they add, 6e-9 of a sum of one sign per element; the sums meet in fp32.
template <int DT, bool TRANS>
__global__ void __launch_bounds__(kShrinkThreads, 1)
shrink_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_x1,
              const __grid_constant__ CUtensorMap map_w, const LoraParams p) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ Adapters<kShrinkRows> lists[2];
  __shared__ uint64_t bars[4 * kMaxStages + 9];
  __shared__ uint32_t holder[2];
  const uint32_t sbase = (saddr(smem_raw) + 1023) & ~1023u;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t bar0 = saddr(bars);
  auto xfull = [&](int s) { return bar0 + 8 * s; };
  auto xempty = [&](int s) { return bar0 + 8 * (kMaxStages + s); };
  auto wfull = [&](int s) { return bar0 + 8 * (2 * kMaxStages + s); };
  auto wempty = [&](int s) { return bar0 + 8 * (3 * kMaxStages + s); };
  const uint32_t tail = bar0 + 8 * 4 * kMaxStages;
  auto acc_full = [&](int b) { return tail + 8 * b; };
  auto acc_empty = [&](int b) { return tail + 16 + 8 * b; };
  auto list_full = [&](int b) { return tail + 32 + 8 * b; };
  auto list_empty = [&](int b) { return tail + 48 + 8 * b; };
  const uint32_t drain = tail + 64;
  if (tid == 0) {
    holder[1] = (uint32_t)*reinterpret_cast<volatile int*>(p.err);   // an earlier launch gave up a wait: no work then
    prefetch_map(&map_w);
    for (int s = 0; s < 4 * kMaxStages; ++s) mbar_init(bar0 + 8 * s, 1);
    for (int b = 0; b < 2; ++b) {
      mbar_init(acc_full(b), 1);
      mbar_init(acc_empty(b), kEpi / 32);
      mbar_init(list_full(b), 1);
      mbar_init(list_empty(b), 2);
    }
    mbar_init(drain, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) tmem_alloc<1>(saddr(holder), kTmemCols);
  if (DT == SITU_DT_F16 && TRANS && blockIdx.x == 0)
    for (int i = tid; i < 2 * p.n; i += kShrinkThreads) p.far.most[i] = 0;
  if (p.mixed) griddep_wait();       // the rows' order is the predecessor's
  const Rows rows(p);
  const long total = (long)((rows.count + kShrinkRows - 1) / kShrinkRows) * p.chunks, G = sharers(total, p.shrink_ctas, p.least);
  const bool shares = blockIdx.x < G;
  const long i0 = shares ? first_item(blockIdx.x, total, G) : 0, i1 = shares ? first_item(blockIdx.x + 1, total, G) : 0;
  int e_first = -1;                  // of the first tile: on its way while the barriers are set up
  if (warp >= 2 && i0 < i1) e_first = tile_adapter(p, rows, (int)(i0 / p.chunks) * kShrinkRows, tid - 64);
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = holder[0];
  const bool dead = holder[1] != 0;
  griddep_launch_dependents();       // its CTAs start where these have left, and fetch base
  constexpr int kSumCols = kTmemCols / 2, kHalfCols = kSumCols / 2;   // of a sum's columns, those of 128 rows
  const int per = kHalfCols / p.r16;                    // adapters of a pass
  const uint32_t wbase = sbase + p.x_stages * 2 * kXBytes;

  if (warp == 0 && !dead) {
    // ---------------- copies ----------------
    const bool leader = elect_one();
    const int wboxes = (p.r + 63) / 64;
    Turns x(p.x_stages), w(p.stages), l(2);
    bool ok = true;
    for (Segment g(i0, i1, p.chunks); g.more() && ok; g.next()) {
      if (!warp_wait(list_full(l.s), l.ph, p.err, 81)) {
        ok = false;
        break;
      }
      const Adapters<kShrinkRows>& ad = lists[l.s];
      const int nd = ad.count, row0 = g.tile * kShrinkRows, halves = rows.count - row0 > kTile ? 2 : 1;
      int at[2][4];                                     // sorted rows: this lane's four of each 128
      if (rows.perm)
        for (int h = 0; h < 2; ++h)
          for (int j = 0; j < 4; ++j) at[h][j] = rows.row(row0 + h * kTile + 4 * lane + j);
      for (int d0 = 0; d0 < nd && ok; d0 += per) {
        const int d1 = min(nd, d0 + per);
        for (int k = g.from; k < g.to && ok; ++k) {
          if (x.again() && !warp_wait(xempty(x.s), x.ph ^ 1, p.err, 82)) {
            ok = false;
            break;
          }
          if (leader) {
            mbar_expect_tx(xfull(x.s), halves * kXBytes);
            for (int h = 0; h < halves && !rows.perm; ++h)
              copy_2d<1>(sbase + (2 * x.s + h) * kXBytes, &map_x, k * kChunk, row0 + h * kTile, xfull(x.s));
          }
          __syncwarp();
          if (rows.perm)
            for (int h = 0; h < halves; ++h)
              copy_rows4<1>(sbase + (2 * x.s + h) * kXBytes + lane * 512, &map_x1, k * kChunk, at[h][0], at[h][1], at[h][2],
                            at[h][3], xfull(x.s));
          __syncwarp();
          x.next();
          for (int d = d0; d < d1; ++d, w.next()) {
            if (w.again() && !warp_wait(wempty(w.s), w.ph ^ 1, p.err, 83)) {
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
      __syncwarp();
      mbar_arrive_if(list_empty(l.s), lane == 0);
      l.next();
    }
    leave(
        ok,
        [&] {
          const bool a = x.last([&](int j, uint32_t ph) { return warp_wait(xempty(j), ph, p.err, 84); });
          return w.last([&](int j, uint32_t ph) { return warp_wait(wempty(j), ph, p.err, 85); }) && a;
        },
        [&] {
          x.last([&](int j, uint32_t ph) { return drain_wait(xfull(j), ph); });
          w.last([&](int j, uint32_t ph) { return drain_wait(wfull(j), ph); });
        });
  } else if (warp == 1 && !dead) {
    // ---------------- MMAs ----------------
    const bool leader = elect_one();
    const uint32_t idesc = idesc_of(DT == SITU_DT_BF16, false, TRANS, p.r16);
    Turns x(p.x_stages), w(p.stages), l(2), acc(2);
    bool ok = true;
    for (Segment g(i0, i1, p.chunks); g.more() && ok; g.next()) {
      if (!warp_wait(list_full(l.s), l.ph, p.err, 86)) {
        ok = false;
        break;
      }
      const Adapters<kShrinkRows>& ad = lists[l.s];
      const int nd = ad.count;
      for (int d0 = 0; d0 < nd && ok; d0 += per) {
        const int d1 = min(nd, d0 + per);
        for (int from = g.from; from < g.to && ok; from += p.run) {
          const int to = min(g.to, from + p.run);
          if (acc.again() && !warp_wait(acc_empty(acc.s), acc.ph ^ 1, p.err, 87)) {
            ok = false;
            break;
          }
          asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
          for (int k = from; k < to && ok; ++k, x.next()) {
            if (!warp_wait(xfull(x.s), x.ph, p.err, 88)) {
              ok = false;
              break;
            }
            const int steps = min(kChunk / 16, (p.C - k * kChunk + 15) >> 4);
            for (int d = d0; d < d1; ++d, w.next()) {
              if (!warp_wait(wfull(w.s), w.ph, p.err, 89)) {
                ok = false;
                break;
              }
              asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
              if (leader) {
                const uint32_t wa = wbase + w.s * p.w_stage;
                const uint64_t wd = TRANS ? sdesc_mn(wa, 8192) : sdesc(wa);
                const int halves = ad.halves[d];       // the other rows' sums are not read
                for (int h = 0; h < 2; ++h) {
                  if (!(halves >> h & 1)) continue;
                  const uint64_t xd = sdesc(sbase + (2 * x.s + h) * kXBytes);
                  for (int j = 0; j < steps; ++j)
                    mma_f16<1>(tmem + acc.s * kSumCols + h * kHalfCols + (d - d0) * p.r16, xd + 2 * j, wd + (TRANS ? 128 : 2) * j,
                               idesc, ((k - from) | j) != 0);
                }
                mma_commit(wempty(w.s));
                if (d + 1 == d1) mma_commit(xempty(x.s));
              }
              __syncwarp();
            }
          }
          if (ok) {
            if (leader) mma_commit(acc_full(acc.s));
            __syncwarp();
            acc.next();
          }
        }
      }
      __syncwarp();
      mbar_arrive_if(list_empty(l.s), lane == 0);
      l.next();
    }
    leave(
        ok, [&] { return w.last([&](int j, uint32_t ph) { return warp_wait(wempty(j), ph, p.err, 90); }); },
        [&] {
          if (leader) mma_commit(drain);
          __syncwarp();
          drain_wait(drain, 0);
        });
  } else if (warp >= 2 && !dead) {
    // ---------------- lists, and sums to memory, a row per lane ----------------
    const int et = tid - 64, q = warp & 3, h = (warp - 2) >> 2, mine = h * kTile + 32 * q + lane;
    Turns l(2), acc(2);
    bool ok = true;
    auto list = [&](const Segment& g, int e) {          // of a tile, while the one before is worked on
      if (l.again() && !warp_wait(list_empty(l.s), l.ph ^ 1, p.err, 91)) ok = false;
      ok = find_adapters(lists[l.s], rows, g.tile * kShrinkRows, et, e, ok);
      mbar_arrive_if(list_full(l.s), et == 0);
      l.next();
    };
    Segment g(i0, i1, p.chunks);
    if (g.more()) list(g, e_first);
    if (DT == SITU_DT_F16 && TRANS) {                     // before the first sums are there
      constexpr int kWarps = kEpi / 32;
      for (long unit = (long)blockIdx.x * kWarps + warp - 2; unit * RowLanes::rows(p.r) < p.S; unit += (long)gridDim.x * kWarps)
        look_at_u(p, unit);
    }
    for (int b = 0; g.more(); b ^= 1) {
      Segment n = g;
      n.next();
      if (n.more()) list(n, tile_adapter(p, rows, n.tile * kShrinkRows, et));
      const Adapters<kShrinkRows>& ad = lists[b];
      const int nd = ad.count, at = ad.at[mine], row = g.tile * kShrinkRows + mine;
      const int part = (int)((long)blockIdx.x - cta_of((long)g.tile * p.chunks, total, G));
      float* out = p.part + ((size_t)part * p.S + row) * p.r;
      for (int d0 = 0; d0 < nd && ok; d0 += per) {
        const int d1 = min(nd, d0 + per);
        for (int from = g.from; from < g.to && ok; from += p.run, acc.next()) {
          if (!warp_wait(acc_full(acc.s), acc.ph, p.err, 92)) {
            ok = false;
            break;
          }
          asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
          for (int d = d0; d < d1; ++d) {
            if (!__any_sync(0xffffffffu, at == d)) continue;
            for (int j = 0; j < p.r16; j += 16) {
              uint32_t v[16];
              __syncwarp();
              tmem_ld16_nowait(tmem + ((uint32_t)(32 * q) << 16) + acc.s * kSumCols + h * kHalfCols + (d - d0) * p.r16 + j, v);
              tmem_ld_wait<16>(v);
              if (at == d) {
#pragma unroll
                for (int t = 0; t < 16; t += 8) {
                  if (j + t >= p.r) break;
                  float f[8];
#pragma unroll
                  for (int i = 0; i < 8; ++i)
                    f[i] = __uint_as_float(v[t + i]) + (from > g.from ? out[j + t + i] : 0.f);   // onto the run before
                  put8(out + j + t, f);
                }
              }
              __syncwarp();
            }
          }
          asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
          mbar_arrive_if(acc_empty(acc.s), lane == 0);
        }
      }
      g = n;
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

// out[i][c] = base[i][c] + s[e] sum_j u[i][j] W[e][c][j] (TRANS: W[e][j][c]),
// u the sum of its parts: the tile's rows on the MMA's M side, 128 columns
// (fp32: 64) on its N side.  Base comes into shared memory by TMA, two boxes of
// 128 rows by 128 bytes an item, several items ahead; the epilogue adds each
// adapter's sums to its rows there, and TMA takes the boxes to out.  So
// rows without an adapter pass through, and no thread waits for memory: with
// base loaded and out stored by the epilogue's own instructions, the loads', the
// sums' and the stores' times added up (403 MB in 116 us).  u stays in shared
// memory for all the CTA's items of a tile, its 16-bit terms one after the
// other along the contraction; warps of their own bring the next tile's meanwhile
// (between two tiles it cost each CTA that has two 13 us of 70).  The items are
// dealt out evenly over the CTAs, one per SM.  Waits are bounded from where they begin,
// so those for what comes of u begin when the shrink, however long, has ended.
template <int DT, bool TRANS, bool F32>
__global__ void __launch_bounds__(kExpandThreads, 1)
expand_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_base,
              const __grid_constant__ CUtensorMap map_base1, const __grid_constant__ CUtensorMap map_out, const LoraParams p) {
  constexpr int kTerms = terms_of(DT, F32), kCols = cols_of(F32), kBoxCols = kCols / 2;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Adapters<kTile> lists[2];
  __shared__ float back[2][kTile];   // f16: the power of two that a row's u was divided by
  __shared__ uint64_t bars[4 * kMaxStages + 11];
  __shared__ uint32_t holder[2];
  uint8_t* smem = smem_raw + (((saddr(smem_raw) + 1023) & ~1023u) - saddr(smem_raw));
  const uint32_t sbase = saddr(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t bar0 = saddr(bars);
  auto wfull = [&](int s) { return bar0 + 8 * s; };
  auto wempty = [&](int s) { return bar0 + 8 * (kMaxStages + s); };
  auto yfull = [&](int s) { return bar0 + 8 * (2 * kMaxStages + s); };
  auto ydone = [&](int s) { return bar0 + 8 * (3 * kMaxStages + s); };
  const uint32_t tail = bar0 + 8 * 4 * kMaxStages;
  auto acc_full = [&](int b) { return tail + 8 * b; };
  auto acc_empty = [&](int b) { return tail + 16 + 8 * b; };
  auto list_full = [&](int b) { return tail + 32 + 8 * b; };
  auto u_full = [&](int b) { return tail + 48 + 8 * b; };
  auto tile_empty = [&](int b) { return tail + 64 + 8 * b; };
  const uint32_t drain = tail + 80;
  const int blocks = (p.C + kCols - 1) / kCols;
  const Rows rows(p);
  const long total = (long)((rows.count + kTile - 1) / kTile) * blocks, G = gridDim.x;
  const long i0 = first_item(blockIdx.x, total, G), i1 = first_item(blockIdx.x + 1, total, G);
  int e_first = -1;                  // of the first tile, ahead of the copies of base
  if (warp >= 12 && i0 < i1) e_first = tile_adapter(p, rows, (int)(i0 / blocks) * kTile, tid - 384);
  if (tid == 0) {
    prefetch_map(&map_w);
    if (p.base) prefetch_map(&map_base);
    prefetch_map(&map_out);
    for (int s = 0; s < kMaxStages; ++s) {
      mbar_init(wfull(s), 1);
      mbar_init(wempty(s), 1);
      mbar_init(yfull(s), 1);
      mbar_init(ydone(s), kEpi / 32);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(acc_full(b), 1);
      mbar_init(acc_empty(b), kEpi / 32);
      mbar_init(list_full(b), 1);
      mbar_init(u_full(b), 12);                           // warps of the first tile's; of four, three each
      mbar_init(tile_empty(b), kEpi / 32 + 2);          // the epilogue, the copies of weights, the MMAs
    }
    mbar_init(drain, 1);
    holder[1] = (uint32_t)*reinterpret_cast<volatile int*>(p.err);   // an earlier call gave up a wait: no work then
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) tmem_alloc<1>(saddr(holder), 256);
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = holder[0];
  const bool dead = holder[1] != 0;
  griddep_launch_dependents();       // of the backward pass: the gradients' CTAs fetch x and dy where these have left
  const uint32_t wbase = sbase + p.u_stages * p.u_bytes, ybase = wbase + p.stages * p.w_stage;
  const int rboxes = (p.r + 63) / 64, steps = p.r16 / 16;
  const int rrows = min(64, p.r16);                     // TRANS: contraction rows of a box

  auto parts_of = [&](const Segment& g) {
    const long t0 = (long)(g.tile / (kShrinkRows / kTile)) * p.chunks;
    const long all = (long)((rows.count + kShrinkRows - 1) / kShrinkRows) * p.chunks;
    const long sharing = sharers(all, p.shrink_ctas, p.least);
    return (int)(cta_of(t0 + p.chunks - 1, all, sharing) - cta_of(t0, all, sharing)) + 1;
  };
  // u of a tile in its place ts: what warp `part` of `among` has of it
  auto stage_u = [&](const Segment& g, int ts, int part, int among, int parts) {
    const bool write = p.u16 && g.from == 0 && parts > 0;
    const float times = TRANS && p.times ? __ldg(p.times) : 1.f;
    const Adapters<kTile>& ad = lists[ts];
    uint8_t* us = smem + ts * p.u_bytes;
    const size_t stride = (size_t)p.S * p.r;
    // Eight lanes to a row, four columns each of every 32; four rows at a time
    // and kRows of those together, four parts in flight.
    auto stage = [&](auto cs) {
      constexpr int kC = decltype(cs)::value, kRows = 4 / kC;
      const int c0 = 4 * (lane & 7);
#pragma unroll 1
      for (int r0 = 4 * kRows * part; r0 < kTile; r0 += 4 * kRows * among) {
        float u[kRows][kC][4];
        const float* src[kRows];
        int of[kRows];
        float f[kRows];
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
          const int r = r0 + 4 * i + (lane >> 3);
          of[i] = ad.of[r];
          f[i] = times * (of[i] >= 0 && p.scale ? __ldg(p.scale + of[i]) : 1.f);
          src[i] = p.part + (size_t)(g.tile * kTile + r) * p.r + c0;
#pragma unroll
          for (int c = 0; c < kC; ++c) u[i][c][0] = u[i][c][1] = u[i][c][2] = u[i][c][3] = 0.f;
        }
        for (int s0 = 0; s0 == 0 || s0 < parts; s0 += 4) {
          float4 v[4][kRows][kC];
#pragma unroll
          for (int s = 0; s < 4; ++s)
#pragma unroll
            for (int i = 0; i < kRows; ++i)
#pragma unroll
              for (int c = 0; c < kC; ++c)
                v[s][i][c] = s0 + s < parts && of[i] >= 0 && c0 + 32 * c < p.r
                                 ? __ldcg(reinterpret_cast<const float4*>(src[i] + (s0 + s) * stride + 32 * c))
                                 : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int s = 0; s < 4; ++s)
#pragma unroll
            for (int i = 0; i < kRows; ++i)
#pragma unroll
              for (int c = 0; c < kC; ++c) {
                u[i][c][0] += v[s][i][c].x;
                u[i][c][1] += v[s][i][c].y;
                u[i][c][2] += v[s][i][c].z;
                u[i][c][3] += v[s][i][c].w;
              }
        }
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
          const int r = r0 + 4 * i + (lane >> 3);
#pragma unroll
          for (int c = 0; c < kC; ++c)
#pragma unroll
            for (int k = 0; k < 4; ++k) u[i][c][k] = of[i] >= 0 ? u[i][c][k] * f[i] : 0.f;
          const int row = write ? rows.row(g.tile * kTile + r) : p.S;
          float to = 1.f;
          if (DT == SITU_DT_F16) {
            float m = 0.f;
#pragma unroll
            for (int c = 0; c < kC; ++c)
#pragma unroll
              for (int k = 0; k < 4; ++k) m = finite_max(m, u[i][c][k]);
#pragma unroll
            for (int o = 1; o < 8; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            const int ex = power_of(m);
            to = exp2i(-ex);
            if ((lane & 7) == 0) {
              back[ts][r] = exp2i(ex);
              if (TRANS && row < p.S && of[i] >= 0) raise_most(p.far.most + of[i], m);
            }
          }
#pragma unroll
          for (int c = 0; c < kC; ++c) {
            const int j = c0 + 32 * c;
            if (DT == SITU_DT_F16 && TRANS) {               // v as it is: its terms wait for the largest
              if (row < p.S && j < p.r)
                *reinterpret_cast<float4*>(static_cast<float*>(p.u16) + (size_t)row * p.r + j) =
                    make_float4(u[i][c][0], u[i][c][1], u[i][c][2], u[i][c][3]);
            } else if (row < p.S && j < p.r) {
              uint2 *o = reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.u16) + (size_t)row * 2 * p.r + j), hi, lo;
              two_terms<DT>(u[i][c][0], u[i][c][1], hi.x, lo.x);
              two_terms<DT>(u[i][c][2], u[i][c][3], hi.y, lo.y);
              o[0] = hi;
              o[p.r / 4] = lo;
            }
#pragma unroll
            for (int t = 0; t < kTerms; ++t) {
              uint32_t v[2];
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                const float a = u[i][c][2 * k] * (t == 0 ? to : 1.f), b = u[i][c][2 * k + 1] * (t == 0 ? to : 1.f);
                v[k] = pack16<DT>(a, b);
                // what the term leaves; an infinity leaves nothing
                u[i][c][2 * k] = fabsf(a) < INFINITY ? a - lo16<DT>(v[k]) : 0.f;
                u[i][c][2 * k + 1] = fabsf(b) < INFINITY ? b - hi16<DT>(v[k]) : 0.f;
              }
              const int k = t * p.r16 + j;              // along u's terms: 128-byte swizzled rows of 64
              if (j < p.r16)
                *reinterpret_cast<uint2*>(us + (k >> 6) * kXBytes + r * 128 + ((((k & 63) >> 3) ^ (r & 7)) << 4) +
                                          2 * (k & 4)) = make_uint2(v[0], v[1]);
            }
          }
        }
      }
    };
    using std::integral_constant;
    if (p.r <= 32) stage(integral_constant<int, 1>{});
    else if (p.r <= 64) stage(integral_constant<int, 2>{});
    else stage(integral_constant<int, 4>{});
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
  };

  // Lists and u from its parts, by four warps, for the first tile by those of the
  // epilogue too.  There a round without parts comes first, while the predecessor
  // ends: it brings the instructions in, which took 3.6 us of the 7 between that
  // end and the first MMA.
  bool first_ok = true;
  if (warp >= 4 && !dead) {
    const bool all = warp >= 12;
    const int st = tid - 384;
    Turns tile(p.u_stages);
    bool first = true;
    for (Segment g(i0, i1, blocks); g.more(); g.next(), tile.next(), first = false) {
      if (all) {
        const int e = first ? e_first : tile_adapter(p, rows, g.tile * kTile, st);
        if (tile.again() && !warp_wait(tile_empty(tile.s), tile.ph ^ 1, p.err, 110)) first_ok = false;
        first_ok = find_adapters(lists[tile.s], rows, g.tile * kTile, st, e, first_ok);
        if (!first_ok) break;
        mbar_arrive_if(list_full(tile.s), st == 0);
      } else {
        first_ok = warp_wait(list_full(0), 0, p.err, 104);
      }
      const int parts = parts_of(g);
#pragma unroll 1
      for (int round = first ? 0 : 1; round < 2; ++round) {
        if (first && round == 1) griddep_wait();          // the parts are the predecessor's: base and weights come meanwhile
        if (first_ok) stage_u(g, tile.s, first ? warp - 4 : warp - 12, first ? 12 : 4, round == 0 ? 0 : parts);
      }
      if (lane == 0) mbar_arrive_n(u_full(tile.s), first ? 1 : 3);
      if (!all) break;
    }
  }

  if (warp == 0 && !dead) {
    // ---------------- base in, out ----------------
    const bool leader = elect_one();
    Turns in(p.y_stages), out(p.y_stages);
    bool ok = true;
    long next = i0;
    int of_tile = -1, at[4];                            // sorted rows: this lane's four of a tile
    auto load = [&] {
      const int tile = (int)(next / blocks), c0 = (int)(next - (long)tile * blocks) * kCols;
      const int boxes = c0 + kBoxCols < p.C ? 2 : 1;
      const uint32_t to = ybase + in.s * 2 * kXBytes;
      if (leader) {
        mbar_expect_tx(yfull(in.s), p.base ? boxes * kXBytes : 0);
        if (p.base && !rows.perm)
          for (int h = 0; h < boxes; ++h) copy_2d<1>(to + h * kXBytes, &map_base, c0 + h * kBoxCols, tile * kTile, yfull(in.s));
      }
      __syncwarp();
      if (p.base && rows.perm) {
        if (tile != of_tile)
          for (int j = 0; j < 4; ++j) at[j] = rows.row(tile * kTile + 4 * lane + j);
        of_tile = tile;
        for (int h = 0; h < boxes; ++h)
          copy_rows4<1>(to + h * kXBytes + lane * 512, &map_base1, c0 + h * kBoxCols, at[0], at[1], at[2], at[3], yfull(in.s));
      }
      __syncwarp();
      in.next();
      ++next;
    };
    for (int j = 0; j < p.y_stages - 1 && next < i1; ++j) load();
    griddep_wait();
    for (long i = i0; i < i1; ++i, out.next()) {
      if (!warp_wait(ydone(out.s), out.ph, p.err, 101)) {
        ok = false;
        break;
      }
      if (leader && !rows.perm) {                          // sorted rows: the epilogue has stored them
        const int tile = (int)(i / blocks), c0 = (int)(i - (long)tile * blocks) * kCols;
        for (int h = 0; h < 2 && c0 + h * kBoxCols < p.C; ++h)
          store_2d(&map_out, ybase + out.s * 2 * kXBytes + h * kXBytes, c0 + h * kBoxCols, tile * kTile);
        store_commit();
        store_wait_read<1>();                           // the item before: its place takes the next load
      }
      __syncwarp();
      if (next < i1) load();
    }
    if (leader) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    __syncwarp();
    if (!ok) in.last([&](int j, uint32_t ph) { return drain_wait(yfull(j), ph); });
  } else if (warp == 1 && !dead) {
    // ---------------- MMAs ----------------
    const bool leader = elect_one();
    const uint32_t idesc = idesc_of(DT == SITU_DT_BF16, false, TRANS, kCols);
    Turns w(p.stages), acc(2), tile(p.u_stages);
    bool ok = true;
    griddep_wait();
    for (Segment g(i0, i1, blocks); g.more() && ok; g.next(), tile.next()) {
      if (!warp_wait(u_full(tile.s), tile.ph, p.err, 102)) {
        ok = false;
        break;
      }
      const int nd = lists[tile.s].count;
      const uint32_t ubase = sbase + tile.s * p.u_bytes;
      for (int b = g.from; b < g.to && ok; ++b)
        for (int d = 0; d < nd; ++d, w.next(), acc.next()) {
          if ((acc.again() && !warp_wait(acc_empty(acc.s), acc.ph ^ 1, p.err, 113)) || !warp_wait(wfull(w.s), w.ph, p.err, 105)) {
            ok = false;
            break;
          }
          asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
          if (leader) {
            const uint32_t wa = wbase + w.s * p.w_stage;
            for (int t = kTerms - 1; t >= 0; --t)         // the smallest term first
              for (int j = 0; j < steps; ++j) {
                const int k = t * steps + j;              // sixteens along u's terms
                const uint64_t ud = sdesc(ubase + (k >> 2) * kXBytes) + 2 * (k & 3);
                const uint64_t wd = TRANS ? sdesc_mn(wa + (j >> 2) * (kCols / 64) * rrows * 128, rrows * 128) + 128 * (j & 3)
                                          : sdesc(wa + (j >> 2) * kCols * 128) + 2 * (j & 3);
                mma_f16<1>(tmem + acc.s * kCols, ud, wd, idesc, t != kTerms - 1 || j != 0);
              }
            mma_commit(wempty(w.s));
            mma_commit(acc_full(acc.s));
          }
          __syncwarp();
        }
      if (leader) mma_commit(tile_empty(tile.s));
      __syncwarp();
    }
    leave(
        ok, [&] { return w.last([&](int j, uint32_t ph) { return warp_wait(wempty(j), ph, p.err, 106); }); },
        [&] {
          if (leader) mma_commit(drain);
          __syncwarp();
          drain_wait(drain, 0);
        });
  } else if (warp == 2 && !dead) {
    // ---------------- weights ----------------
    const bool leader = elect_one();
    Turns w(p.stages), tile(p.u_stages);
    bool ok = true;
    for (Segment g(i0, i1, blocks); g.more() && ok; g.next(), tile.next()) {
      if (!warp_wait(list_full(tile.s), tile.ph, p.err, 107)) {
        ok = false;
        break;
      }
      const Adapters<kTile>& ad = lists[tile.s];
      const int nd = ad.count;
      for (int b = g.from; b < g.to && ok; ++b)
        for (int d = 0; d < nd; ++d, w.next()) {
          if (w.again()) {
            griddep_wait();
            ok = warp_wait(wempty(w.s), w.ph ^ 1, p.err, 108);
            if (!ok) break;
          }
          if (leader) {
            const uint32_t to = wbase + w.s * p.w_stage;
            const int c0 = b * kCols, e = ad.list[d];
            if (!TRANS) {
              mbar_expect_tx(wfull(w.s), rboxes * kCols * 128);
              for (int j = 0; j < rboxes; ++j) copy_3d<1>(to + j * kCols * 128, &map_w, 64 * j, c0, e, wfull(w.s));
            } else {
              constexpr int kHalves = kCols / 64;
              mbar_expect_tx(wfull(w.s), rboxes * kHalves * rrows * 128);
              for (int j = 0; j < rboxes; ++j)
                for (int h = 0; h < kHalves; ++h)
                  copy_3d<1>(to + (kHalves * j + h) * rrows * 128, &map_w, c0 + 64 * h, 64 * j, e, wfull(w.s));
            }
          }
          __syncwarp();
        }
      __syncwarp();
      mbar_arrive_if(tile_empty(tile.s), lane == 0);
    }
    griddep_wait();
    leave(
        ok, [&] { return w.last([&](int j, uint32_t ph) { return warp_wait(wempty(j), ph, p.err, 109); }); },
        [&] { w.last([&](int j, uint32_t ph) { return drain_wait(wfull(j), ph); }); });
  } else if (warp == 3 && !dead && rows.perm) {
    // ---------------- rows without an adapter, where they are not in a tile ----------------
    constexpr int kEl = F32 ? 4 : 2;
    for (long r0 = (long)blockIdx.x * 32; r0 < p.S; r0 += G * 32) {
      uint32_t none = __ballot_sync(0xffffffffu, r0 + lane < p.S && __ldcg(p.place + r0 + lane) < 0);
      for (; none; none &= none - 1) {
        const long row = r0 + __ffs(none) - 1;
        uint4* out = reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.out) + (size_t)row * p.ldo * kEl);
        const uint4* base = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p.base) + (size_t)row * p.ld_base * kEl);
        if (p.out != p.base)
          for (int i = lane; i < p.C / (16 / kEl); i += 32) out[i] = p.base ? base[i] : make_uint4(0, 0, 0, 0);
        if (p.u16)
          for (int i = lane; i < p.r / 4; i += 32)
            reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.u16) + (size_t)row * 2 * p.r)[i] = make_uint4(0, 0, 0, 0);
      }
    }
  } else if (DT == SITU_DT_F16 && TRANS && warp == 3 && !dead) {
    // ---------------- the adapters' largest u ----------------
    griddep_wait();
    for (long r0 = (long)blockIdx.x * 32; r0 < p.S; r0 += G * 32) {
      const int e = adapter_of_lane(nullptr, p.offsets, p.n, (int)min(r0 + lane, (long)p.S), p.S);
      const float m = e >= 0 ? fabsf(__ldcg(p.far.row_most + r0 + lane)) : 0.f;
      if (__all_sync(0xffffffffu, e == __shfl_sync(0xffffffffu, e, 0))) {
        const uint32_t all = __reduce_max_sync(0xffffffffu, __float_as_uint(m));
        if (lane == 0 && e >= 0) raise_most(p.far.most + p.n + e, __uint_as_float(all));
      } else if (e >= 0) {
        raise_most(p.far.most + p.n + e, m);
      }
    }
  } else if (warp >= 4 && warp < 12 && !dead) {
    // ---------------- sums onto base ----------------
    const int q = warp & 3, h = (warp - 4) >> 2;        // this warp's 32 rows, and box of an item
    Turns acc(2), y(p.y_stages), tile(p.u_stages);
    bool ok = first_ok;
    for (Segment g(i0, i1, blocks); g.more() && ok; g.next(), tile.next()) {
      if (!warp_wait(u_full(tile.s), tile.ph, p.err, 103)) {
        ok = false;
        break;
      }
      const Adapters<kTile>& ad = lists[tile.s];
      const int nd = ad.count, at = ad.at[32 * q + lane];
      const float my_back = DT == SITU_DT_F16 ? back[tile.s][32 * q + lane] : 1.f;
      const int my_row = rows.perm ? rows.row(g.tile * kTile + 32 * q + lane) : 0;
      for (int b = g.from; b < g.to && ok; ++b, y.next()) {
        uint8_t* mine = smem + (ybase - sbase) + y.s * 2 * kXBytes + h * kXBytes + (32 * q + lane) * 128;
        auto piece = [&](int j) { return reinterpret_cast<uint4*>(mine + ((j ^ (lane & 7)) << 4)); };
        if (!warp_wait(yfull(y.s), y.ph, p.err, 111)) {
          ok = false;
          break;
        }
        if (!p.base) {
#pragma unroll
          for (int j = 0; j < 8; ++j) *piece(j) = make_uint4(0, 0, 0, 0);
        }
        for (int d = 0; d < nd; ++d, acc.next()) {
          if (!warp_wait(acc_full(acc.s), acc.ph, p.err, 112)) {
            ok = false;
            break;
          }
          asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
          if (__any_sync(0xffffffffu, at == d)) {
            const uint32_t from = tmem + ((uint32_t)(32 * q) << 16) + acc.s * kCols + kBoxCols * h;
#pragma unroll
            for (int c = 0; c < kBoxCols / 32; ++c) {
              uint32_t v[32];
              __syncwarp();
              tmem_ld32_nowait(from + 32 * c, v);
              tmem_ld_wait<32>(v);
              if (DT == SITU_DT_F16) {
#pragma unroll
                for (int t = 0; t < 32; ++t) v[t] = __float_as_uint(__uint_as_float(v[t]) * my_back);
              }
              if (at == d && F32) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                  uint4 o = *piece(j);
                  o.x = __float_as_uint(__uint_as_float(o.x) + __uint_as_float(v[4 * j]));
                  o.y = __float_as_uint(__uint_as_float(o.y) + __uint_as_float(v[4 * j + 1]));
                  o.z = __float_as_uint(__uint_as_float(o.z) + __uint_as_float(v[4 * j + 2]));
                  o.w = __float_as_uint(__uint_as_float(o.w) + __uint_as_float(v[4 * j + 3]));
                  *piece(j) = o;
                }
              } else if (at == d) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                  uint4 o = *piece(4 * c + j);
                  uint32_t* ow = reinterpret_cast<uint32_t*>(&o);
#pragma unroll
                  for (int t = 0; t < 4; ++t)
                    ow[t] = pack16<DT>(lo16<DT>(ow[t]) + __uint_as_float(v[8 * j + 2 * t]),
                                       hi16<DT>(ow[t]) + __uint_as_float(v[8 * j + 2 * t + 1]));
                  *piece(4 * c + j) = o;
                }
              }
            }
            __syncwarp();
          }
          asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
          mbar_arrive_if(acc_empty(acc.s), lane == 0);
        }
        if (!ok) break;
        if (rows.perm) {                                   // 32 rows of 128 bytes, four a time
          __syncwarp();
          const uint8_t* box = smem + (ybase - sbase) + y.s * 2 * kXBytes + h * kXBytes + 32 * q * 128;
          const int col = b * kCols + kBoxCols * h + (lane & 7) * (kBoxCols / 8);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int r = 4 * j + (lane >> 3), row = __shfl_sync(0xffffffffu, my_row, r);
            const uint4 o = *reinterpret_cast<const uint4*>(box + r * 128 + (((lane & 7) ^ (r & 7)) << 4));
            if (row < p.S && col < p.C)
              *reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.out) + ((size_t)row * p.ldo + col) * (F32 ? 4 : 2)) = o;
          }
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        mbar_arrive_if(ydone(y.s), lane == 0);
      }
      mbar_arrive_if(tile_empty(tile.s), lane == 0);
    }
  }
  if (dead || i0 == i1) griddep_wait();   // the others have, or wait for a warp that has
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    tmem_free<1>(tmem, 256);
  }
}

// --------------------------------------------------------------------------
// launches
// --------------------------------------------------------------------------

Shares shares_of(int S, int C) {
  return Shares((S + kShrinkRows - 1) / kShrinkRows, (C + kChunk - 1) / kChunk, sm_count());
}

struct Maps {
  CUtensorMap x, x1, w, other, base, base1, out;   // x1, base1: row by row, for sorted rows
};

// *mixed: whether going through the rows as they are takes the tiles through many
// more adapters than sorted.  Counted over up to kLooked tiles: neighbours that
// differ, and one, but no more than there are adapters; sorted, a tile takes one
// and each adapter one more.  Five per tile are as many as the sorted rows' way of
// copying costs (16,384 rows at rank 16 in any order of 4 adapters 159 us as they are
// and 202 sorted, of 9 311 and 205, of 256 3430 and 262; in runs of 256 150 and 237).
constexpr int kLooked = 1024;
// by 1,024 threads, the answer in every one
__device__ __forceinline__ bool is_mixed(const int32_t* ids, int S, int n) {
  __shared__ int found[32];
  const int tiles = (S + kTile - 1) / kTile, step = (tiles + kLooked - 1) / kLooked, looked = (tiles + step - 1) / step;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int sum = 0;
#pragma unroll 4
  for (int t = warp; t < looked; t += 32) {
    const long r0 = (long)t * step * kTile;
    int changes = 0;
#pragma unroll
    for (int j = 0; j < kTile / 32; ++j) {
      const long r = r0 + 32 * j + lane;
      changes += __popc(__ballot_sync(0xffffffffu, r > r0 && r < S && __ldg(ids + r) != __ldg(ids + r - 1)));
    }
    sum += min(changes + 1, n);
  }
  if (lane == 0) found[warp] = sum;
  __syncthreads();
  long total = 0;
  for (int w = 0; w < 32; ++w) total += found[w];
  return total * tiles / looked > 5l * tiles + n;
}
__global__ void __launch_bounds__(1024)
mixed_kernel(const int32_t* ids, int S, int n, int32_t* mixed) {
  const bool yes = is_mixed(ids, S, n);
  if (threadIdx.x == 0) *mixed = yes;
}

// The look and, where it says so, the stable sort of up to kSortRows rows by
// adapter, by one CTA: a warp counts and then places the rows of its share, 32 at
// a time, in their order.  perm: the rows' numbers; place: of each row, its place
// (-1: no adapter); *kept: how many have one.
constexpr int kSortRows = 16384, kSortAdapters = 1024, kSortPitch = 33;   // pitch: of an adapter's counts, a warp each
__global__ void __launch_bounds__(1024)
sort_kernel(const int32_t* ids, int S, int n, int32_t* mixed, int32_t* perm, int32_t* place, int32_t* kept) {
  extern __shared__ int count[];     // [n][kSortPitch], and [n]
  __shared__ int sums[32];
  griddep_launch_dependents();
  int* first = count + n * kSortPitch;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool yes = is_mixed(ids, S, n);
  if (threadIdx.x == 0) *mixed = yes;
  if (!yes) return;
  for (int i = threadIdx.x; i < n * kSortPitch; i += 1024) count[i] = 0;
  __syncthreads();
  const int per = (S + 1023) / 1024 * 32, r0 = warp * per, r1 = min(S, r0 + per);
  auto each = [&](auto&& f) {        // f(row, adapter or -1, lanes of the same one)
    for (int r = r0; r < r1; r += 32) {
      const int row = r + lane, id = row < r1 ? __ldg(ids + row) : -1, e = id >= 0 && id < n ? id : -1;
      f(row, e, __match_any_sync(0xffffffffu, e));
      __syncwarp();
    }
  };
  each([&](int, int e, uint32_t same) {
    if (e >= 0 && __ffs(same) - 1 == lane) count[e * kSortPitch + warp] += __popc(same);
  });
  __syncthreads();
  auto scan = [&](int v) {           // of a warp, up to and with this lane
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += u;
    }
    return v;
  };
  for (int e = warp; e < n; e += 32) {
    const int v = count[e * kSortPitch + lane], up = scan(v);
    count[e * kSortPitch + lane] = up - v;
    if (lane == 31) first[e] = up;
  }
  __syncthreads();
  const int mine = (int)threadIdx.x < n ? first[threadIdx.x] : 0, up = scan(mine);   // n is at most 1,024
  if (lane == 31) sums[warp] = up;
  __syncthreads();
  int before = 0, all = 0;
  for (int w = 0; w < 32; ++w) {
    before += w < warp ? sums[w] : 0;
    all += sums[w];
  }
  if ((int)threadIdx.x < n) first[threadIdx.x] = before + up - mine;
  if (threadIdx.x == 0) *kept = all;
  __syncthreads();
  each([&](int row, int e, uint32_t same) {
    int* const at = count + e * kSortPitch + warp;
    const int to = e >= 0 ? first[e] + *at + __popc(same & ((1u << lane) - 1)) : -1;
    __syncwarp();
    if (e >= 0 && __ffs(same) - 1 == lane) *at += __popc(same);
    if (row < r1) place[row] = to;
    if (to >= 0) perm[to] = row;
  });
}

template <int DT, bool TRANS, bool F32>
cudaError_t launch_pair(const Maps& m, LoraParams s, LoraParams x, cudaStream_t st) {
  auto* shrink = shrink_kernel<DT, TRANS>;
  auto* expand = expand_kernel<DT, TRANS, F32>;
  static std::atomic<uint64_t> raised{0};   // the shared memory limits, once per device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (bit == 0 || !(raised.load() & bit)) {
    std::lock_guard<std::mutex> lock(attr_mutex());
    e = cudaFuncSetAttribute(shrink, cudaFuncAttributeMaxDynamicSharedMemorySize, kShrinkSmem);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(expand, cudaFuncAttributeMaxDynamicSharedMemorySize, kExpandSmem);
    if (e != cudaSuccess) return e;
    raised.fetch_or(bit);
  }
  // four stages of x, and as many of weights as fit beside them: with five and seven
  // at rank 64 a tile of two adapters waited for weights (16,384 rows backwards 170
  // us, four and eleven 165)
  s.x_stages = 4;
  s.stages = (kShrinkSmem - 1024 - s.x_stages * 2 * kXBytes) / s.w_stage;
  if (s.stages > kMaxStages) s.stages = kMaxStages;
  const long sms = sm_count();
  const dim3 grid((unsigned)s.shrink_ctas), block(kShrinkThreads);
  const size_t smem = 1024 + s.x_stages * 2 * kXBytes + s.stages * s.w_stage;
  if (s.mixed) {
    e = launch_pdl(shrink, grid, block, smem, st, m.x, m.x1, m.w, s);
  } else {
    shrink<<<grid, block, smem, st>>>(m.x, m.x1, m.w, s);
    e = cudaGetLastError();
  }
  if (e != cudaSuccess) return e;
  x.u_bytes = (terms_of(DT, F32) * x.r16 + 63) / 64 * kXBytes;
  // two tiles of u where three items of base and two of weights fit beside them;
  // then as many items of base as fit, up to four, and of weights (16,384 x 6144
  // bf16 at rank 64: four and three 113 us for both kernels, three and four 121)
  x.u_stages = 1024 + 2 * x.u_bytes + 2 * x.w_stage + 3 * 2 * kXBytes <= kExpandSmem ? 2 : 1;
  x.y_stages = 0;
  for (int w = 4; w >= 2; --w) {
    const int y = (kExpandSmem - 1024 - x.u_stages * x.u_bytes - w * x.w_stage) / (2 * kXBytes);
    if (x.y_stages < 4 && y > x.y_stages) {
      x.y_stages = y < 4 ? y : 4;
      x.stages = w;
    }
  }
  const int rest = 1024 + x.u_stages * x.u_bytes + x.stages * x.w_stage;
  const long items = (long)((x.S + kTile - 1) / kTile) * ((x.C + cols_of(F32) - 1) / cols_of(F32));
  return launch_pdl(expand, dim3((unsigned)(items < sms ? items : sms)), dim3(kExpandThreads), rest + x.y_stages * 2 * kXBytes,
                    st, m.other, m.base, m.base1, m.out, x);
}

// x [S, C] times the adapters' w [n, r, C] (TRANS: [n, C, r]), and that times
// the other factor [n, C', r] (TRANS: [n, r, C']), onto out.
template <bool TRANS>
situ_status launch_tiles(int dtype, bool f32, const void* rows, int64_t ld_rows, const void* w, const void* other, LoraParams s,
                         LoraParams x, cudaStream_t st) {
  const uint64_t S = (uint64_t)s.S, C = (uint64_t)s.C, O = (uint64_t)x.C, r = (uint64_t)s.r, n = (uint64_t)s.n;
  s.r16 = x.r16 = (s.r + 15) / 16 * 16;
  s.chunks = (s.C + kChunk - 1) / kChunk;
  const Shares shares = shares_of(s.S, s.C);
  s.shrink_ctas = x.shrink_ctas = shares.ctas;
  s.least = x.least = shares.least;
  s.run = f32 ? 1024 / kChunk : s.chunks;
  x.chunks = s.chunks;
  const int boxes = (s.r + 63) / 64;
  s.w_stage = TRANS ? boxes * 8192 : (s.r16 * 128 + 1023) / 1024 * 1024;
  const int rrows = s.r16 < 64 ? s.r16 : 64;
  const int cols = cols_of(f32);
  x.w_stage = TRANS ? boxes * (cols / 64) * rrows * 128 : boxes * cols * 128;
  const CUtensorMapDataType dt = dtype == SITU_DT_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  Maps m;
  const uint64_t dx[2] = {C, S}, sx[1] = {(uint64_t)ld_rows * 2};
  const uint32_t bx[2] = {64, kTile}, bx1[2] = {64, 1};
  bool ok = make_map_nd(&m.x, dt, rows, 2, dx, sx, bx);
  m.x1 = m.x;
  if (s.mixed) ok = ok && make_map_nd(&m.x1, dt, rows, 2, dx, sx, bx1);
  if (TRANS) {
    const uint64_t dw[3] = {r, C, n}, sw[2] = {r * 2, r * C * 2}, dof[3] = {O, r, n}, so[2] = {O * 2, r * O * 2};
    const uint32_t bw[3] = {64, kChunk, 1}, bo[3] = {64, (uint32_t)rrows, 1};
    ok = ok && make_map_nd(&m.w, dt, w, 3, dw, sw, bw) && make_map_nd(&m.other, dt, other, 3, dof, so, bo);
  } else {
    const uint64_t dw[3] = {C, r, n}, sw[2] = {C * 2, r * C * 2}, dof[3] = {r, O, n}, so[2] = {r * 2, r * O * 2};
    const uint32_t bw[3] = {64, (uint32_t)s.r16, 1}, bo[3] = {64, (uint32_t)cols, 1};
    ok = ok && make_map_nd(&m.w, dt, w, 3, dw, sw, bw) && make_map_nd(&m.other, dt, other, 3, dof, so, bo);
  }
  const uint64_t dy[2] = {O, S}, el = f32 ? 4 : 2, syo[1] = {(uint64_t)x.ldo * el};
  const uint32_t by[2] = {(uint32_t)cols / 2, kTile};
  const CUtensorMapDataType ot = f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : dt;
  ok = ok && make_map_nd(&m.out, ot, x.out, 2, dy, syo, by);
  m.base = m.base1 = m.out;
  if (x.base) {
    const uint64_t syb[1] = {(uint64_t)x.ld_base * el};
    const uint32_t by1[2] = {(uint32_t)cols / 2, 1};
    ok = ok && make_map_nd(&m.base, ot, x.base, 2, dy, syb, by);
    if (s.mixed) ok = ok && make_map_nd(&m.base1, ot, x.base, 2, dy, syb, by1);
  }
  if (!ok) return SITU_ERR_CUDA;
  constexpr int kB = SITU_DT_BF16, kF = SITU_DT_F16;
  const cudaError_t e = dtype == kB ? (f32 ? launch_pair<kB, TRANS, true>(m, s, x, st) : launch_pair<kB, TRANS, false>(m, s, x, st))
                                    : (f32 ? launch_pair<kF, TRANS, true>(m, s, x, st) : launch_pair<kF, TRANS, false>(m, s, x, st));
  return e == cudaSuccess ? SITU_OK : SITU_ERR_CUDA;
}

// Whether rows named by ids are looked at and, where they are mixed, sorted by
// adapter first.  The look costs 5 us by one CTA (8 to 17 with the permute's kernels,
// which run whatever it says) also where the rows come in runs, so with up to 16
// adapters it is taken only where any order would cost some 70 us more than
// sorted rows: 16,384 rows at rank 16 of 9 adapters 311 and 205 us, of 16 515 and 211.
// One CTA sorts up to kSortRows: 16,384 rows of 64 adapters in any order 228 us and in
// runs 112, with the permute's kernels 213 and 124; half as many, no difference mixed.
bool sortable(int S, int n) {
  return n <= SITU_MAX_LOCAL_EXPERTS && (n > 16 || (n > 8 && (long)S * (n - 5) > 40000));
}
bool by_one_cta(int S, int n) { return S <= kSortRows && n <= kSortAdapters; }
// A cluster per row, or tiles.  A row's cluster reads its adapter whatever the
// others take: 4 us and about 0.07 a row at rank 16, in proportion to the rank above
// (3584 x 6144).  Tiles take 15 us, and about 1.3 at low ranks and 2.6 at 128 for each
// adapter that rows of a tile take: in any order up to n of them, sorted, for 16
// us, as many as 256 rows hold.  By rows and in tiles, us: 128 rows at rank 16 of one
// adapter 14 and 16, 256 20 and 17, 512 of 16 adapters 37 and 52 (30 where they come in
// runs), 1,024 of 64 70 and 62; at rank 64 32 rows of one 14 and 17, 64 22 and 17, 128
// of 64 48 and 103, 512 of 256 175 and 403; at rank 128 64 of one 40 and 21, of 16 39
// and 52.
bool by_rows(int S, int r, int n) {
  const float each = 1.3f * (1.f + r / 128.f), mixed = each * (n < kTile ? n : kTile);
  const float sorted = sortable(S, n) ? 16.f + each * (1.f + 256.f * n / S) : mixed;
  return 4.f + (float)S * (r < 16 ? 16 : r) / 244.f <= 15.f + (mixed < sorted ? mixed : sorted);
}
// its scratch: *mixed; numbers, places; counts, offsets, the permute's own
size_t sort_ints(int S, int n) { return 1 + 2 * (size_t)S + 2 * (size_t)n + 1 + permute_scratch_bytes(S, 1, n) / 4; }

size_t part_bytes(int S, int C, int r) { return S == 0 ? 0 : (size_t)shares_of(S, C).most * S * r * 4; }

// of the backward pass: first the parts of v, then those of the gradients
size_t shared_bytes(int S, int N, int r) {
  const size_t a = part_bytes(S, N, r), b = outer_bytes(r);
  return a > b ? a : b;
}
// behind them v, and for f16 u, its rows' largest and the adapters' largest of both
size_t kept_bytes(int S, int r) { return (size_t)S * r * 4 + 32; }
size_t row_bytes(int S) { return ((size_t)S * 4 + 31) / 32 * 32; }
constexpr size_t kMostBytes = 2 * SITU_GEMM_MAX_GROUPS * 4;

bool bad_extent(int C) { return C < 8 || C % 8 != 0 || C > SITU_GEMM_MAX_DIM; }
bool bad_sizes(int S, int K, int N, int r, int n) {
  return S < 0 || S > SITU_GEMM_MAX_ROWS || bad_extent(K) || bad_extent(N) || r < 8 || r % 8 != 0 || r > kMaxRank || n < 1 ||
         n > SITU_LORA_MAX_ADAPTERS;
}

}  // namespace
}  // namespace situ

extern "C" size_t situ_moe_lora_workspace_size(int32_t S, int32_t K, int32_t N, int32_t r, int32_t n) {
  using namespace situ;
  if (bad_sizes(S, K, N, r, n) || S == 0 || by_rows(S, r, n)) return 0;
  return part_bytes(S, K, r) + (sortable(S, n) ? (sort_ints(S, n) * 4 + 31) / 32 * 32 : 0);
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
  if (by_rows(a->S, a->r, a->n)) {
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
  if (bad(workspace, 31) || bad(a->device_status, 3)) return SITU_ERR_MISALIGNED;
  if (workspace_bytes < situ_moe_lora_workspace_size(a->S, a->K, a->N, a->r, a->n)) return SITU_ERR_WORKSPACE_TOO_SMALL;
  LoraParams s = {};
  s.ids = a->ids;
  s.offsets = a->offsets;
  s.S = a->S;
  s.r = a->r;
  s.n = a->n;
  s.part = static_cast<float*>(workspace);
  s.scale = a->scale;
  s.err = a->device_status;
  if (a->ids && sortable(a->S, a->n)) {
    int32_t* mixed = reinterpret_cast<int32_t*>(static_cast<uint8_t*>(workspace) + part_bytes(a->S, a->K, a->r));
    int32_t *perm = mixed + 1, *place = perm + a->S, *counts = place + a->S, *offsets = counts + a->n,
            *scratch = offsets + a->n + 1;
    bool ok;
    if (by_one_cta(a->S, a->n)) {
      const size_t smem = (size_t)a->n * (kSortPitch + 1) * 4;
      ok = smem <= 40 * 1024 ||      // 48 KB with the static part
           cudaFuncSetAttribute(sort_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                kSortAdapters * (kSortPitch + 1) * 4) == cudaSuccess;
      if (ok) sort_kernel<<<1, 1024, smem, st>>>(a->ids, a->S, a->n, mixed, perm, place, offsets + a->n);
      ok = ok && cudaGetLastError() == cudaSuccess;
    } else {
      mixed_kernel<<<1, 1024, 0, st>>>(a->ids, a->S, a->n, mixed);
      ok = cudaGetLastError() == cudaSuccess &&
           launch_permute(a->ids, a->S, 1, a->n, 0, 1, counts, offsets, nullptr, nullptr, perm, place, nullptr, scratch, st) ==
               cudaSuccess;
    }
    if (!ok) return SITU_ERR_CUDA;
    s.mixed = mixed;
    s.perm = perm;
    s.place = place;
    s.kept = offsets + a->n;
  }
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
  return shared_bytes(S, N, r) + 2 * kept_bytes(S, r) + row_bytes(S) + kMostBytes;
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
  const void* ptrs[] = {a->dy, a->x, a->a, a->b, a->u, a->dx0, a->dx, a->da, a->db};
  for (const void* q : ptrs)
    if (bad(q, 15)) return SITU_ERR_MISALIGNED;
  if (bad(workspace, 31)) return SITU_ERR_MISALIGNED;
  if (bad(a->offsets, 3) || bad(a->scale, 3) || bad(a->device_status, 3) || bad(a->dy_scale, 3)) return SITU_ERR_MISALIGNED;
  if (workspace_bytes < situ_moe_lora_backward_workspace_size(a->S, a->K, a->N, a->r)) return SITU_ERR_WORKSPACE_TOO_SMALL;
  uint8_t* v = static_cast<uint8_t*>(workspace) + shared_bytes(a->S, a->N, a->r);
  FarParams far = {};
  if (a->dtype == SITU_DT_F16) {
    uint8_t* u32 = v + kept_bytes(a->S, a->r);
    uint8_t* row_most = u32 + kept_bytes(a->S, a->r);
    far.u = static_cast<const uint16_t*>(a->u);
    far.x = static_cast<const uint16_t*>(a->x);
    far.a = static_cast<const uint16_t*>(a->a);
    far.ldx = (long)a->ldx;
    far.K = a->K;
    far.u32 = reinterpret_cast<float*>(u32);
    far.row_most = reinterpret_cast<float*>(row_most);
    far.most = reinterpret_cast<uint32_t*>(row_most + row_bytes(a->S));
  }
  OuterArgs o;
  o.dtype = a->dtype;
  o.S = a->S;
  o.K = a->K;
  o.N = a->N;
  o.r = a->r;
  o.n = a->n;
  o.x = a->x;
  o.dy = a->dy;
  o.v = v;
  o.u = a->u;
  o.u32 = far.u32;
  o.row_most = far.row_most;
  o.most = far.most;
  o.dy_scale = a->dy_scale;
  o.ldx = a->ldx;
  o.ld_dy = a->ld_dy;
  o.offsets = a->offsets;
  o.da = a->da;
  o.db = a->db;
  o.parts = static_cast<float*>(workspace);             // u's parts have been read
  o.err = a->device_status;
  if (a->S > 0) {
    LoraParams s = {};
    s.offsets = a->offsets;
    s.S = a->S;
    s.r = a->r;
    s.n = a->n;
    s.part = static_cast<float*>(workspace);
    s.scale = a->scale;
    s.err = a->device_status;
    s.far = far;
    s.times = a->dy_scale;
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
    return t != SITU_OK ? t : launch_outer(o, (cudaStream_t)stream);
  }
  const bool zero = cudaMemsetAsync(a->da, 0, (size_t)a->n * a->r * a->K * 2, (cudaStream_t)stream) == cudaSuccess &&
                    cudaMemsetAsync(a->db, 0, (size_t)a->n * a->N * a->r * 2, (cudaStream_t)stream) == cudaSuccess;
  return zero ? SITU_OK : SITU_ERR_CUDA;
}
