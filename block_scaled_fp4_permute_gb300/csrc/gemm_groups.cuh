// gemm_groups.cuh -- what the products over ragged expert groups share: the
// groups' row ranges and their token tiles, the tile walk, the CTA-pair forms
// of the tcgen05 and mbarrier instructions, and the tensor-map encoders.
//
// Rows are sorted by expert: group e holds rows [offsets[e], offsets[e + 1]).
// The offsets live on the device (the permute writes them), so the host never
// sees them: grids are sized for the GPU, and every CTA scans the groups'
// bounds and tile counts into shared memory once and walks its share of the
// tiles (the weight gradient, whose tiles do not depend on the rows and whose
// shared memory is full, reads the bounds of each tile).
// Offsets are clamped to [0, S] and to ascending order before use: group e
// starts at the largest of offsets[0..e] and ends at the largest of
// offsets[0..e + 1].  So whatever the array holds, the groups are disjoint,
// lie inside the operands and have S rows together at most.
#pragma once
#include "situ_internal.h"
#include "tc_common.cuh"

namespace situ {
namespace gg {

using namespace tc;

constexpr int kMaxGroups = 1024;
constexpr int kScanInts = 2 * (kMaxGroups + 1);   // of a scan in shared memory
constexpr int64_t kMaxStride = int64_t(1) << 39;   // elements; the tensor maps' own limit is 2^40 bytes

__host__ __device__ __forceinline__ int offset_at(const int32_t* off, int i, int S) {
#ifdef __CUDA_ARCH__
  const int v = __ldg(off + i);
#else
  const int v = off[i];
#endif
  return v < 0 ? 0 : v < S ? v : S;
}
// (first row, rows) of group e; ascending offsets, the usual case, need no
// look at the groups before
__host__ __device__ __forceinline__ int2 group_rows(const int32_t* off, int e, int S, bool ascending) {
  int b = offset_at(off, e, S);
  const int end = offset_at(off, e + 1, S);
  if (!ascending) {
#pragma unroll 1
    for (int i = 0; i < e; ++i) {
      const int o = offset_at(off, i, S);
      b = o > b ? o : b;
    }
  }
  return make_int2(b, end > b ? end - b : 0);
}
// Whether the offsets that this one of the block's `threads` threads looks at ascend.
__device__ __forceinline__ bool offsets_ascend(const int32_t* off, int E, int S, int threads) {
  bool ok = true;
  for (int e = threadIdx.x; e < E; e += threads) ok = ok && offset_at(off, e, S) <= offset_at(off, e + 1, S);
  return ok;
}

// tp[e] = token tiles of the groups before e, tp[E] = all of them; row[e] =
// the first row of e, row[E] = the end of the last (E <= kMaxGroups).  Called
// by all `threads` threads of the block; ends synced.
__device__ __forceinline__ void scan_tiles(const int32_t* off, int E, int S, int tile, int* tp, int* row, int threads) {
  __shared__ int warp_sum[32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (off == nullptr) {   // one dense group
    if (tid == 0) {
      tp[0] = row[0] = 0;
      tp[1] = (S + tile - 1) / tile;
      row[1] = S;
    }
    __syncthreads();
    return;
  }
  const int per = (E + threads - 1) / threads;
  int cnt[(kMaxGroups + 255) / 256], sum = 0;   // blocks here have at least 256 threads
  bool ok = true;
#pragma unroll
  for (int j = 0; j < (kMaxGroups + 255) / 256; ++j) {
    const int e = tid * per + j;
    cnt[j] = 0;
    if (j < per && e < E) {
      const int from = offset_at(off, e, S), to = offset_at(off, e + 1, S);
      row[e] = from;
      if (e == E - 1) row[E] = to;
      ok = ok && from <= to;
      cnt[j] = (to - from + tile - 1) / tile;
    }
    sum += cnt[j];
  }
  int inc = sum;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, inc, d);
    if (lane >= d) inc += o;
  }
  if (lane == 31) warp_sum[warp] = inc;
  const bool ascending = __syncthreads_and(ok);
  int base = 0;
  for (int w = 0; w < warp; ++w) base += warp_sum[w];
  int run = base + inc - sum;
#pragma unroll
  for (int j = 0; j < (kMaxGroups + 255) / 256; ++j) {
    const int e = tid * per + j;
    if (j < per && e < E) tp[e] = run;
    run += cnt[j];
  }
  if (tid == threads - 1) tp[E] = base + inc;
  __syncthreads();
  if (!ascending) {   // counted anew from the clamped order, by one thread
    if (tid == 0) {
      tp[0] = 0;
#pragma unroll 1
      for (int e = 0; e < E; ++e) {
        row[e + 1] = max(row[e + 1], row[e]);
        tp[e + 1] = tp[e] + (row[e + 1] - row[e] + tile - 1) / tile;
      }
    }
    __syncthreads();
  }
}

// the group of token tile v: the largest e with tp[e] <= v (v < tp[E])
__device__ __forceinline__ int find_group(const int* tp, int E, int v) {
  int lo = 0, hi = E;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (tp[mid] <= v) lo = mid;
    else hi = mid;
  }
  return lo;
}

// ---------------------------------------------------------------------------
// CTA pairs
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// the shared::cluster address of `a` in the pair's even CTA
__device__ __forceinline__ uint32_t leader_addr(uint32_t a) { return a & 0xFEFFFFFFu; }
// One arrival where p holds, as a predicated instruction without a branch: on
// a barrier of this CTA, or of CTA `rank` of the cluster.  The latter orders
// tensor memory reads (with the tcgen05 fences around it) and nothing in
// global memory: with release at cluster scope it would wait for the thread's
// output stores, about 1 us each time.
__device__ __forceinline__ void mbar_arrive_if(uint32_t a, bool p) {
  asm volatile("{\n .reg .pred q;\n setp.ne.b32 q, %1, 0;\n @q mbarrier.arrive.shared::cta.b64 _, [%0];\n}" ::"r"(a),
               "r"((uint32_t)p)
               : "memory");
}
__device__ __forceinline__ void mbar_arrive_at_if(uint32_t a, uint32_t rank, bool p) {
  asm volatile(
      "{\n .reg .pred q;\n .reg .b32 r;\n setp.ne.b32 q, %2, 0;\n mapa.shared::cluster.u32 r, %0, %1;\n"
      " @q mbarrier.arrive.shared::cluster.b64 _, [r];\n}" ::"r"(a),
      "r"(rank), "r"((uint32_t)p)
      : "memory");
}

__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}

template <int CG>
__device__ __forceinline__ void tmem_alloc(uint32_t dst, uint32_t cols) {
  if (CG == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst), "r"(cols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  } else {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst), "r"(cols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
}
template <int CG>
__device__ __forceinline__ void tmem_free(uint32_t tmem, uint32_t cols) {
  if (CG == 1)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(cols) : "memory");
  else
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(cols) : "memory");
}
// one arrival on `bar` of every CTA of the group once the MMAs issued so far are done
template <int CG>
__device__ __forceinline__ void commit(uint32_t bar) {
  if (CG == 1) {
    mma_commit(bar);
  } else {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
        "h"((uint16_t)3)
        : "memory");
  }
}
template <int CG>
__device__ __forceinline__ void mma_f16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  if (CG == 1)
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
  else
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}
template <int CG>
__device__ __forceinline__ void mma_f8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  if (CG == 1)
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
  else
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}

// Tile copies.  In a pair both CTAs' copies complete on the even CTA's
// barrier (it alone issues the MMAs).
template <int CG>
__device__ __forceinline__ void copy_2d(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
  if (CG == 1)
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
            dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], "
        "[%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(leader_addr(bar))
        : "memory");
}
template <int CG>
__device__ __forceinline__ void copy_3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
  if (CG == 1)
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
            dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, "
        "%4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(leader_addr(bar))
        : "memory");
}
// four rows named by index (a map whose box is one row high); an index past
// the map's last row gives zeros
template <int CG>
__device__ __forceinline__ void copy_rows4(uint32_t dst, const CUtensorMap* map, int x, int r0, int r1, int r2, int r3,
                                           uint32_t bar) {
  if (CG == 1)
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, "
        "%4, %5, %6}], [%7];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(r0), "r"(r1), "r"(r2), "r"(r3), "r"(bar)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes [%0], "
        "[%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(r0), "r"(r1), "r"(r2), "r"(r3), "r"(leader_addr(bar))
        : "memory");
}

// tcgen05 descriptor of an operand whose M or N elements are contiguous
// (MN-major, 128-byte swizzle): chunks of 64 elements x `rows` contraction
// rows of 128 bytes, `chunk` bytes apart; 8-row groups are 1,024 bytes apart.
__device__ __forceinline__ uint64_t sdesc_mn(uint32_t a, uint32_t chunk) {
  uint64_t d = 0;
  d |= (uint64_t)((a >> 4) & 0x3FFFu);
  d |= (uint64_t)(chunk >> 4) << 16;   // leading byte offset: the next 64 elements
  d |= (uint64_t)(1024u >> 4) << 32;   // stride byte offset: the next 8 contraction rows
  d |= (uint64_t)1u << 46;
  d |= (uint64_t)2u << 61;
  return d;
}

// mbar_wait by a converged warp, the usual case (the phase completes within
// the first try, which itself waits a while) without a vote: 60 clocks instead
// of 88.  A lane that did not see the phase complete tries again; if another
// lane saw it, so does this one then, so the lanes' answers agree.
__device__ __forceinline__ bool mbar_wait_slow(uint32_t a, uint32_t parity, int* err, int code) {
  return __all_sync(__activemask(), mbar_wait(a, parity, err, code));
}
__device__ __forceinline__ bool warp_wait(uint32_t a, uint32_t parity, int* err, int code) {
  bool ok = mbar_try(a, parity);
  if (!ok) ok = mbar_wait_slow(a, parity, err, code);
  __syncwarp();
  return ok;
}
// two barriers at once
__device__ __forceinline__ bool warp_wait2(uint32_t a, uint32_t pa, uint32_t b, uint32_t pb, int* err, int code) {
  const bool oa = mbar_try(a, pa), ob = mbar_try(b, pb);
  bool ok = oa && ob;
  if (!ok) ok = mbar_wait_slow(a, pa, err, code) && mbar_wait_slow(b, pb, err, code + 1);
  __syncwarp();
  return ok;
}

// A place in a ring of N and the parity of its current round.
template <int N>
struct Ring {
  int s = 0;
  uint32_t ph = 0;
  int used = 0;   // steps taken, up to N
  __host__ __device__ __forceinline__ void next() {
    if (used < N) ++used;
    if (++s == N) {
      s = 0;
      ph ^= 1;
    }
  }
};

// Bounded wait (kWaitNs) for what this CTA itself put in flight, on the way
// out after a failure; unlike mbar_wait it does not give up on another CTA's
// error.
__device__ __forceinline__ bool drain_wait(uint32_t a, uint32_t parity) {
  const unsigned long long t0 = globaltimer();
  while (!mbar_try(a, parity))
    if (globaltimer() - t0 > kWaitNs) return false;
  return true;
}

// wait(stage, parity) for the last use of each stage of a ring; whether all came
template <int N, class Wait>
__host__ __device__ __forceinline__ bool last_uses(const Ring<N>& r, Wait&& wait) {
  bool ok = true;
  for (int j = 0; j < r.used; ++j) ok = wait(j, j < r.s ? r.ph : r.ph ^ 1) && ok;
  return ok;
}
// the same for the ring's last stage alone: it stands for all where each use
// ends after those before it, as MMAs committed by one thread do
template <int N, class Wait>
__host__ __device__ __forceinline__ bool last_use(const Ring<N>& r, Wait&& wait) {
  return r.used == 0 || (r.s > 0 ? wait(r.s - 1, r.ph) : wait(N - 1, r.ph ^ 1));
}
// How a warp that puts copies or MMAs in flight leaves: ok, it has been through
// all of its stages, and then arrived() tells whether their last uses are over.
// If a wait was given up, here or before (an error of any CTA ends them all),
// that is not known, and drain() waits for what this warp has in flight, so that
// none of it reaches into shared memory or TMEM that is no longer the CTA's.
template <class Arrived, class Drain>
__host__ __device__ __forceinline__ void leave(bool ok, Arrived&& arrived, Drain&& drain) {
  if (ok) ok = arrived();
  if (!ok) drain();
}
// drain() of copies that complete on the other CTA's barriers
__device__ __forceinline__ void pause_2ms() {
  const unsigned long long t0 = globaltimer();
  while (globaltimer() - t0 < 2000000ull) {
  }
}

// tcgen05.ld of 32 columns, without the wait
__device__ __forceinline__ void tmem_ld32_nowait(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld16_nowait(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
// waits for the loads above and ties their registers to the wait, so that no
// use of them moves ahead of it
template <int N>
__device__ __forceinline__ void tmem_ld_wait(uint32_t* r) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[i]));
}

// tcgen05.ld of 16 lanes x 32 columns as 8 x 8 fragments: thread t gets, of
// eight columns i, elements (t / 4, 2 (t % 4)), (.., + 1) in r[4 i], r[4 i + 1]
// and those of row t / 4 + 8 in r[4 i + 2], r[4 i + 3]
__device__ __forceinline__ void tmem_ld_frag_nowait(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
// four 8 x 8 matrices of 16-bit elements stored transposed; lane l names the
// 16 bytes of row l % 8 of matrix l / 8
__device__ __forceinline__ void store_transposed(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b),
               "r"(c), "r"(d)
               : "memory");
}

// ---------------------------------------------------------------------------
// Split contractions: a cluster of up to 8 CTAs takes one tile, each a part of
// the contraction, and adds the parts up through distributed shared memory in
// the order of the ranks (so the result does not depend on timing).  For
// launches whose tiles alone would leave most of the GPU idle.
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ float2 peer_f32x2(uint32_t addr, uint32_t rank) {
  float2 v;
  asm volatile("{\n .reg .b32 r;\n mapa.shared::cluster.u32 r, %2, %3;\n ld.shared::cluster.v2.f32 {%0, %1}, [r];\n}"
               : "=f"(v.x), "=f"(v.y)
               : "r"(addr), "r"(rank));
  return v;
}
// The parts [cols][pitch] at `part` of every CTA (128 sums of a row in use),
// added up; emit(col, m, sums of m and m + 1) for this CTA's share, over n threads of which this is number t.
template <class Emit>
__device__ __forceinline__ void join_parts(uint32_t part, int pitch, int cols, int t, int n, Emit&& emit) {
  const uint32_t ranks = cluster_size();
  for (int i = (int)cluster_rank() * n + t; i < cols * 64; i += (int)ranks * n) {
    const int col = i >> 6, m = 2 * (i & 63);
    float2 s = make_float2(0.f, 0.f);
    for (uint32_t r = 0; r < ranks; ++r) {
      const float2 v = peer_f32x2(part + (uint32_t)(col * pitch + m) * 4, r);
      s.x += v.x;
      s.y += v.y;
    }
    emit(col, m, s);
  }
}
__device__ __forceinline__ float4 peer_f32x4(uint32_t addr, uint32_t rank) {
  float4 v;
  asm volatile(
      "{\n .reg .b32 r;\n mapa.shared::cluster.u32 r, %4, %5;\n ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [r];\n}"
      : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
      : "r"(addr), "r"(rank));
  return v;
}
// The most token tiles of `tile` rows that S rows in E groups can take: G
// groups with rows, r each, take floor((r - 1) / tile) + 1, together at most
// G + floor((S - G) / tile), which grows with G.
inline double most_tiles(int S, int E, int tile) {
  const int G = S < E ? S : E;
  return (double)G + (S - G) / tile;
}
// zeros to rows [from, to) of a row-major output (width and pitch in bytes,
// multiples of 16), spread over `n` threads of which this is number `t`
__device__ __forceinline__ void zero_rows(uint8_t* out, long from, long to, size_t width, size_t pitch, long t, long n) {
  const long per = (long)(width / 16);
  for (long i = t; i < (to - from) * per; i += n)
    *reinterpret_cast<uint4*>(out + (size_t)(from + i / per) * pitch + (size_t)(i % per) * 16) = make_uint4(0, 0, 0, 0);
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

// The map encoder needs a current context, which a host thread that has made
// no runtime call yet (autograd's backward threads) does not have: binds the
// thread to its device's primary context, once.
inline bool bind_thread() {
  static thread_local bool bound = false;
  if (!bound) {
    int dev = 0;
    bound = cudaGetDevice(&dev) == cudaSuccess && cudaSetDevice(dev) == cudaSuccess;
  }
  return bound;
}

// dims[i] elements, stride[i - 1] bytes between elements of dims[i] (i >= 1)
inline bool make_map_nd(CUtensorMap* m, CUtensorMapDataType dt, const void* base, int nd, const uint64_t* dims,
                        const uint64_t* strides, const uint32_t* box,
                        CUtensorMapSwizzle swizzle = CU_TENSOR_MAP_SWIZZLE_128B) {
  PFN_cuTensorMapEncodeTiled_v12000 fn = encode_fn();
  if (!fn || !bind_thread()) return false;
  const cuuint32_t estr[3] = {1, 1, 1};
  cuuint64_t d[3], st[2];
  cuuint32_t b[3];
  for (int i = 0; i < nd; ++i) {
    d[i] = dims[i];
    b[i] = box[i];
    if (i > 0) st[i - 1] = strides[i - 1];
  }
  return fn(m, dt, (cuuint32_t)nd, const_cast<void*>(base), d, st, b, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// SMs of the current device (looked up once per device)
inline int sm_count() {
  static std::atomic<int> known[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  int n = dev < 64 ? known[dev].load() : 0;
  if (n == 0) {
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    if (dev < 64) known[dev].store(n);
  }
  return n;
}

// Raises a kernel's dynamic shared memory limit once per device, then
// launches it in clusters of `cluster` CTAs.
template <class Kernel, class... Args>
cudaError_t launch_cluster(Kernel k, std::atomic<uint64_t>* raised, int cluster, int grid, int threads, size_t smem,
                           cudaStream_t st, Args&&... args) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (bit == 0 || !(raised->load() & bit)) {
    std::lock_guard<std::mutex> lock(attr_mutex());
    e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    raised->fetch_or(bit);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)cluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, k, args...);
}

// How many clusters of c CTAs (one per SM) the current device holds at once
// (152, 76, 46, 36, 28, 23, 15, 15 of 1 to 8 here: clusters do not span the
// GPU's processing clusters).  Asked once per device; k is any of the kernels
// that fill an SM.
template <class Kernel>
int clusters_at_once(Kernel k, int threads, size_t smem, int c) {
  static std::atomic<int> known[64][9];
  int dev = 0;
  if (c < 1 || c > 8 || cudaGetDevice(&dev) != cudaSuccess) return 0;
  int n = dev < 64 ? known[dev][c].load() : 0;
  if (n != 0) return n;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)c;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)c);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  {
    std::lock_guard<std::mutex> lock(attr_mutex());
    if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&n, k, &cfg) != cudaSuccess)
      return 0;
  }
  if (dev < 64) known[dev][c].store(n);
  return n;
}
// CTAs per tile: the largest cluster of which the device holds one per tile
// at once and whose CTAs keep at least `least` of the `steps` contraction steps
template <class Kernel>
int split_of(Kernel k, int threads, size_t smem, double tiles, int steps, int least) {
  for (int c = steps / least < 8 ? steps / least : 8; c > 1; --c)
    if (tiles * c <= sm_count() && tiles <= clusters_at_once(k, threads, smem, c)) return c;
  return 1;
}

}  // namespace gg
}  // namespace situ
