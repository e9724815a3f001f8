// grouped_gemm.cu -- 16-bit products over ragged expert groups and their
// gradients on tcgen05 (kind::f16, fp32 accumulation in TMEM).
//
// Rows r of x [S, K] are sorted by expert, e(r) is the group that holds r:
//   forward   y[r, n]     = sum_k  x[r, k]  w[e(r), n, k]
//   dgrad     dx[r, k]    = sum_n  dy[r, n] w[e(r), n, k]
//   wgrad     dw[e, n, k] = sum_{r in e} dy[r, n] x[r, k]
// The weights take the MMA's M side (128 per CTA) in all three and the
// tokens its N side (dw: n and k), so that a ragged group's last tile costs
// an N rounded up to 16, not a whole tile of rows, and a group of few tokens
// streams its weights once.  Operands whose contraction index is contiguous
// are K-major (x, w in the forward, dy in dgrad), the others MN-major (w in
// dgrad; dy and x in wgrad), both as 128-byte-swizzled TMA tiles.
//
// Per CTA: warp 0 copies stages of 64 contraction elements into a ring,
// warp 1 issues the MMAs into two TMEM accumulators in turn, warps 4..11 read
// the accumulator of the previous tile and store it meanwhile.  CTAs are
// persistent and walk the tiles with a fixed stride.
//
// The contraction's end: k and n past the weight's extent read as zeros (the
// maps end there; w is a 3D map, so that rows past n = N do not run into the
// next expert).  In wgrad the contraction runs over a group's rows and ends
// anywhere: a last stage of fewer than 64 rows comes in whole sixteens and one
// gather of the rest, with the rows past the group's end named out of bounds,
// so that the MMA sees zeros in both operands there (a zero in one of them
// would not do: the neighbour's rows may hold infinities).
//
// 16-bit results keep one TMEM sum, up to a length; fp32 results and longer
// contractions take it out every 512 elements and add in registers, because the
// tensor cores' additions truncate (the entry point has the figures).
//
// Large groups run on CTA pairs (cta_group::2, 256 x 256 per pair: each CTA
// copies half of the N-side operand, so a stage is 32 KB per CTA and not 48).
// Launches of few tiles split the contraction over a cluster.
//
// Measured (bf16, 4096 x 3584, 32 experts, 1,024 rows each): forward 0.51 to
// 0.56 ms, dgrad 0.54 to 0.59, wgrad 0.53 to 0.61, that is 1.9 to 1.6 PFLOP/s,
// where cuBLAS sustains 1.70 under the power limit: bound by the tensor cores.
// With 128 rows each 0.16 / 0.15 / 0.18 ms, 1.0 GB at 6.4, 6.8 and 5.5 TB/s:
// forward and dgrad are bound by the weights' bytes, wgrad by its stores (a
// fill of dw reaches 7.7).  One row per expert (896 experts, 768 x 3584): 7.3
// TB/s.
#include "../../include/situ_moe.h"
#include "gemm_groups.cuh"

#include <type_traits>

namespace situ {

using namespace gg;

namespace {

constexpr int kFwd = SITU_GROUPED_FORWARD, kDgrad = SITU_GROUPED_DGRAD, kWgrad = SITU_GROUPED_WGRAD;
constexpr int kBK = 64;             // contraction elements per stage
constexpr int kABytes = 128 * 128;  // 128 weights (or n) x 64 elements
constexpr int kBoxRows = 32;        // token rows per copy (forward, dgrad)
constexpr int kThreads = 384;
constexpr int kEpiWarp = 4;         // first of the eight epilogue warps: two per TMEM lane quarter
constexpr int kEpiThreads = 256;
constexpr int kSplitLeast = 8;      // stages that a CTA of a split tile takes at least
constexpr int kSumStages = 8;       // stages summed in TMEM before the fp32 registers take them
constexpr int kOneSum = 0, kSums = 1, kLongSums = 2;   // how a tile is summed, see gg_kernel
constexpr int kLaunchRegs = 168;    // per thread of a launch, what kSplitRegs shares out
constexpr int kPartPitch = 260;     // floats of a row of a split wgrad tile's part: 256 and 4
constexpr int kJoinPitch = 132;     // floats of a token of a split forward or dgrad tile's part
constexpr int kOutPitch = 80;       // bytes of a staged token row: 32 elements and 16 bytes
constexpr int kOutPitchF = 144;     // the same of 32 floats; 16 rows
static_assert(16 * kOutPitchF <= 32 * kOutPitch, "staging");

struct GgParams {
  const int32_t* offsets;
  int E, S;
  int M, L, Ncol;   // M side extent; contraction (fwd, dgrad); N side extent (wgrad)
  int n_mt, n_nt;   // M tiles; N tiles (wgrad)
  void* out;
  long ld_out;      // elements
  int bf16, out_f32, accumulate, zero_rest;
  int store8;       // 16-bit dw stored by all eight epilogue warps
  int one_sum;      // stages that 16-bit results take in one TMEM sum at most
  int* err;
};

template <int CG, int MODE, int TN>
struct Cfg {
  static constexpr int kTNB = TN / CG;                // N-side rows of one CTA
  static constexpr int kBBytes = kTNB * 128;
  static constexpr int kStageBytes = kABytes + kBBytes;
  // output staging of the eight epilogue warps: wgrad 4 KB boxes (and no
  // scan), else 32 tokens x 32 elements at a pitch without conflicts (tiles of
  // 32 tokens: four of the warps)
  static constexpr int kOutBytes = MODE == kWgrad ? 8 * 4096 : (TN > 32 ? 8 : 4) * 32 * kOutPitch;
  static constexpr int kTpBytes = MODE == kWgrad ? 0 : 4 * kScanInts;
  static constexpr int kMaxBytes = 232448 - 1024 - kTpBytes - kOutBytes - 512;
  static constexpr int kStages = kMaxBytes / kStageBytes;
  static constexpr int kOffB = kStages * kABytes;
  static constexpr int kOffOut = kOffB + kStages * kBBytes;
  static constexpr int kOffTp = kOffOut + kOutBytes;
  static constexpr int kOffBar = (kOffTp + kTpBytes + 15) / 16 * 16;
  static constexpr int kNumBars = 2 * kStages + 5;    // full, empty; acc_full[2], acc_empty[2]; drain
  static constexpr int kOffTm = kOffBar + 8 * kNumBars;
  static constexpr int kSmem = kOffTm + 16 + 1024;
  static constexpr int kTmemCols = 2 * TN;
  // 256 columns are 128 sums per epilogue thread: warps 0..3 hand registers
  // over (56 * 128 + 224 * 256 = 168 * 384, the launch's total)
  static constexpr bool kSplitRegs = TN >= 256;
  static_assert(kSmem <= 232448 && kTmemCols <= 512 && kTmemCols >= 32, "shared memory and TMEM");
};

__device__ __forceinline__ uint32_t to_16x2(float a, float b, int bf16) {
  return bf16 ? f32x2_to_bf16x2(a, b) : pack_f16x2(a, b);
}
__device__ __forceinline__ float from_16(uint32_t v, int bf16) {
  return bf16 ? __uint_as_float(v << 16) : f16_to_f32(v);
}

// What one tile is: the group's rows, the tile's corner and its N extent.
struct Tile {
  int e, row0, rows;   // group and its rows
  int m0, c0, cols;    // M-side start, N-side start (row in the group; k in wgrad) and extent
  int nk;              // stages
};

// tp: what scan_tiles wrote, first tiles and then rows; wgrad: whether the offsets ascend
template <int CG, int MODE, int TN>
__device__ __forceinline__ Tile tile_of(const GgParams& p, const int* tp, int idx) {
  Tile t;
  int mt;
  if (MODE == kWgrad) {
    const int per = p.n_mt * p.n_nt;
    t.e = idx / per;
    const int r = idx - t.e * per;
    mt = r / p.n_nt;
    t.c0 = (r - mt * p.n_nt) * TN;
    const int2 g = group_rows(p.offsets, t.e, p.S, tp[0] != 0);
    t.row0 = g.x;
    t.rows = g.y;
    t.cols = min(TN, p.Ncol - t.c0);
    t.nk = (t.rows + kBK - 1) / kBK;
  } else {
    t.e = find_group(tp, p.E, idx / p.n_mt);
    const int r = idx - tp[t.e] * p.n_mt, tt = tp[t.e + 1] - tp[t.e];
    mt = r / tt;   // a group's token tiles run side by side: they read the same weights
    t.c0 = (r - mt * tt) * TN;
    const int* row = tp + kMaxGroups + 1;
    t.row0 = row[t.e];
    t.rows = row[t.e + 1] - t.row0;
    t.cols = min(TN, t.rows - t.c0);
    t.nk = (p.L + kBK - 1) / kBK;
  }
  t.m0 = mt * 128 * CG;
  return t;
}

// Where element c of a thread's 32 of a 32-lane x 32-column load lies
// (tmem_ld_frag_nowait of its two halves): lane and column.
__device__ __forceinline__ int frag_row(int c, int lane) { return (lane >> 2) + 8 * ((c >> 1) & 1) + 16 * (c >> 4); }
__device__ __forceinline__ int frag_col(int c, int lane) { return 8 * ((c >> 2) & 3) + 2 * (lane & 3) + (c & 1); }

// dw[at..at + 7] += v
__device__ __forceinline__ void add_dw(const GgParams& p, size_t at, const float* v) {
  if (p.out_f32) {
    float4* dst = reinterpret_cast<float4*>(reinterpret_cast<float*>(p.out) + at);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float4 o = dst[h];
      dst[h] = make_float4(v[4 * h] + o.x, v[4 * h + 1] + o.y, v[4 * h + 2] + o.z, v[4 * h + 3] + o.w);
    }
  } else {
    uint4* dst = reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(p.out) + at);
    const uint4 o = *dst;
    const uint32_t w[4] = {o.x, o.y, o.z, o.w};
    uint32_t r[4];
#pragma unroll
    for (int h = 0; h < 4; ++h)
      r[h] = to_16x2(v[2 * h] + from_16(w[h] & 0xFFFFu, p.bf16), v[2 * h + 1] + from_16(w[h] >> 16, p.bf16), p.bf16);
    *dst = make_uint4(r[0], r[1], r[2], r[3]);
  }
}

// Adds up the parts of a split wgrad tile: this CTA's share of its rows, four
// k per thread, over the parts that had stages.
__device__ __forceinline__ void join_dw(const GgParams& p, const Tile& t, uint32_t part_at, int part, int parts, int tid) {
  const int quads = (t.cols + 3) / 4, rows = min(128, p.M - t.m0);   // columns come in eights
  for (int i = part * kEpiThreads + tid; i < rows * quads; i += parts * kEpiThreads) {
    const int n = i / quads, c = 4 * (i - n * quads);
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int r = 0; r < parts; ++r) {
      if (t.nk * r / parts == t.nk * (r + 1) / parts) continue;
      const float4 v = peer_f32x4(part_at + (uint32_t)(n * kPartPitch + c) * 4, (uint32_t)r);
      s = make_float4(s.x + v.x, s.y + v.y, s.z + v.z, s.w + v.w);
    }
    const size_t at = ((size_t)t.e * p.M + t.m0 + n) * (size_t)p.ld_out + t.c0 + c;
    if (p.out_f32) {
      float4* dst = reinterpret_cast<float4*>(reinterpret_cast<float*>(p.out) + at);
      if (p.accumulate) {
        const float4 o = *dst;
        s = make_float4(s.x + o.x, s.y + o.y, s.z + o.z, s.w + o.w);
      }
      *dst = s;
    } else {
      uint2* dst = reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(p.out) + at);
      if (p.accumulate) {
        const uint2 o = *dst;
        s.x += from_16(o.x & 0xFFFFu, p.bf16);
        s.y += from_16(o.x >> 16, p.bf16);
        s.z += from_16(o.y & 0xFFFFu, p.bf16);
        s.w += from_16(o.y >> 16, p.bf16);
      }
      *dst = make_uint2(to_16x2(s.x, s.y, p.bf16), to_16x2(s.z, s.w, p.bf16));
    }
  }
}

// SUMS: kOneSum, 16-bit results go straight from TMEM to memory; kSums, the
// sums of a chunk of stages are added up in registers (fp32 results, additions
// to dw, split tiles); kLongSums, so are those of 16-bit results whose
// contraction takes more than one_sum stages.  A build of each: carrying two
// cost the first 2 to 4 %, additions to dw 3 to 4.
template <int CG, int MODE, int TN, int SUMS, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1)
gg_kernel(const __grid_constant__ CUtensorMap mapA, const __grid_constant__ CUtensorMap mapB,
          const __grid_constant__ CUtensorMap mapA1, const __grid_constant__ CUtensorMap mapB1,
          const __grid_constant__ CUtensorMap mapA16, const __grid_constant__ CUtensorMap mapB16,
          const __grid_constant__ CUtensorMap mapO, const GgParams p) {
  using C = Cfg<CG, MODE, TN>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = CG == 2 ? cluster_rank() : 0;
  static_assert(!SPLIT || (CG == 1 && SUMS == kSums), "split tiles");
  const int part = SPLIT ? (int)cluster_rank() : 0, parts = SPLIT ? (int)cluster_size() : 1;
  const uint32_t sbase = saddr(smem);
  int* tp = reinterpret_cast<int*>(smem + (MODE == kWgrad ? C::kOffTm + 4 : C::kOffTp));
  const uint32_t bar0 = sbase + C::kOffBar;
  auto full = [&](int s) { return bar0 + 8 * s; };
  auto empty = [&](int s) { return bar0 + 8 * (C::kStages + s); };
  auto acc_full = [&](int b) { return bar0 + 8 * (2 * C::kStages + b); };
  auto acc_empty = [&](int b) { return bar0 + 8 * (2 * C::kStages + 2 + b); };
  const uint32_t drain = bar0 + 8 * (2 * C::kStages + 4);
  uint32_t* tm_holder = reinterpret_cast<uint32_t*>(smem + C::kOffTm);

  int status = 0;   // an earlier launch gave up a wait: no work then; read once, so that all warps do the same
  if (tid == 0) {
    status = *reinterpret_cast<volatile int*>(p.err);
    prefetch_map(&mapA);
    prefetch_map(&mapB);
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(acc_full(b), 1);
      mbar_init(acc_empty(b), 8 * CG);
    }
    mbar_init(drain, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) tmem_alloc<CG>(saddr(tm_holder), C::kTmemCols);
  bool ascend = true;
  if (MODE == kWgrad) ascend = offsets_ascend(p.offsets, p.E, p.S, kThreads);
  else scan_tiles(p.offsets, p.E, p.S, TN, tp, tp + kMaxGroups + 1, kThreads);
  if (tid == 0) tm_holder[2] = (uint32_t)status;
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  if (MODE == kWgrad) tp[0] = __syncthreads_and(ascend);   // each thread writes it, the same: a register would be spilled
  else __syncthreads();
  if (CG == 2) cluster_sync();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = *tm_holder;

  int total = MODE == kWgrad ? p.E * p.n_mt * p.n_nt : tp[p.E] * p.n_mt;
  if (tm_holder[2] != 0) total = 0;
  const int first = blockIdx.x / (CG * parts), stride = gridDim.x / (CG * parts);
  // a split tile's CTAs take neighbouring ranges of its stages
  auto stage_from = [&](const Tile& t) { return SPLIT ? t.nk * part / parts : 0; };
  auto stage_to = [&](const Tile& t) { return SPLIT ? t.nk * (part + 1) / parts : t.nk; };
  auto chunk = [&](const Tile& t) {   // stages of one sum in TMEM
    return SUMS == kOneSum || (SUMS == kLongSums && t.nk <= p.one_sum) ? t.nk : kSumStages;
  };

  if (warp < kEpiWarp) {
    if (C::kSplitRegs && SUMS != kOneSum) asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    if (warp == 0) {
      // ---------------- copies ----------------
      const bool leader = elect_one();
      Ring<C::kStages> r;
      bool ok = true;
      for (int idx = first; idx < total && ok; idx += stride) {
        const Tile t = tile_of<CG, MODE, TN>(p, tp, idx);
        const int nact = (t.cols + 16 * CG - 1) / (16 * CG) * (16 * CG);   // the MMA's N
        const int half = nact / CG;                                       // this CTA's part of it
        const int ma = t.m0 + 128 * (int)rank, cb = t.c0 + half * (int)rank;
        const int nchunk = (half + 63) / 64;
        for (int kk = stage_from(t), to = stage_to(t); kk < to; ++kk, r.next()) {
          const int s = r.s;
          if (r.used == C::kStages && !warp_wait(empty(s), r.ph ^ 1, p.err, 71)) {
            ok = false;
            break;
          }
          if (leader) {
            const uint32_t a = sbase + s * kABytes, b = sbase + C::kOffB + s * C::kBBytes;
            const int k0 = kk * kBK;
            if (MODE != kWgrad) {
              const int nbox = (half + kBoxRows - 1) / kBoxRows;   // token rows in boxes of 32: a short tile reads few
              if (CG == 1 || rank == 0) mbar_expect_tx(full(s), CG * (kABytes + nbox * kBoxRows * 128));
              if (MODE == kFwd) {
                copy_3d<CG>(a, &mapA, k0, ma, t.e, full(s));
              } else {   // w as [n, k], k contiguous: two chunks of 64 k
                copy_3d<CG>(a, &mapA, ma, k0, t.e, full(s));
                copy_3d<CG>(a + kABytes / 2, &mapA, ma + 64, k0, t.e, full(s));
              }
              for (int i = 0; i < nbox; ++i)
                copy_2d<CG>(b + i * kBoxRows * 128, &mapB, k0, t.row0 + cb + i * kBoxRows, full(s));
            } else {
              const int rows = t.rows - k0;
              if (rows >= kBK) {
                if (CG == 1 || rank == 0) mbar_expect_tx(full(s), CG * (kABytes + nchunk * 8192));
                for (int c = 0; c < 2; ++c) copy_2d<CG>(a + 8192 * c, &mapA, ma + 64 * c, t.row0 + k0, full(s));
                for (int c = 0; c < nchunk; ++c) copy_2d<CG>(b + 8192 * c, &mapB, cb + 64 * c, t.row0 + k0, full(s));
              } else {
                // whole sixteens in boxes, the rest row by row below
                const int whole = rows & ~15;
                if (CG == 1 || rank == 0) mbar_expect_tx(full(s), CG * (2 + nchunk) * ((rows + 15) & ~15) * 128);
                for (int i = 0; i < whole; i += 16) {
                  for (int c = 0; c < 2; ++c) copy_2d<CG>(a + 8192 * c + i * 128, &mapA16, ma + 64 * c, t.row0 + k0 + i, full(s));
                  for (int c = 0; c < nchunk; ++c)
                    copy_2d<CG>(b + 8192 * c + i * 128, &mapB16, cb + 64 * c, t.row0 + k0 + i, full(s));
                }
              }
            }
          }
          __syncwarp();
          if (MODE == kWgrad && t.rows - kk * kBK < kBK && (t.rows & 15) != 0 && lane < 4 * (2 + nchunk)) {
            // the last, partial sixteen: a lane per chunk and four rows; rows past
            // the group's end are named S, out of bounds, and read as zeros
            const int c = lane >> 2, i = (t.rows & ~15) - kk * kBK + 4 * (lane & 3), r0 = kk * kBK + i;
            int row[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) row[j] = r0 + j < t.rows ? t.row0 + r0 + j : p.S;
            const bool is_a = c < 2;
            copy_rows4<CG>(sbase + (is_a ? s * kABytes + 8192 * c : C::kOffB + s * C::kBBytes + 8192 * (c - 2)) + i * 128,
                           is_a ? &mapA1 : &mapB1, is_a ? ma + 64 * c : cb + 64 * (c - 2), row[0], row[1], row[2], row[3],
                           full(s));
          }
          __syncwarp();
        }
      }
      leave(
          ok, [&] { return last_uses(r, [&](int j, uint32_t ph) { return warp_wait(empty(j), ph, p.err, 72); }); },
          [&] {
            if (rank == 0) last_uses(r, [&](int j, uint32_t ph) { return drain_wait(full(j), ph); });
            else pause_2ms();
          });
    } else if (warp == 1 && rank == 0) {
      // ---------------- MMAs ----------------
      const bool leader = elect_one();
      Ring<C::kStages> r;
      Ring<2> ab;
      bool ok = true;
      const uint32_t id0 = (1u << 4) | (p.bf16 ? (1u << 7) | (1u << 10) : 0u) | (MODE != kFwd ? 1u << 15 : 0u) |
                           (MODE == kWgrad ? 1u << 16 : 0u) | ((uint32_t)(128 * CG >> 4) << 24);
      for (int idx = first; idx < total && ok; idx += stride) {
        const Tile t = tile_of<CG, MODE, TN>(p, tp, idx);
        if (stage_from(t) == stage_to(t)) continue;
        const int nact = (t.cols + 16 * CG - 1) / (16 * CG) * (16 * CG);
        const uint32_t idesc = id0 | ((uint32_t)(nact >> 3) << 17);
        const int len = MODE == kWgrad ? t.rows : p.L;
        const int from = stage_from(t), to = stage_to(t);
        for (int k0 = from; k0 < to && ok;) {   // a chunk's sums start from zero in the other accumulator
          const int k1 = SUMS == kOneSum ? to : min(k0 + chunk(t), to), buf = ab.s;
          if (ab.used == 2 && !warp_wait(acc_empty(buf), ab.ph ^ 1, p.err, 73)) {
            ok = false;
            break;
          }
          ab.next();
          asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
          for (int kk = k0; kk < k1; ++kk, r.next()) {
            const int s = r.s;
            if (!warp_wait(full(s), r.ph, p.err, 74)) {
              ok = false;
              break;
            }
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            if (leader) {
              const uint32_t a = sbase + s * kABytes, b = sbase + C::kOffB + s * C::kBBytes;
              const uint64_t ad = MODE == kFwd ? sdesc(a) : sdesc_mn(a, 8192);
              const uint64_t bd = MODE != kWgrad ? sdesc(b) : sdesc_mn(b, 8192);
              const int steps = min(4, (len - kk * kBK + 15) >> 4);
              // per 16 contraction elements: 32 bytes along a K-major row, 16 rows of 128 bytes else
              for (int k = 0; k < steps; ++k)
                mma_f16<CG>(tmem + buf * TN, ad + (MODE == kFwd ? 2 : 128) * k, bd + (MODE != kWgrad ? 2 : 128) * k, idesc,
                            ((kk - k0) | k) != 0);
              commit<CG>(empty(s));
            }
            __syncwarp();
          }
          if (ok) {
            if (leader) commit<CG>(acc_full(buf));
            __syncwarp();
          }
          k0 = k1;
        }
      }
      leave(
          ok, [&] { return last_use(r, [&](int j, uint32_t ph) { return warp_wait(empty(j), ph, p.err, 76); }); },
          [&] {
            if (leader) commit<CG>(drain);
            __syncwarp();
            drain_wait(drain, 0);
          });
    }
  } else {
    // ---------------- epilogue ----------------
    if (C::kSplitRegs && SUMS != kOneSum) asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
    const int q = warp & 3, h = (warp - kEpiWarp) >> 2, ew = warp - kEpiWarp;
    Ring<2> ab;
    // this warp's 32 lanes and every other 32 columns (wgrad: 64)
    constexpr int kOwn = TN >= 64 ? TN / 64 : 1;
    auto own = [&](int i) { return MODE == kWgrad ? 128 * (i >> 1) + 64 * h + 32 * (i & 1) : 64 * i + 32 * h; };
    auto release = [&](int buf) {   // the accumulator may be written again
      asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
      if (CG == 1) mbar_arrive_if(acc_empty(buf), lane == 0);
      else mbar_arrive_at_if(acc_empty(buf), 0, lane == 0);
    };
    // 32 tokens x 32 elements as 8 x 8 fragments to 16-bit token rows, transposed
    // through shared memory: a store instruction is then 64 bytes of 8 rows (a
    // column a store, 2 bytes a lane, made the epilogue 2.5 times as long)
    auto store_16 = [&](const Tile& t, int m0, int c0, const uint32_t* v) {
      uint8_t* box = smem + C::kOffOut + ew * 32 * kOutPitch;
      const int chunk = lane & 3, n = m0 + 8 * chunk;
      auto two = [&](int c) { return to_16x2(__uint_as_float(v[c]), __uint_as_float(v[c + 1]), p.bf16); };
      __syncwarp();
#pragma unroll
      for (int g = 0; g < 4; ++g)
        store_transposed(saddr(box) + (8 * g + (lane & 7)) * kOutPitch + (lane >> 3) * 16, two(4 * g), two(4 * g + 2),
                         two(16 + 4 * g), two(16 + 4 * g + 2));
      __syncwarp();
      if (n >= p.M) return;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int tok = (lane >> 2) + 8 * j;
        if (c0 + tok < t.cols)
          *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(p.out) +
                                    (size_t)(t.row0 + t.c0 + c0 + tok) * (size_t)p.ld_out + n) =
              *reinterpret_cast<const uint4*>(box + tok * kOutPitch + chunk * 16);
      }
    };
    // 128 bytes x 32 rows of dw through shared memory (128-byte swizzle) and
    // TMA; the map ends at N and K
    auto store_box = [&](uint8_t* box, const Tile& t, int m0, int c0, const uint4* v) {
#pragma unroll
      for (int j = 0; j < 8; ++j) *reinterpret_cast<uint4*>(box + lane * 128 + ((j ^ (lane & 7)) << 4)) = v[j];
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) {
        asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
                         reinterpret_cast<uint64_t>(&mapO)),
                     "r"(t.c0 + c0), "r"(m0), "r"(t.e), "r"(saddr(box))
                     : "memory");
        asm volatile("cp.async.bulk.commit_group;" ::: "memory");
      }
    };
    uint32_t obuf = 0;
    for (int idx = first; idx < total && SUMS == kOneSum; idx += stride) {
      const Tile t = tile_of<CG, MODE, TN>(p, tp, idx);
      const int m0 = t.m0 + 128 * (int)rank + 32 * q;
      const bool sums = t.nk > 0;   // else an expert without rows: zeros
      int buf = 0;
      if (sums) {
        buf = ab.s;
        if (!warp_wait(acc_full(buf), ab.ph, p.err, 75)) break;
        ab.next();
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      }
      const uint32_t trow = tmem + buf * TN + ((uint32_t)(32 * q) << 16);
      if (MODE != kWgrad) {
#pragma unroll 1
        for (int c0 = 32 * h; c0 < t.cols; c0 += 64) {
          uint32_t d[32];
          __syncwarp();
          tmem_ld_frag_nowait(trow + c0, d);
          tmem_ld_frag_nowait(trow + (16u << 16) + c0, d + 16);
          tmem_ld_wait<32>(d);
          store_16(t, m0, c0, d);
        }
      } else if (m0 < p.M) {
        // by one warp per lane quarter with two boxes, or by two with one each
        auto store_dw = [&](auto eight) {
          constexpr bool kEight = decltype(eight)::value;
#pragma unroll 1
          for (int c0 = kEight ? 64 * h : 0; c0 < t.cols; c0 += kEight ? 128 : 64) {
            uint32_t d[64];
            if (sums) {
              tmem_ld32_nowait(trow + c0, d);
              tmem_ld32_nowait(trow + c0 + 32, d + 32);
              tmem_ld_wait<64>(d);
            } else {
#pragma unroll
              for (int i = 0; i < 64; ++i) d[i] = 0u;
            }
            uint4 v[8];
            auto two = [&](int c) { return to_16x2(__uint_as_float(d[c]), __uint_as_float(d[c + 1]), p.bf16); };
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = make_uint4(two(8 * j), two(8 * j + 2), two(8 * j + 4), two(8 * j + 6));
            if (lane == 0) {   // the box's last store has read it
              if (kEight) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
              else asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
            }
            __syncwarp();
            store_box(smem + C::kOffOut + (kEight ? ew : 2 * q + obuf) * 4096, t, m0, c0, v);
            obuf ^= 1;
          }
        };
        if (p.store8) store_dw(std::true_type{});
        else if (h == 0) store_dw(std::false_type{});
      }
      __syncwarp();
      if (sums) release(buf);
    }
    for (int idx = first; idx < total && SUMS != kOneSum; idx += stride) {
      const Tile t = tile_of<CG, MODE, TN>(p, tp, idx);
      float acc[kOwn][32];
#pragma unroll
      for (int i = 0; i < kOwn; ++i)
#pragma unroll
        for (int c = 0; c < 32; ++c) acc[i][c] = 0.f;
      bool ok = true;
      for (int kk = stage_from(t), to = stage_to(t); kk < to; kk += chunk(t)) {
        const int buf = ab.s;
        if (!warp_wait(acc_full(buf), ab.ph, p.err, 75)) {
          ok = false;
          break;
        }
        ab.next();
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        const uint32_t trow = tmem + buf * TN + ((uint32_t)(32 * q) << 16);
#pragma unroll
        for (int i = 0; i < kOwn; ++i) {
          if (own(i) >= t.cols) continue;
          uint32_t d[32];
          if (MODE == kWgrad) {   // a lane is a row of dw
            tmem_ld32_nowait(trow + own(i), d);
          } else {                // 8 x 8 fragments, to be stored transposed
            tmem_ld_frag_nowait(trow + own(i), d);
            tmem_ld_frag_nowait(trow + (16u << 16) + own(i), d + 16);
          }
          tmem_ld_wait<32>(d);
#pragma unroll
          for (int c = 0; c < 32; ++c) acc[i][c] += __uint_as_float(d[c]);
        }
        release(buf);
      }
      if (!ok) break;
      const int m0 = t.m0 + 128 * (int)rank + 32 * q;
      if (SPLIT) {   // this CTA's part, over the ring: its copies and MMAs are done
        float* part_at = reinterpret_cast<float*>(smem);
#pragma unroll
        for (int i = 0; i < kOwn; ++i) {
          if (own(i) >= t.cols) continue;
          if (MODE == kWgrad) {
#pragma unroll
            for (int c = 0; c < 32; c += 4)
              *reinterpret_cast<float4*>(part_at + (32 * q + lane) * kPartPitch + own(i) + c) =
                  make_float4(acc[i][c], acc[i][c + 1], acc[i][c + 2], acc[i][c + 3]);
          } else {
#pragma unroll
            for (int c = 0; c < 32; ++c) part_at[(own(i) + frag_col(c, lane)) * kJoinPitch + 32 * q + frag_row(c, lane)] = acc[i][c];
          }
        }
      } else if (MODE == kWgrad && SUMS == kSums && p.accumulate) {
        if (m0 + lane < p.M && t.nk > 0) {
#pragma unroll
          for (int i = 0; i < kOwn; ++i)
#pragma unroll
            for (int c = 0; c < 32; c += 8)   // columns come in eights
              if (own(i) + c < t.cols)
                add_dw(p, ((size_t)t.e * p.M + m0 + lane) * (size_t)p.ld_out + t.c0 + own(i) + c, acc[i] + c);
        }
      } else if (MODE == kWgrad) {
        uint8_t* box = smem + C::kOffOut + ew * 4096;
        auto box_free = [&] {   // the store before has read it
          if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
          __syncwarp();
        };
        auto two = [&](int i, int c) { return to_16x2(acc[i][c], acc[i][c + 1], p.bf16); };
#pragma unroll
        for (int i = 0; i < kOwn; ++i) {
          if (own(i) >= t.cols || m0 >= p.M) continue;
          uint4 v[8];
          if (SUMS == kSums) {   // fp32
#pragma unroll
            for (int j = 0; j < 8; ++j)
              v[j] = make_uint4(__float_as_uint(acc[i][4 * j]), __float_as_uint(acc[i][4 * j + 1]),
                                __float_as_uint(acc[i][4 * j + 2]), __float_as_uint(acc[i][4 * j + 3]));
          } else if (i % 2 == 0) {   // 64 columns a box: this one's 32 and the next's
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const int k = i + j / 4, c = 8 * (j % 4);
              v[j] = make_uint4(two(k, c), two(k, c + 2), two(k, c + 4), two(k, c + 6));
            }
          } else {
            continue;
          }
          box_free();
          store_box(box, t, m0, own(i), v);
        }
      } else if (SUMS == kLongSums) {
#pragma unroll
        for (int i = 0; i < kOwn; ++i)
          if (own(i) < t.cols) store_16(t, m0, own(i), reinterpret_cast<const uint32_t*>(acc[i]));
      } else {   // fp32: 16 tokens x 32 elements at a time, 128 bytes of 4 token rows a store
        uint8_t* box = smem + C::kOffOut + ew * 32 * kOutPitch;
        const int chunk = lane & 7, n = m0 + 4 * chunk;
#pragma unroll
        for (int i = 0; i < kOwn; ++i) {
          const int c0 = own(i);
          if (c0 >= t.cols) continue;
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            __syncwarp();
#pragma unroll
            for (int c = 0; c < 32; ++c)
              if (((c >> 3) & 1) == s)
                *reinterpret_cast<float*>(box + (frag_col(c, lane) - 16 * s) * kOutPitchF + 4 * frag_row(c, lane)) = acc[i][c];
            __syncwarp();
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int tok = (lane >> 3) + 4 * j;
              if (n < p.M && c0 + 16 * s + tok < t.cols)
                *reinterpret_cast<uint4*>(reinterpret_cast<float*>(p.out) +
                                          (size_t)(t.row0 + t.c0 + c0 + 16 * s + tok) * (size_t)p.ld_out + n) =
                    *reinterpret_cast<const uint4*>(box + tok * kOutPitchF + chunk * 16);
            }
          }
        }
      }
      __syncwarp();
    }
    if (MODE == kWgrad && lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    // rows of no group
    if (MODE != kWgrad && p.zero_rest && *reinterpret_cast<volatile int*>(p.err) == 0) {
      const long t = (long)blockIdx.x * kEpiThreads + tid - 32 * kEpiWarp, n = (long)gridDim.x * kEpiThreads;
      const int el = p.out_f32 ? 4 : 2;
      uint8_t* out = reinterpret_cast<uint8_t*>(p.out);
      const int* row = tp + kMaxGroups + 1;
      zero_rows(out, 0, row[0], (size_t)p.M * el, (size_t)p.ld_out * el, t, n);
      zero_rows(out, row[p.E], p.S, (size_t)p.M * el, (size_t)p.ld_out * el, t, n);
    }
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  if (CG == 2) cluster_sync();   // no CTA leaves while the other may still signal it
  if (SPLIT) {
    cluster_sync();              // every part is there
    // by the epilogue warps: the others may have handed registers back
    if (warp >= kEpiWarp && first < total && *reinterpret_cast<volatile int*>(p.err) == 0) {
      const Tile t = tile_of<CG, MODE, TN>(p, tp, first);
      if (MODE == kWgrad) join_dw(p, t, sbase, part, parts, tid - 32 * kEpiWarp);
      else join_parts(sbase, kJoinPitch, t.cols, tid - 32 * kEpiWarp, kEpiThreads, [&](int col, int m, float2 v) {
        if (t.m0 + m >= p.M) return;   // M is even
        const size_t at = (size_t)(t.row0 + t.c0 + col) * (size_t)p.ld_out + t.m0 + m;
        if (p.out_f32) *reinterpret_cast<float2*>(reinterpret_cast<float*>(p.out) + at) = v;
        else *reinterpret_cast<uint32_t*>(reinterpret_cast<uint16_t*>(p.out) + at) = to_16x2(v.x, v.y, p.bf16);
      });
    }
    cluster_sync();              // and read
  }
  if (warp == 1) {
    __syncwarp();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    tmem_free<CG>(tmem, C::kTmemCols);
  }
}

// operands; wgrad: their rows four by index and in sixteens, and the output
struct Maps {
  CUtensorMap a, b, a1, b1, a16, b16, out;
};

// split: CTAs per tile (SPLIT), with one tile per cluster
template <int CG, int MODE, int TN, int SUMS, bool SPLIT = false>
cudaError_t launch_t(const Maps& m, const GgParams& p, long max_items, cudaStream_t st, int split = 1) {
  static std::atomic<uint64_t> raised{0};
  const long sms = sm_count();
  if (sms <= 0) return cudaErrorInvalidDevice;
  if (Cfg<CG, MODE, TN>::kSplitRegs && SUMS != kOneSum) {   // the shares need the launch to hold their sum
    static const int regs = [] {
      cudaFuncAttributes fa;
      return cudaFuncGetAttributes(&fa, gg_kernel<CG, MODE, TN, SUMS, SPLIT>) == cudaSuccess ? fa.numRegs : 0;
    }();
    if (regs < kLaunchRegs) return cudaErrorInvalidConfiguration;
  }
  const int cluster = SPLIT ? split : CG;
  const long tiles = SPLIT || max_items < sms / CG ? max_items : sms / CG;
  return launch_cluster(gg_kernel<CG, MODE, TN, SUMS, SPLIT>, &raised, cluster, (int)(tiles < 1 ? 1 : tiles) * cluster, kThreads,
                        Cfg<CG, MODE, TN>::kSmem, st, m.a, m.b, m.a1, m.b1, m.a16, m.b16, m.out, p);
}

// forward and dgrad by their tiles
template <int MODE, int SUMS>
cudaError_t launch_rows(int tn, int cg, const Maps& m, const GgParams& p, long cap, cudaStream_t st) {
  return tn == 32    ? launch_t<1, MODE, 32, SUMS>(m, p, cap, st)
         : tn == 64  ? launch_t<1, MODE, 64, SUMS>(m, p, cap, st)
         : tn == 128 ? launch_t<1, MODE, 128, SUMS>(m, p, cap, st)
         : cg == 2   ? launch_t<2, MODE, 256, SUMS>(m, p, cap, st)
                     : launch_t<1, MODE, 256, SUMS>(m, p, cap, st);
}
template <int MODE>
cudaError_t launch_split(int tn, const Maps& m, const GgParams& p, long cap, cudaStream_t st, int split) {
  return tn == 32   ? launch_t<1, MODE, 32, kSums, true>(m, p, cap, st, split)
         : tn == 64 ? launch_t<1, MODE, 64, kSums, true>(m, p, cap, st, split)
                    : launch_t<1, MODE, 128, kSums, true>(m, p, cap, st, split);
}

bool fits16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

}  // namespace
}  // namespace situ

extern "C" situ_status situ_moe_grouped_gemm(const situ_grouped_gemm_args* g, void* stream) {
  using namespace situ;
  if (!g) return SITU_ERR_NULL_ARG;
  const int mode = g->direction;
  if (mode != kFwd && mode != kDgrad && mode != kWgrad) return SITU_ERR_UNSUPPORTED;
  if (g->dtype != SITU_DT_BF16 && g->dtype != SITU_DT_F16) return SITU_ERR_UNSUPPORTED;
  if (g->out_dtype != g->dtype && g->out_dtype != SITU_DT_F32) return SITU_ERR_UNSUPPORTED;
  if (g->accumulate != 0 && (g->accumulate != 1 || mode != kWgrad)) return SITU_ERR_UNSUPPORTED;
  if (g->keep_rest != 0 && (g->keep_rest != 1 || mode == kWgrad)) return SITU_ERR_UNSUPPORTED;
  if (g->S < 0 || g->N < 8 || g->K < 8 || g->N % 8 != 0 || g->K % 8 != 0 || g->E < 1 || g->E > kMaxGroups ||
      g->N > SITU_GEMM_MAX_DIM || g->K > SITU_GEMM_MAX_DIM || g->S > SITU_GEMM_MAX_ROWS)
    return SITU_ERR_BAD_SHAPE;
  const int64_t ca = mode == kFwd ? g->K : g->N;                         // columns of the first operand's rows
  const int64_t cb = mode == kFwd ? 0 : mode == kDgrad ? 0 : g->K;       // of the second's (wgrad: x)
  const int64_t co = mode == kFwd ? g->N : g->K;
  if (g->lda < ca || g->lda % 8 != 0 || (mode == kWgrad && (g->ldb < cb || g->ldb % 8 != 0)) ||
      (mode != kWgrad && (g->ldo < co || g->ldo % 8 != 0)))
    return SITU_ERR_BAD_SHAPE;
  const int64_t ldw = g->ldw ? g->ldw : g->K;
  if (g->lda > kMaxStride || (mode == kWgrad ? g->ldb : g->ldo) > kMaxStride || ldw > kMaxStride) return SITU_ERR_BAD_SHAPE;
  const int64_t stride_w = g->stride_w ? g->stride_w : g->N * ldw;
  if (mode == kWgrad ? g->ldw != 0 || g->stride_w != 0
                     : ldw < g->K || ldw % 8 != 0 || stride_w < g->N * ldw || stride_w % ldw != 0)
    return SITU_ERR_BAD_SHAPE;
  if (g->S == 0 && mode != kWgrad) return SITU_OK;
  if (!g->out || !g->offsets || !g->device_status || (g->S > 0 && (!g->a || !g->b)) || (mode != kWgrad && !g->b))
    return SITU_ERR_NULL_ARG;
  if (!fits16(g->a) || !fits16(g->b) || !fits16(g->out) || (reinterpret_cast<uintptr_t>(g->offsets) & 3) ||
      (reinterpret_cast<uintptr_t>(g->device_status) & 3))
    return SITU_ERR_MISALIGNED;
  cudaStream_t st = (cudaStream_t)stream;
  const size_t out_el = g->out_dtype == SITU_DT_F32 ? 4 : 2;
  if (mode == kWgrad && g->S == 0) {
    if (g->accumulate) return SITU_OK;
    return cudaMemsetAsync(g->out, 0, (size_t)g->E * g->N * g->K * out_el, st) == cudaSuccess ? SITU_OK : SITU_ERR_CUDA;
  }

  GgParams p = {};
  p.offsets = g->offsets;
  p.E = g->E;
  p.S = g->S;
  p.out = g->out;
  p.ld_out = mode == kWgrad ? g->K : g->ldo;
  p.bf16 = g->dtype == SITU_DT_BF16;
  p.out_f32 = g->out_dtype == SITU_DT_F32;
  p.accumulate = g->accumulate;
  p.zero_rest = !g->keep_rest;
  p.err = g->device_status;
  p.M = mode == kDgrad ? g->K : g->N;
  p.L = mode == kDgrad ? g->N : g->K;
  p.Ncol = g->K;

  // Tokens per tile: a group of few rows is bound by its weights' bytes, and a
  // narrow tile leaves the ring more stages; the widths leave most groups room
  // above the average (a second tile reads the weights again, from L2).  One
  // group's rows are known.  112 experts of 6144 x 3584 with 75 rows each: 64
  // tokens 0.91 ms, 128 0.77, 256 0.78; 32 of 4096 x 3584 with 128: 0.26, 0.18,
  // 0.16.  256 tokens go to CTA pairs (32 experts, 1,024 rows: 0.56 ms, single
  // CTAs 0.60), unless tiles of 128 fit the SMs once (512 rows, 4096 x 4096:
  // 23 us, pairs 25).
  const double per = (double)g->S / g->E;
  const double room[3] = {g->E == 1 ? 32. : 20., g->E == 1 ? 64. : 44., g->E == 1 ? 128. : 98.};
  const int tn = mode == kWgrad     ? 256
                 : per <= room[0] ? 32
                 : per <= room[1] ? 64
                 : per <= room[2] || most_tiles(g->S, g->E, 128) * ((p.M + 127) / 128) <= sm_count() ? 128 : 256;
  // wgrad's short contractions are bound by the stores, which eight warps issue
  // faster (896 experts, one row each, 768 x 3584: 0.79 ms, four warps 0.89;
  // 112 of 6144 x 3584, 75 rows: 0.93, 0.94; 32 of 4096 x 3584, 128 rows: 0.21,
  // 0.18).
  p.store8 = per <= 75;
  // wgrad of few output tiles: the rows of a group split over clusters (a
  // skewed group's rows are taken as up to twice the average)
  const double wtiles = (double)p.E * ((p.M + 127) / 128) * ((p.Ncol + 255) / 256);
  const int wsteps = (int)((g->E > 1 ? 2 * per : per) / kBK);
  const int wsplit = mode == kWgrad ? split_of(gg_kernel<1, kWgrad, 256, kSums, true>, kThreads,
                                               Cfg<1, kWgrad, 256>::kSmem, wtiles, wsteps, kSplitLeast)
                                    : 1;
  const int cg = tn == 256 && p.M > 128 && wsplit == 1 ? 2 : 1;
  p.n_mt = (p.M + 128 * cg - 1) / (128 * cg);
  p.n_nt = (p.Ncol + tn - 1) / tn;
  const double items = mode == kWgrad ? (double)p.E * p.n_mt * p.n_nt : ((double)g->S / tn + p.E) * p.n_mt;
  if (items > 2.0e9) return SITU_ERR_BAD_SHAPE;

  const CUtensorMapDataType dt = p.bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  Maps m = {};
  bool ok;
  const uint64_t S = (uint64_t)g->S, N = (uint64_t)g->N, K = (uint64_t)g->K, E = (uint64_t)g->E;
  if (mode == kWgrad) {
    const uint64_t da[2] = {N, S}, sa[1] = {(uint64_t)g->lda * 2}, db[2] = {K, S}, sb[1] = {(uint64_t)g->ldb * 2};
    const uint32_t box[2] = {64, 64}, box1[2] = {64, 1}, box16[2] = {64, 16};
    const uint64_t dout[3] = {K, N, E}, sout[2] = {K * out_el, N * K * out_el};
    const uint32_t boxo[3] = {(uint32_t)(128 / out_el), 32, 1};
    ok = make_map_nd(&m.a, dt, g->a, 2, da, sa, box) && make_map_nd(&m.b, dt, g->b, 2, db, sb, box) &&
         make_map_nd(&m.a1, dt, g->a, 2, da, sa, box1) && make_map_nd(&m.b1, dt, g->b, 2, db, sb, box1) &&
         make_map_nd(&m.a16, dt, g->a, 2, da, sa, box16) && make_map_nd(&m.b16, dt, g->b, 2, db, sb, box16) &&
         make_map_nd(&m.out, p.out_f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : dt, g->out, 3, dout, sout, boxo);
  } else {
    const uint64_t dw[3] = {K, N, E}, sw[2] = {(uint64_t)ldw * 2, (uint64_t)stride_w * 2};
    const uint32_t boxw[3] = {64, mode == kFwd ? 128u : 64u, 1};
    const uint64_t dx[2] = {(uint64_t)p.L, S}, sx[1] = {(uint64_t)g->lda * 2};
    const uint32_t boxx[2] = {64, (uint32_t)kBoxRows};
    ok = make_map_nd(&m.a, dt, g->b, 3, dw, sw, boxw) && make_map_nd(&m.b, dt, g->a, 2, dx, sx, boxx);
  }
  if (!ok) return SITU_ERR_CUDA;
  const double most = most_tiles(g->S, g->E, tn) * p.n_mt;
  const long cap = most > 1e6 ? 1000000 : (long)most;
  const int steps = (p.L + kBK - 1) / kBK;
  const int split = tn <= 128 ? split_of(gg_kernel<1, kFwd, 32, kSums, true>, kThreads, Cfg<1, kFwd, 32>::kSmem, most, steps, kSplitLeast) : 1;
  // The tensor cores truncate when they add: sums of one sign come out smaller
  // by 6e-9 of themselves per contraction element.  16-bit results take that
  // in one TMEM sum while it stays below a tenth of their last unit (largest
  // error 0.6 units where rounding alone is 0.5: f16 at 8,192, bf16 at 65,536
  // elements; f16 at 262,144: 3.7 units in one sum, 0.5 in chunks).  A group's
  // rows are not known here, but are S at most; its own tiles then count.
  p.one_sum = (p.bf16 ? 65536 : 8192) / kBK;
  const bool longer = ((mode == kWgrad ? p.S : p.L) + kBK - 1) / kBK > p.one_sum;
  const int sums = p.out_f32 || p.accumulate ? kSums : longer ? kLongSums : kOneSum;
  cudaError_t e;
  if (mode == kWgrad && wsplit > 1) {
    e = launch_t<1, kWgrad, 256, kSums, true>(m, p, (long)items, st, wsplit);
  } else if (split > 1) {
    e = mode == kFwd ? launch_split<kFwd>(tn, m, p, cap, st, split) : launch_split<kDgrad>(tn, m, p, cap, st, split);
  } else {
    const long all = items > 1e6 ? 1000000 : (long)items;
    auto launch = [&](auto form) {
      constexpr int F = decltype(form)::value;
      return mode == kFwd      ? launch_rows<kFwd, F>(tn, cg, m, p, cap, st)
             : mode == kDgrad  ? launch_rows<kDgrad, F>(tn, cg, m, p, cap, st)
             : cg == 2         ? launch_t<2, kWgrad, 256, F>(m, p, all, st)
                               : launch_t<1, kWgrad, 256, F>(m, p, all, st);
    };
    e = sums == kOneSum ? launch(std::integral_constant<int, kOneSum>{})
        : sums == kSums ? launch(std::integral_constant<int, kSums>{})
                        : launch(std::integral_constant<int, kLongSums>{});
  }
  return e == cudaSuccess ? SITU_OK : SITU_ERR_CUDA;
}
