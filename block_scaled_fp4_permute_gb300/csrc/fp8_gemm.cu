// fp8_gemm.cu -- products of E4M3 operands with one fp32 scale per block of
// 128, dense or over ragged expert groups, on tcgen05 (kind::f8f6f4).
//
//   y[r, n] = sum_b sx[r, b] * sw[e(r), n / 128, b] * sum_{k in block b} qx[r, k] * qw[e(r), n, k]
// The scales are arbitrary fp32 numbers, so they cannot ride along in the
// MMA (its block scales are powers of two): each block's 128-element product
// goes to its own TMEM accumulator, and the epilogue warps add it, times its
// scales, to fp32 sums that they keep in registers over the whole of K.  The
// two scales are multiplied first, in fp32, one factor for the block.
//
// Two kernels.  f8_kernel, for groups of few rows and launches of few tiles:
// weights on the MMA's M side (128 rows per CTA, one weight scale per block),
// 32 or 64 tokens on its N side, a token's scale being a column's factor.  It
// streams the weights (112 experts of 6144 x 3584, 128 rows: 0.26 ms,
// 6.5 TB/s).  Per CTA: warp 0 copies stages of one block (128 elements = one
// 128-byte swizzled row), warp 1 issues the four MMAs of a block, warps 4..11
// promote: each owns 32 lanes and half of the columns.  Warps 2 and 3 copy
// the scales, up to 16 blocks and the tile's end ahead.
// f8w_kernel, for the rest, is described below.
#include "../../include/situ_moe.h"
#include "gemm_groups.cuh"

#include <cuda_bf16.h>

namespace situ {

using namespace gg;

namespace {

constexpr int kABytes = 128 * 128;
constexpr int kThreads = 384;
constexpr int kEpiWarp = 4;
constexpr int kEpiThreads = 256;
constexpr int kSG = 4;   // blocks per slot of scales
constexpr int kOutPitch = 80, kOutPitchF = 144;   // bytes of a staged token row of 32 outputs, bf16 and fp32
constexpr int kBoxBytes = 16 * kOutPitchF;        // of a warp: 16 rows
constexpr int kSplitLeast = 2;   // blocks that a CTA of a split tile takes at least

struct F8Params {
  const int32_t* offsets;   // null: one dense group of S rows
  int E, S, N, K, nkb;
  int n_mt;
  const float* xs;          // [S, nkb]
  const float* ws;          // [E, ceil(N / 128), nkb]
  int nrb;
  void* out;
  long ld_out;
  int out_f32, zero_rest;
  int* err;
};

template <int TN>
struct Cfg {
  static constexpr int kBBytes = TN * 128;
  static constexpr int kStageBytes = kABytes + kBBytes;
  static constexpr int kBufs = 4;                              // TMEM accumulators
  static constexpr int kSlots = 4;                             // of scales: [block][token], then the weights'
  static constexpr int kSPitch = TN + 8;                       // conflict-free rows
  static constexpr int kSlotBytes = 4 * kSG * (kSPitch + 1);
  static constexpr int kOutBytes = 8 * kBoxBytes;              // output staging
  static constexpr int kMaxBytes = 232448 - 1024 - 4 * kScanInts - 512 - kSlots * kSlotBytes - kOutBytes;
  // 8 stages, 160 or 192 KB: all that fit at 32 tokens (10) made the HBM
  // slower (112 experts of 6144 x 3584: 0.267 ms, 8: 0.255, 6: 0.257)
  static constexpr int kStages = 8;
  static_assert(kStages * kStageBytes <= kMaxBytes, "shared memory");
  static constexpr int kOffB = kStages * kABytes;
  static constexpr int kOffS = kOffB + kStages * kBBytes;
  static constexpr int kOffOut = kOffS + kSlots * kSlotBytes;
  static constexpr int kOffTp = kOffOut + kOutBytes;
  static constexpr int kOffBar = (kOffTp + 4 * kScanInts + 15) / 16 * 16;
  static constexpr int kNumBars = 2 * kStages + kBufs + 1 + 2 * kSlots;
  static constexpr int kOffTm = kOffBar + 8 * kNumBars;
  static constexpr int kSmem = kOffTm + 16 + 1024;
  static constexpr int kTmemCols = kBufs * TN;
  static constexpr int kCh = TN / 2;                           // columns of a promoting warp: one TMEM load
  static_assert(kCh == 16 || kCh == 32, "TMEM loads");
  static_assert(kSmem <= 232448 && kTmemCols <= 512, "shared memory and TMEM");
};

struct Tile {
  int e, row0, mt, c0, cols;
};
template <int TN>
__device__ __forceinline__ Tile tile_of(const F8Params& p, const int* tp, int idx) {
  Tile t;
  t.e = find_group(tp, p.E, idx / p.n_mt);
  const int r = idx - tp[t.e] * p.n_mt, tt = tp[t.e + 1] - tp[t.e];
  t.mt = r / tt;
  t.c0 = (r - t.mt * tt) * TN;
  const int* row = tp + kMaxGroups + 1;
  t.row0 = row[t.e];
  t.cols = min(TN, row[t.e + 1] - t.row0 - t.c0);
  return t;
}

__device__ __forceinline__ void fma2(uint64_t& acc, uint64_t a, uint64_t b) {
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(acc) : "l"(a), "l"(b));
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ void copy_f32(uint32_t dst, const float* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ uint64_t pack2(uint32_t lo, uint32_t hi) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(lo), "r"(hi));
  return d;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& lo, float& hi) {
  uint32_t a, b;
  asm("mov.b64 {%0, %1}, %2;" : "=r"(a), "=r"(b) : "l"(v));
  lo = __uint_as_float(a);
  hi = __uint_as_float(b);
}

// zeros to the rows of no group (row: scan_tiles'); et: this thread's number
// among the CTA's per_cta promoting threads
__device__ __forceinline__ void zero_rest(const F8Params& p, const int* row, int et, int per_cta) {
  if (!p.offsets || !p.zero_rest || *reinterpret_cast<volatile int*>(p.err) != 0) return;
  const long t = (long)blockIdx.x * per_cta + et, n = (long)gridDim.x * per_cta;
  const int el = p.out_f32 ? 4 : 2;
  uint8_t* out = reinterpret_cast<uint8_t*>(p.out);
  zero_rows(out, 0, row[0], (size_t)p.N * el, (size_t)p.ld_out * el, t, n);
  zero_rows(out, row[p.E], p.S, (size_t)p.N * el, (size_t)p.ld_out * el, t, n);
}

template <int TN, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1)
f8_kernel(const __grid_constant__ CUtensorMap mapA, const __grid_constant__ CUtensorMap mapB, const F8Params p) {
  using C = Cfg<TN>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int part = SPLIT ? (int)cluster_rank() : 0, parts = SPLIT ? (int)cluster_size() : 1;
  // a split tile's CTAs take neighbouring ranges of its blocks
  const int kb0 = p.nkb * part / parts, kb1 = p.nkb * (part + 1) / parts;
  const uint32_t sbase = saddr(smem);
  int* tp = reinterpret_cast<int*>(smem + C::kOffTp);
  const uint32_t bar0 = sbase + C::kOffBar;
  auto full = [&](int s) { return bar0 + 8 * s; };
  auto done = [&](int s) { return bar0 + 8 * (C::kStages + s); };
  auto acc_empty = [&](int b) { return bar0 + 8 * (2 * C::kStages + b); };
  auto sc_full = [&](int i) { return bar0 + 8 * (2 * C::kStages + C::kBufs + i); };
  auto sc_empty = [&](int i) { return bar0 + 8 * (2 * C::kStages + C::kBufs + C::kSlots + i); };
  const uint32_t drain = bar0 + 8 * (2 * C::kStages + C::kBufs + 2 * C::kSlots);
  uint32_t* tm_holder = reinterpret_cast<uint32_t*>(smem + C::kOffTm);

  int status = 0;   // an earlier launch gave up a wait: no work then; read once, so that all warps do the same
  if (tid == 0) {
    status = *reinterpret_cast<volatile int*>(p.err);
    prefetch_map(&mapA);
    prefetch_map(&mapB);
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(full(s), 1);
      mbar_init(done(s), 1);
    }
    for (int b = 0; b < C::kBufs; ++b) mbar_init(acc_empty(b), 8);
    for (int i = 0; i < C::kSlots; ++i) {
      mbar_init(sc_full(i), 64);
      mbar_init(sc_empty(i), 8);
    }
    mbar_init(drain, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) tmem_alloc<1>(saddr(tm_holder), C::kTmemCols);
  scan_tiles(p.offsets, p.E, p.S, TN, tp, tp + kMaxGroups + 1, kThreads);
  if (tid == 0) tm_holder[2] = (uint32_t)status;
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = *tm_holder;

  int total = tp[p.E] * p.n_mt;
  if (tm_holder[2] != 0) total = 0;
  const int first = blockIdx.x / parts, stride = gridDim.x / parts;

  if (warp < kEpiWarp) {
    if (warp == 0) {
      // ---------------- copies ----------------
      const bool leader = elect_one();
      Ring<C::kStages> r;
      bool ok = true;
      for (int idx = first; idx < total && ok; idx += stride) {
        const Tile t = tile_of<TN>(p, tp, idx);
        const int m0 = t.mt * 128, row = t.row0 + t.c0;
        for (int kb = kb0; kb < kb1; ++kb, r.next()) {
          const int s = r.s;
          if (r.used == C::kStages && !warp_wait(done(s), r.ph ^ 1, p.err, 81)) {
            ok = false;
            break;
          }
          if (leader) {
            mbar_expect_tx(full(s), C::kStageBytes);
            copy_3d<1>(sbase + s * kABytes, &mapA, kb * 128, m0, t.e, full(s));
            copy_2d<1>(sbase + C::kOffB + s * C::kBBytes, &mapB, kb * 128, row, full(s));
          }
          __syncwarp();
        }
      }
      leave(
          ok, [&] { return last_uses(r, [&](int j, uint32_t ph) { return warp_wait(done(j), ph, p.err, 82); }); },
          [&] { last_uses(r, [&](int j, uint32_t ph) { return drain_wait(full(j), ph); }); });
    } else if (warp == 1) {
      // ---------------- MMAs ----------------
      const bool leader = elect_one();
      Ring<C::kStages> r;
      Ring<C::kBufs> ab;
      bool ok = true;
      const uint32_t id0 = (1u << 4) | ((uint32_t)(128 >> 4) << 24);   // E4M3 x E4M3 -> fp32, K-major
      for (int idx = first; idx < total && ok; idx += stride) {
        const Tile t = tile_of<TN>(p, tp, idx);
        const int nact = (t.cols + 15) / 16 * 16;
        const uint32_t idesc = id0 | ((uint32_t)(nact >> 3) << 17);
        for (int kb = kb0; kb < kb1; ++kb, r.next(), ab.next()) {
          const int s = r.s, buf = ab.s;
          // the first blocks find their accumulators empty: any completed phase will do
          if (!warp_wait2(acc_empty(buf), ab.ph ^ 1, full(s), r.ph, p.err, 83)) {
            ok = false;
            break;
          }
          asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
          if (leader) {
            const uint64_t ad = sdesc(sbase + s * kABytes), bd = sdesc(sbase + C::kOffB + s * C::kBBytes);
            // 32 bytes along the rows each; past K the stage holds zeros
#pragma unroll
            for (int k = 0; k < 4; ++k) mma_f8<1>(tmem + buf * TN, ad + 2 * k, bd + 2 * k, idesc, k != 0);
            commit<1>(done(s));   // the stage is free, its product there
          }
          __syncwarp();
        }
      }
      leave(
          ok, [&] { return last_use(r, [&](int j, uint32_t ph) { return warp_wait(done(j), ph, p.err, 88); }); },
          [&] {
            if (leader) commit<1>(drain);
            __syncwarp();
            drain_wait(drain, 0);
          });
    } else {
      // ---------------- scales ----------------
      Ring<C::kSlots> sr;
      bool ok = true;
      const int st = tid - 64, j = st & (kSG - 1);   // this thread's block of a slot
      for (int idx = first; idx < total && ok; idx += stride) {
        const Tile t = tile_of<TN>(p, tp, idx);
        const float* xs = p.xs + (size_t)(t.row0 + t.c0) * p.nkb;
        const float* ws = p.ws + ((size_t)t.e * p.nrb + t.mt) * p.nkb;
        for (int kb = kb0; kb < kb1; kb += kSG, sr.next()) {
          if (sr.used == C::kSlots && !warp_wait(sc_empty(sr.s), sr.ph ^ 1, p.err, 87)) {
            ok = false;
            break;
          }
          const uint32_t slot = sbase + C::kOffS + sr.s * C::kSlotBytes;
          const int b = min(kb + j, kb1 - 1);
#pragma unroll
          for (int i = 0; i < TN; i += 64 / kSG) {
            const int r = i + st / kSG;
            if (r < t.cols) copy_f32(slot + 4 * (j * C::kSPitch + r), xs + (size_t)r * p.nkb + b);
          }
          if (st < kSG) copy_f32(slot + 4 * (kSG * C::kSPitch + st), ws + b);
          asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(sc_full(sr.s)) : "memory");
        }
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
    }
  } else {
    // ---------------- promotion and store ----------------
    const int q = warp & 3, h = (warp - kEpiWarp) >> 2, et = tid - 32 * kEpiWarp;
    Ring<C::kStages> r;
    Ring<C::kBufs> ab;
    Ring<C::kSlots> sr;
    bool ok = true;
    for (int idx = first; idx < total && ok; idx += stride) {
      const Tile t = tile_of<TN>(p, tp, idx);
      uint64_t acc[C::kCh / 2];
#pragma unroll
      for (int c = 0; c < C::kCh / 2; ++c) acc[c] = 0ull;
      for (int k0 = kb0; k0 < kb1 && ok; k0 += kSG, sr.next()) {
        if (!warp_wait(sc_full(sr.s), sr.ph, p.err, 86)) {
          ok = false;
          break;
        }
        const float* slot = reinterpret_cast<const float*>(smem + C::kOffS + sr.s * C::kSlotBytes);
        const float4 fw = *reinterpret_cast<const float4*>(slot + kSG * C::kSPitch);
#pragma unroll
        for (int j = 0; j < kSG; ++j) {
          if (k0 + j >= kb1) break;
          const float w = j == 0 ? fw.x : j == 1 ? fw.y : j == 2 ? fw.z : fw.w;
          const uint64_t w2 = pack2(__float_as_uint(w), __float_as_uint(w));
          const float* fac = slot + j * C::kSPitch + h * C::kCh;
          if (!warp_wait(done(r.s), r.ph, p.err, 85)) {
            ok = false;
            break;
          }
          asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
          const uint32_t trow = tmem + ab.s * TN + ((uint32_t)(32 * q) << 16) + h * C::kCh;
          uint32_t d[C::kCh];
          if (C::kCh == 32) tmem_ld32_nowait(trow, d);
          else tmem_ld16_nowait(trow, d);
          uint64_t f[C::kCh / 2];
#pragma unroll
          for (int c = 0; c < C::kCh / 4; ++c) {
            const ulonglong2 x = *reinterpret_cast<const ulonglong2*>(fac + 4 * c);
            f[2 * c] = mul2(x.x, w2);
            f[2 * c + 1] = mul2(x.y, w2);
          }
          tmem_ld_wait<C::kCh>(d);
          // read: the accumulator may be written again
          asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
          mbar_arrive_if(acc_empty(ab.s), lane == 0);
#pragma unroll
          for (int c = 0; c < C::kCh / 2; ++c) fma2(acc[c], pack2(d[2 * c], d[2 * c + 1]), f[c]);
          ab.next();
          r.next();
        }
        __syncwarp();
        mbar_arrive_if(sc_empty(sr.s), lane == 0);
      }
      if (!ok) break;
      // column c is token c; a warp's lanes are 32 neighbouring outputs of it
      if (SPLIT) {   // this CTA's part, [token][128], over the ring: its copies and MMAs are done
        float* dst = reinterpret_cast<float*>(smem) + 32 * q + lane;
#pragma unroll
        for (int c = 0; c < C::kCh / 2; ++c) {
          float v[2];
          unpack2(acc[c], v[0], v[1]);
          dst[(h * C::kCh + 2 * c) * 128] = v[0];
          dst[(h * C::kCh + 2 * c + 1) * 128] = v[1];
        }
      } else {
        // through shared memory, 16 tokens at a time: 16-byte stores
        uint8_t* box = smem + C::kOffOut + (warp - kEpiWarp) * kBoxBytes;
        const int el = p.out_f32 ? 4 : 2, pitch = p.out_f32 ? kOutPitchF : kOutPitch;
        const int cpr = 2 * el, chunk = lane & (cpr - 1);   // 16-byte chunks of a row
        const int nn = t.mt * 128 + 32 * q + chunk * (16 / el);
#pragma unroll
        for (int c0 = 0; c0 < C::kCh; c0 += 16) {
          const int col = h * C::kCh + c0;
          if (col >= t.cols) continue;
          __syncwarp();
#pragma unroll
          for (int c = 0; c < 16; c += 2) {
            float v[2];
            unpack2(acc[(c0 + c) >> 1], v[0], v[1]);
            if (p.out_f32) {
              *reinterpret_cast<float*>(box + c * kOutPitchF + 4 * lane) = v[0];
              *reinterpret_cast<float*>(box + (c + 1) * kOutPitchF + 4 * lane) = v[1];
            } else {
              *reinterpret_cast<__nv_bfloat16*>(box + c * kOutPitch + 2 * lane) = __float2bfloat16_rn(v[0]);
              *reinterpret_cast<__nv_bfloat16*>(box + (c + 1) * kOutPitch + 2 * lane) = __float2bfloat16_rn(v[1]);
            }
          }
          __syncwarp();
          for (int tok = lane / cpr; tok < 16; tok += 32 / cpr)
            if (nn < p.N && col + tok < t.cols)
              *reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.out) +
                                        ((size_t)(t.row0 + t.c0 + col + tok) * (size_t)p.ld_out + nn) * el) =
                  *reinterpret_cast<const uint4*>(box + tok * pitch + chunk * 16);
        }
      }
      __syncwarp();
    }
    zero_rest(p, tp + kMaxGroups + 1, et, kEpiThreads);
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  if (SPLIT) {
    cluster_sync();              // every part is there
    if (warp >= kEpiWarp && first < total && *reinterpret_cast<volatile int*>(p.err) == 0) {
      const Tile t = tile_of<TN>(p, tp, first);
      join_parts(sbase, 128, t.cols, tid - 32 * kEpiWarp, kEpiThreads, [&](int col, int m, float2 v) {
        if (t.mt * 128 + m >= p.N) return;   // N is even
        const size_t at = (size_t)(t.row0 + t.c0 + col) * (size_t)p.ld_out + t.mt * 128 + m;
        if (p.out_f32) *reinterpret_cast<float2*>(reinterpret_cast<float*>(p.out) + at) = v;
        else *reinterpret_cast<uint32_t*>(reinterpret_cast<uint16_t*>(p.out) + at) = f32x2_to_bf16x2(v.x, v.y);
      });
    }
    cluster_sync();              // and read
  }
  if (warp == 1) {
    __syncwarp();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    tmem_free<1>(tmem, C::kTmemCols);
  }
}

// ---------------------------------------------------------------------------
// Wide tiles: tokens on the MMA's M side (128 per CTA), 256 weight rows on its
// N side.  A lane is a token, so a block's factor is one register and the
// additions need nothing from shared memory (with tokens along the columns the
// factors were a broadcast load per column, more shared-memory wavefronts than
// the MMA and the copies together: 8,192 x 6144 x 3584 0.33 ms, now 0.139).
//
// A tile is two halves of 128 weight rows, that is of one weight block each,
// with an MMA issuer and a promoting warpgroup per half and two accumulators
// each in TMEM: warp 0 copies, warps 1 and 2 issue, warp 3 copies scales ahead,
// warps 4..11 promote (32 lanes x 128 columns, 128 sums a thread).  That is
// more registers than an even split leaves: warps 0..3 hand back to 40 each,
// the promoting warps take 232 (40 * 128 + 232 * 256 = 168 * 384, the
// launch's own total).  No spills: a spilled value in these loops comes back
// through an L1 that the scales and results thrash, and cost 40 %.
//
// Bound by the promotion: 102 us of that case without its additions and
// stores, 28 more for the additions; stores by the promoting warps took 16,
// boxes that TMA takes away while the next tile is promoted take 7 (fp32
// results: 172 to 153 us).
// ---------------------------------------------------------------------------

constexpr int kWideN = 256;
constexpr int kWideParts = 2;                          // halves of a tile: an MMA and a promoting warpgroup each
constexpr int kWideThreads = 128 + 128 * kWideParts;

template <int CG, int BOXES>
struct WCfg {
  static constexpr int kTM = 128 * CG;                 // tokens per tile
  static constexpr int kTN = kWideN;                     // weight rows per tile
  static constexpr int kCols = kTN / kWideParts;       // of one half
  static constexpr int kBBytes = kTN / CG * 128;
  static constexpr int kStageBytes = kABytes + kBBytes;
  // scales: slots of four blocks, 128 tokens' and two weight blocks' factors
  static constexpr int kSlots = 4;
  static constexpr int kSlotBytes = (128 + 2) * 16;
  // output boxes of a promoting warp, 32 rows: a CTA of its own has no room
  // for more than one of 64 bytes beside four stages (three: 16,384 rows of 64
  // experts, 3584 x 2048: 152 us, four 145); a pair has five stages and a box
  // of 128 bytes, or four and two
  static constexpr int kRow = CG == 2 ? 128 : 64;
  static constexpr int kBoxBytes = 32 * kRow;
  static constexpr int kOutBytes = BOXES * kBoxBytes;
  static constexpr int kMaxBytes = 232448 - 1024 - 4 * kScanInts - 512 - kSlots * kSlotBytes - 4 * kWideParts * kOutBytes;
  static constexpr int kStages = kMaxBytes / kStageBytes;
  static constexpr int kOffB = kStages * kABytes;
  static constexpr int kOffOut = kOffB + kStages * kBBytes;
  static constexpr int kOffS = kOffOut + 4 * kWideParts * kOutBytes;
  static constexpr int kOffTp = kOffS + kSlots * kSlotBytes;
  static constexpr int kOffBar = (kOffTp + 4 * kScanInts + 15) / 16 * 16;
  // full, done[2] per stage; acc_empty[2][2]; drain[2]; scale slots full, empty
  static constexpr int kNumBars = 3 * kStages + 6 + 2 * kSlots;
  static constexpr int kOffTm = kOffBar + 8 * kNumBars;
  static constexpr int kSmem = kOffTm + 16 + 1024;
  static_assert(kSmem <= 232448, "shared memory");
};

constexpr int kLaunchRegs = 168;   // per thread of a launch, what the warps share out

struct WTile {
  int e, row0, rows, t0, n0, cols;
};
template <int CG>
__device__ __forceinline__ WTile wide_tile_of(const F8Params& p, const int* tp, int idx) {
  using C = WCfg<CG, 1>;
  WTile t;
  t.e = find_group(tp, p.E, idx / p.n_mt);
  const int r = idx - tp[t.e] * p.n_mt, tt = tp[t.e + 1] - tp[t.e], nt = r / tt;
  t.t0 = (r - nt * tt) * C::kTM;   // a group's token tiles run side by side: they read the same weights
  t.n0 = nt * C::kTN;
  const int* row = tp + kMaxGroups + 1;
  t.row0 = row[t.e];
  t.rows = row[t.e + 1] - t.row0;
  t.cols = min(C::kTN, p.N - t.n0);
  return t;
}

// src[i..i + 3] of n to 16 bytes of shared memory, zeros past the end; vec:
// src is 16-byte aligned and n a multiple of 4
__device__ __forceinline__ void copy_scales(uint32_t dst, const float* src, int i, int n, bool vec) {
  if (vec) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src + i) : "memory");
    return;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j)
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst + 4 * j), "l"(src + (i + j < n ? i + j : i)),
                 "r"(i + j < n ? 4 : 0)
                 : "memory");
}

__device__ __forceinline__ float4 lds_f32x4(uint32_t a) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a));
  return v;
}
// Where a box of 32 rows x ROW bytes in the ROW-byte swizzle holds the 16-byte
// chunk c of row r: neither a column of chunks nor whole rows conflict.
template <int ROW>
__device__ __forceinline__ int box_at(int r, int c) {
  return r * ROW + ((c ^ (ROW == 128 ? r & 7 : (r >> 1) & 3)) << 4);
}
// acc += d * f, kept in its place between the TMEM loads and the arrivals
__device__ __forceinline__ void fma_in_order(float& acc, uint32_t d, float f) {
  asm volatile("fma.rn.f32 %0, %1, %2, %0;" : "+f"(acc) : "f"(__uint_as_float(d)), "f"(f));
}

// the MMA's N of half h of a tile
template <int CG>
__device__ __forceinline__ int half_cols(const WTile& t, int h) {
  const int c = min(max(t.cols - 128 * h, 0), 128);
  return (c + 16 * CG - 1) / (16 * CG) * (16 * CG);
}

template <int CG, int BOXES>
__global__ void __launch_bounds__(kWideThreads, 1)
f8w_kernel(const __grid_constant__ CUtensorMap mapX, const __grid_constant__ CUtensorMap mapW,
           const __grid_constant__ CUtensorMap mapO, const F8Params p) {
  using C = WCfg<CG, BOXES>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = CG == 2 ? cluster_rank() : 0;
  const uint32_t sbase = saddr(smem);
  int* tp = reinterpret_cast<int*>(smem + C::kOffTp);
  const uint32_t bar0 = sbase + C::kOffBar;
  auto full = [&](int s) { return bar0 + 8 * s; };
  auto done = [&](int h, int s) { return bar0 + 8 * (C::kStages * (1 + h) + s); };
  auto acc_empty = [&](int h, int b) { return bar0 + 8 * (3 * C::kStages + 2 * h + b); };
  auto drain = [&](int h) { return bar0 + 8 * (3 * C::kStages + 4 + h); };
  auto sc_full = [&](int i) { return bar0 + 8 * (3 * C::kStages + 6 + i); };
  auto sc_empty = [&](int i) { return bar0 + 8 * (3 * C::kStages + 6 + C::kSlots + i); };
  uint32_t* tm_holder = reinterpret_cast<uint32_t*>(smem + C::kOffTm);

  int status = 0;   // an earlier launch gave up a wait: no work then; read once, so that all warps do the same
  if (tid == 0) {
    status = *reinterpret_cast<volatile int*>(p.err);
    prefetch_map(&mapX);
    prefetch_map(&mapW);
    prefetch_map(&mapO);
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(full(s), 1);
      mbar_init(done(0, s), 1);
      mbar_init(done(1, s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(acc_empty(0, b), 4 * CG);
      mbar_init(acc_empty(1, b), 4 * CG);
    }
    mbar_init(drain(0), 1);
    mbar_init(drain(1), 1);
    for (int i = 0; i < C::kSlots; ++i) {
      mbar_init(sc_full(i), 32);
      mbar_init(sc_empty(i), 4 * kWideParts);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) tmem_alloc<CG>(saddr(tm_holder), 512);
  scan_tiles(p.offsets, p.E, p.S, C::kTM, tp, tp + kMaxGroups + 1, kWideThreads);
  if (tid == 0) tm_holder[2] = (uint32_t)status;
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  if (CG == 2) cluster_sync();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = *tm_holder;

  int total = tp[p.E] * p.n_mt;
  if (tm_holder[2] != 0) total = 0;
  const int first = blockIdx.x / CG, stride = gridDim.x / CG;

  const bool xvec = (p.nkb & 3) == 0 && ((reinterpret_cast<uintptr_t>(p.xs) | reinterpret_cast<uintptr_t>(p.ws)) & 15) == 0;
  if (warp < kEpiWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
    if (warp == 0) {
      // ---------------- copies ----------------
      const bool leader = elect_one();
      Ring<C::kStages> r;
      bool ok = true;
      for (int idx = first; idx < total && ok; idx += stride) {
        const WTile t = wide_tile_of<CG>(p, tp, idx);
        int n[2];   // this CTA's first weight row of each half's product
#pragma unroll
        for (int h = 0; h < 2; ++h) n[h] = t.n0 + C::kCols * h + half_cols<CG>(t, h) / CG * (int)rank;
        const int row = t.row0 + t.t0 + 128 * (int)rank;
        for (int kb = 0; kb < p.nkb; ++kb, r.next()) {
          const int s = r.s;
          if (r.used == C::kStages && !warp_wait2(done(0, s), r.ph ^ 1, done(1, s), r.ph ^ 1, p.err, 91)) {
            ok = false;
            break;
          }
          if (leader) {
            if (CG == 1 || rank == 0) mbar_expect_tx(full(s), CG * C::kStageBytes);
            copy_2d<CG>(sbase + s * kABytes, &mapX, kb * 128, row, full(s));
#pragma unroll
            for (int h = 0; h < 2; ++h)
              copy_3d<CG>(sbase + C::kOffB + s * C::kBBytes + h * (C::kBBytes / 2), &mapW, kb * 128, n[h], t.e, full(s));
          }
          __syncwarp();
        }
      }
      leave(
          ok,
          [&] {
            return last_uses(r, [&](int j, uint32_t ph) {
              const bool first_half = warp_wait(done(0, j), ph, p.err, 92);
              return warp_wait(done(1, j), ph, p.err, 92) && first_half;
            });
          },
          [&] {
            if (rank == 0) last_uses(r, [&](int j, uint32_t ph) { return drain_wait(full(j), ph); });
            else pause_2ms();
          });
    } else if (warp <= 2) {
      // ---------------- MMAs ----------------
      // A warp per half: the waits and the commit of a product take an issuer
      // about as long as its MMAs run.
      if (rank == 0) {
        const int h = warp - 1;
        const bool leader = elect_one();
        Ring<C::kStages> r;
        Ring<2> ab;
        bool ok = true;
        for (int idx = first; idx < total && ok; idx += stride) {
          const WTile t = wide_tile_of<CG>(p, tp, idx);
          const int nact = half_cols<CG>(t, h);
          // E4M3 x E4M3 -> fp32, K-major
          const uint32_t idesc = (1u << 4) | ((uint32_t)(128 * CG >> 4) << 24) | ((uint32_t)(nact >> 3) << 17);
          for (int kb = 0; kb < p.nkb; ++kb, r.next(), ab.next()) {
            // the first two blocks find their accumulators empty: any completed phase will do
            if (!warp_wait2(acc_empty(h, ab.s), ab.ph ^ 1, full(r.s), r.ph, p.err, 93)) {
              ok = false;
              break;
            }
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            if (leader) {
              const uint64_t ad = sdesc(sbase + r.s * kABytes),
                             bd = sdesc(sbase + C::kOffB + r.s * C::kBBytes + h * (C::kBBytes / 2));
              if (nact > 0) {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                  mma_f8<CG>(tmem + ab.s * C::kTN + h * C::kCols, ad + 2 * k, bd + 2 * k, idesc, k != 0);
              }
              // this half is done with the stage, and its product is there
              commit<CG>(done(h, r.s));
            }
            __syncwarp();
          }
        }
        leave(
            ok, [&] { return last_use(r, [&](int j, uint32_t ph) { return warp_wait(done(h, j), ph, p.err, 98); }); },
            [&] {
              if (leader) commit<CG>(drain(h));
              __syncwarp();
              drain_wait(drain(h), 0);
            });
      }
    } else {
      // ---------------- scales ----------------
      // Copied ahead of the promotion, up to four slots (16 blocks): read
      // when they are needed, from an L2 busy with the tiles, they would
      // stall every block.
      const int st = tid - 96;
      Ring<C::kSlots> sr;
      bool ok = true;
      for (int idx = first; idx < total && ok; idx += stride) {
        const WTile t = wide_tile_of<CG>(p, tp, idx);
        const int row = t.t0 + 128 * (int)rank, wb = t.n0 >> 7;
        for (int kb = 0; kb < p.nkb; kb += 4, sr.next()) {
          if (sr.used == C::kSlots && !warp_wait(sc_empty(sr.s), sr.ph ^ 1, p.err, 96)) {
            ok = false;
            break;
          }
          const uint32_t slot = sbase + C::kOffS + sr.s * C::kSlotBytes;
          for (int i = st; i < 128 + 2; i += 32) {   // tokens, then weight blocks
            const bool tok = i < 128;
            const float* src = tok ? p.xs + (size_t)(t.row0 + min(row + i, t.rows - 1)) * p.nkb
                                   : p.ws + ((size_t)t.e * p.nrb + min(wb + i - 128, p.nrb - 1)) * p.nkb;
            copy_scales(slot + 16 * i, src, kb, p.nkb, xvec);
          }
          asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(sc_full(sr.s)) : "memory");
        }
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
    }
  } else {
    // ---------------- promotion and store ----------------
    asm volatile("setmaxnreg.inc.sync.aligned.u32 232;");
    const int q = warp & 3, h = (warp - kEpiWarp) >> 2, et = tid - 32 * kEpiWarp;
    Ring<C::kSlots> sr;
    Ring<2> ab;
    Ring<C::kStages> r;
    bool ok = true;
    const uint32_t tbase = tmem + C::kCols * h + ((uint32_t)(32 * q) << 16);
    for (int idx = first; idx < total && ok; idx += stride) {
      // a half's 128 columns lie in one block of weight rows
      float acc[C::kCols];
#pragma unroll
      for (int c = 0; c < C::kCols; ++c) acc[c] = 0.f;
      for (int k0 = 0; k0 < p.nkb && ok; k0 += 4) {
        if (!warp_wait(sc_full(sr.s), sr.ph, p.err, 97)) {
          ok = false;
          break;
        }
        const uint32_t slot = sbase + C::kOffS + sr.s * C::kSlotBytes;
        float f[4];
        {
          const float4 x = lds_f32x4(slot + 16 * (32 * q + lane)), w = lds_f32x4(slot + 16 * (128 + h));
          f[0] = x.x * w.x;
          f[1] = x.y * w.y;
          f[2] = x.z * w.z;
          f[3] = x.w * w.w;
        }
        __syncwarp();
        mbar_arrive_if(sc_empty(sr.s), lane == 0);
        sr.next();
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (k0 + j >= p.nkb) break;
          if (!warp_wait(done(h, r.s), r.ph, p.err, 95)) {
            ok = false;
            break;
          }
          asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
          // 64 columns at a time
          uint32_t d[64];
#pragma unroll
          for (int l = 0; l < C::kCols; l += 64) {
            tmem_ld32_nowait(tbase + ab.s * C::kTN + l, d);
            tmem_ld32_nowait(tbase + ab.s * C::kTN + l + 32, d + 32);
            tmem_ld_wait<64>(d);
            if (l + 64 == C::kCols) {   // read: the accumulator may be written again
              asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
              if (CG == 1) mbar_arrive_if(acc_empty(h, ab.s), lane == 0);
              else mbar_arrive_at_if(acc_empty(h, ab.s), 0, lane == 0);
            }
#pragma unroll
            for (int c = 0; c < 64; ++c) fma_in_order(acc[l + c], d[c], f[j]);
          }
          ab.next();
          r.next();
        }
      }
      if (!ok) break;
      const WTile t = wide_tile_of<CG>(p, tp, idx);
      // through shared memory, kRow bytes of the warp's 32 rows at a time: whole
      // boxes by TMA, which takes them away while the next tile is promoted,
      // and a group's last rows, next to another group's, by plain stores.
      // Boxes are used in turn and a tile takes a multiple of them; every use
      // commits one group, empty where TMA reads nothing, so that all but the
      // newest BOXES - 1 groups read means that the next box is free.
      static_assert(C::kCols * 2 / C::kRow % BOXES == 0, "a tile's boxes");
      const int row0 = t.t0 + 128 * (int)rank + 32 * q, n0 = t.n0 + C::kCols * h;
      if (row0 >= t.rows) continue;   // past the group's end: no rows, no boxes
      uint8_t* boxes = smem + C::kOffOut + (warp - kEpiWarp) * C::kOutBytes;
      auto store = [&](int i, int el, auto value) {
        uint8_t* box = boxes + C::kBoxBytes * (i % BOXES);
        const int n = n0 + i * (C::kRow / el);
        if (lane == 0) asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(BOXES - 1) : "memory");   // the box is free
        __syncwarp();
#pragma unroll
        for (int c = 0; c < C::kRow / 16; ++c) *reinterpret_cast<uint4*>(box + box_at<C::kRow>(lane, c)) = value(c);
        if (row0 + 32 <= t.rows) {
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          if (lane == 0) {
            if (n < p.N)
              asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                               reinterpret_cast<uint64_t>(&mapO)),
                           "r"(n), "r"(t.row0 + row0), "r"(saddr(box))
                           : "memory");
          }
        } else {
          constexpr int kCpr = C::kRow / 16;
          const int c = lane % kCpr, col = n + c * (16 / el);
          __syncwarp();
#pragma unroll
          for (int k = 0; k < kCpr; ++k) {
            const int r = lane / kCpr + 32 / kCpr * k;
            if (row0 + r < t.rows && col < p.N)
              *reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.out) +
                                        ((size_t)(t.row0 + row0 + r) * (size_t)p.ld_out + col) * el) =
                  *reinterpret_cast<const uint4*>(box + box_at<C::kRow>(r, c));
          }
        }
        if (lane == 0) asm volatile("cp.async.bulk.commit_group;" ::: "memory");
      };
      if (p.out_f32) {
#pragma unroll
        for (int i = 0; i < C::kCols * 4 / C::kRow; ++i) {
          const float* v = acc + C::kRow / 4 * i;
          store(i, 4, [&](int c) {
            return make_uint4(__float_as_uint(v[4 * c]), __float_as_uint(v[4 * c + 1]), __float_as_uint(v[4 * c + 2]),
                              __float_as_uint(v[4 * c + 3]));
          });
        }
      } else {
#pragma unroll
        for (int i = 0; i < C::kCols * 2 / C::kRow; ++i) {
          const float* v = acc + C::kRow / 2 * i;
          store(i, 2, [&](int c) {
            return make_uint4(f32x2_to_bf16x2(v[8 * c], v[8 * c + 1]), f32x2_to_bf16x2(v[8 * c + 2], v[8 * c + 3]),
                              f32x2_to_bf16x2(v[8 * c + 4], v[8 * c + 5]), f32x2_to_bf16x2(v[8 * c + 6], v[8 * c + 7]));
          });
        }
      }
    }
    if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    zero_rest(p, tp + kMaxGroups + 1, et, 128 * kWideParts);
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  if (CG == 2) cluster_sync();   // no CTA leaves while the other may still signal it
  if (warp == 1) {
    __syncwarp();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    tmem_free<CG>(tmem, 512);
  }
}

// split: CTAs per tile (SPLIT), with one tile per cluster
template <int TN, bool SPLIT>
cudaError_t launch_t(const CUtensorMap& a, const CUtensorMap& b, const F8Params& p, long max_items, cudaStream_t st,
                     int split = 1) {
  static std::atomic<uint64_t> raised{0};
  const long sms = sm_count();
  if (sms <= 0) return cudaErrorInvalidDevice;
  const long tiles = SPLIT || max_items < sms ? max_items : sms;
  return launch_cluster(f8_kernel<TN, SPLIT>, &raised, split, (int)(tiles < 1 ? 1 : tiles) * split, kThreads,
                        Cfg<TN>::kSmem, st, a, b, p);
}

template <int CG, int BOXES>
cudaError_t launch_wide(const CUtensorMap& x, const CUtensorMap& w, const CUtensorMap& o, const F8Params& p, long max_items,
                        cudaStream_t st) {
  static std::atomic<uint64_t> raised{0};
  // the register shares need the launch to hold their sum
  static const int regs = [] {
    cudaFuncAttributes fa;
    return cudaFuncGetAttributes(&fa, f8w_kernel<CG, BOXES>) == cudaSuccess ? fa.numRegs : 0;
  }();
  const long sms = sm_count();
  if (sms <= 0 || regs < kLaunchRegs) return cudaErrorInvalidConfiguration;
  const long ctas = max_items < sms / CG ? max_items * CG : sms / CG * CG;
  return launch_cluster(f8w_kernel<CG, BOXES>, &raised, CG, (int)(ctas < CG ? CG : ctas), kWideThreads,
                        WCfg<CG, BOXES>::kSmem, st, x, w, o, p);
}

}  // namespace
}  // namespace situ

extern "C" situ_status situ_moe_fp8_gemm(const situ_fp8_gemm_args* g, void* stream) {
  using namespace situ;
  if (!g) return SITU_ERR_NULL_ARG;
  if (g->out_dtype != SITU_DT_BF16 && g->out_dtype != SITU_DT_F32) return SITU_ERR_UNSUPPORTED;
  if (g->keep_rest != 0 && g->keep_rest != 1) return SITU_ERR_UNSUPPORTED;
  if (g->S < 0 || g->N < 8 || g->N % 8 != 0 || g->K < 16 || g->K % 16 != 0 || g->E < 1 || g->E > kMaxGroups ||
      g->N > SITU_GEMM_MAX_DIM || g->K > SITU_GEMM_MAX_DIM || g->S > SITU_GEMM_MAX_ROWS || (!g->offsets && g->E != 1) ||
      g->ldx < g->K || g->ldx % 16 != 0 || g->ldo < g->N || g->ldo % 8 != 0)
    return SITU_ERR_BAD_SHAPE;
  const int64_t ldw = g->ldw ? g->ldw : g->K;
  if (g->ldx > kMaxStride || g->ldo > kMaxStride || ldw > kMaxStride) return SITU_ERR_BAD_SHAPE;
  const int64_t stride_w = g->stride_w ? g->stride_w : g->N * ldw;
  if (ldw < g->K || ldw % 16 != 0 || stride_w < g->N * ldw || stride_w % ldw != 0) return SITU_ERR_BAD_SHAPE;
  if (g->S == 0) return SITU_OK;
  if (!g->x_q || !g->x_scale || !g->w_q || !g->w_scale || !g->out || !g->device_status) return SITU_ERR_NULL_ARG;
  for (const void* q : {(const void*)g->x_q, (const void*)g->w_q, (const void*)g->out})
    if (reinterpret_cast<uintptr_t>(q) & 15) return SITU_ERR_MISALIGNED;
  for (const void* q : {(const void*)g->x_scale, (const void*)g->w_scale, (const void*)g->offsets, (const void*)g->device_status})
    if (reinterpret_cast<uintptr_t>(q) & 3) return SITU_ERR_MISALIGNED;

  F8Params p = {};
  p.offsets = g->offsets;
  p.E = g->E;
  p.S = g->S;
  p.N = g->N;
  p.K = g->K;
  p.nkb = (g->K + 127) / 128;
  p.xs = g->x_scale;
  p.ws = g->w_scale;
  p.nrb = (g->N + 127) / 128;
  p.out = g->out;
  p.ld_out = g->ldo;
  p.out_f32 = g->out_dtype == SITU_DT_F32;
  p.zero_rest = !g->keep_rest;
  p.err = g->device_status;

  // Tiles: up to about 20 rows per group (one group's rows are known) 32
  // tokens on the MMA's N side, up to about 50 of them 64, which stream the
  // weights and little else; above, wide tiles (40 experts of 4096 x 2048 with
  // 10 / 25 / 45 / 64 / 80 rows each: 32 tokens 57 / 59 / 80 / 98 / 116 us, 64
  // tokens 57 / 58 / 60 / 72 / 92, wide 62 / 66 / 65 / 65 / 67; one of 24,576 x
  // 4096, 64 and 100 rows: 64 tokens 27, 32 us, wide 31, 27).  But 64 tokens
  // while such tiles fit the SMs once (256 rows, 4096 x 4096: 13.5 us, wide
  // 19), with the contraction split.
  const double per = (double)g->S / g->E;
  const bool one = g->E == 1;
  const int tn = per <= (one ? 32. : 20.) ? 32
                 : per <= (one ? 64. : 50.) || most_tiles(g->S, g->E, 64) * ((p.N + 127) / 128) <= sm_count() ? 64
                                                                                                             : 256;
  // Wide tiles of one CTA (128 tokens) waste less of a group's last tile, a
  // pair copies the weights half as often: 64 experts of 3584 x 2048, 256 rows:
  // 143 us, pairs 159; 32, 512 rows: 128, 130; 16, 1,024: 119, 119; 8, 2,048:
  // 117, 109.  Rows that do not start on 128-byte lines cost about twice the L2
  // requests: 64 experts of 3584 x 2000, 100 / 128 rows: 93 / 121 us, pairs 118 /
  // 119; 100 of 2048 x 2064, 164 rows: 135, 117.
  const bool lines = ldw % 128 == 0 && g->ldx % 128 == 0;
  const int cg = tn < 256 || per < (lines ? 1024. : 150.) ? 1 : 2;
  // A pair's second output box costs it its fifth stage: 8,192 rows, 6144 x
  // 3584: 146 us, two boxes 143; rows off the lines need the stage (16,384 rows,
  // 4096 x 2000, fp32: 148 us, two boxes 163).
  const bool two = lines;
  const int tm = tn < 256 ? tn : 128 * cg;        // tokens per tile
  p.n_mt = tn < 256 ? (p.N + 127) / 128 : (p.N + kWideN - 1) / kWideN;
  if (most_tiles(g->S, g->E, tm) * p.n_mt > 2.0e9) return SITU_ERR_BAD_SHAPE;
  CUtensorMap mw, mx, mo = {};
  const uint64_t S = (uint64_t)g->S, N = (uint64_t)g->N, K = (uint64_t)g->K, E = (uint64_t)g->E;
  const uint64_t dw[3] = {K, N, E}, sw[2] = {(uint64_t)ldw, (uint64_t)stride_w}, dx[2] = {K, S}, sx[1] = {(uint64_t)g->ldx};
  const uint32_t boxw[3] = {128, tn < 256 ? 128u : (uint32_t)(kWideN / 2 / cg), 1}, boxx[2] = {128, tn < 256 ? (uint32_t)tn : 128u};
  if (!make_map_nd(&mw, CU_TENSOR_MAP_DATA_TYPE_UINT8, g->w_q, 3, dw, sw, boxw) ||
      !make_map_nd(&mx, CU_TENSOR_MAP_DATA_TYPE_UINT8, g->x_q, 2, dx, sx, boxx))
    return SITU_ERR_CUDA;
  if (tn == 256) {
    const uint64_t el = p.out_f32 ? 4 : 2, dout[2] = {N, S}, so[1] = {(uint64_t)g->ldo * el};
    const int row = cg == 1 ? WCfg<1, 1>::kRow : WCfg<2, 1>::kRow;
    const uint32_t boxo[2] = {(uint32_t)(row / el), 32};
    if (!make_map_nd(&mo, p.out_f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, g->out, 2, dout, so,
                     boxo, row == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B))
      return SITU_ERR_CUDA;
  }
  cudaStream_t st = (cudaStream_t)stream;
  const double most = most_tiles(g->S, g->E, tm) * p.n_mt;
  const long cap = most > 1e6 ? 1000000 : (long)most;
  const int split = tn < 256 ? split_of(f8_kernel<32, true>, kThreads, Cfg<32>::kSmem, most, p.nkb, kSplitLeast) : 1;
  cudaError_t e;
  if (split > 1)
    e = tn == 32 ? launch_t<32, true>(mw, mx, p, cap, st, split) : launch_t<64, true>(mw, mx, p, cap, st, split);
  else
    e = tn == 32   ? launch_t<32, false>(mw, mx, p, cap, st)
        : tn == 64 ? launch_t<64, false>(mw, mx, p, cap, st)
        : cg == 1  ? launch_wide<1, 1>(mx, mw, mo, p, cap, st)
        : two      ? launch_wide<2, 2>(mx, mw, mo, p, cap, st)
                   : launch_wide<2, 1>(mx, mw, mo, p, cap, st);
  return e == cudaSuccess ? SITU_OK : SITU_ERR_CUDA;
}
