// fp8_gemm.cu -- products of E4M3 operands with one fp32 scale per block of
// 128, dense or over ragged expert groups, on tcgen05 (kind::f8f6f4).
//
//   y[r, n] = sum_b sx[r, b] * sw[e(r), n / 128, b] * sum_{k in block b} qx[r, k] * qw[e(r), n, k]
// The scales are arbitrary fp32 numbers, so they cannot ride along in the
// MMA (its block scales are powers of two): each block's 128-element product
// goes to its own TMEM accumulator, and the epilogue warps add it, times its
// scales, to fp32 sums that they keep in registers over the whole of K.
//
// 256 tokens per tile are 128 sums per promoting thread, more than an even
// split of the registers over twelve warps leaves room for: warps 0..3 hand
// back to 56 each and the promoting warps take 224 (56 * 128 + 224 * 256 =
// 168 * 384, the launch's own total).
//
// Weights on the MMA's M side (128 rows per CTA: one weight scale per block
// and CTA), tokens on its N side: a token's scale is a column's factor.  Per
// CTA: warp 0 copies stages of one block (128 elements = one 128-byte
// swizzled row), warp 1 issues the four MMAs of a block, warps 4..11 promote:
// each owns 32 lanes and half of the columns.  The factors sx * sw of four
// blocks at a time are staged in shared memory, one group ahead.
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
constexpr int kSG = 4;   // blocks per group of staged factors

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

template <int CG, int TN>
struct Cfg {
  static constexpr int kTNB = TN / CG;
  static constexpr int kBBytes = kTNB * 128;
  static constexpr int kStageBytes = kABytes + kBBytes;
  static constexpr int kBufs = TN >= 256 ? 2 : 4;              // TMEM accumulators
  static constexpr int kSPitch = TN + 8;                       // staged factors, conflict-free rows
  static constexpr int kSBytes = 2 * kSG * kSPitch * 4;
  static constexpr int kMaxBytes = 232448 - 1024 - 4 * (kMaxGroups + 1) - 512 - kSBytes;
  static constexpr int kStages = kMaxBytes / kStageBytes;
  static constexpr int kOffB = kStages * kABytes;
  static constexpr int kOffS = kOffB + kStages * kBBytes;
  static constexpr int kOffTp = kOffS + kSBytes;
  static constexpr int kOffBar = (kOffTp + 4 * (kMaxGroups + 1) + 15) / 16 * 16;
  static constexpr int kNumBars = 2 * kStages + 2 * kBufs + 1;
  static constexpr int kOffTm = kOffBar + 8 * kNumBars;
  static constexpr int kSmem = kOffTm + 16 + 1024;
  static constexpr int kTmemCols = kBufs * TN;
  static constexpr int kCh = TN >= 64 ? 32 : 16;               // columns per TMEM load
  static constexpr int kNch = TN / (2 * kCh);                  // loads per promoting warp and block
  static constexpr bool kSplitRegs = TN >= 256;
  static_assert(kSmem <= 232448 && kTmemCols <= 512, "shared memory and TMEM");
};
constexpr int kLaunchRegs = 168;   // per thread, what kSplitRegs shares out

struct Tile {
  int e, row0, mt, c0, cols;
};
template <int CG, int TN>
__device__ __forceinline__ Tile tile_of(const F8Params& p, const int* tp, int idx) {
  Tile t;
  t.e = find_group(tp, p.E, idx / p.n_mt);
  const int r = idx - tp[t.e] * p.n_mt, tt = tp[t.e + 1] - tp[t.e];
  t.mt = r / tt;
  t.c0 = (r - t.mt * tt) * TN;
  const int2 g = group_rows(p.offsets, t.e, p.S);
  t.row0 = g.x;
  t.cols = min(TN, g.y - t.c0);
  return t;
}

__device__ __forceinline__ void fma2(uint64_t& acc, uint64_t a, uint64_t b) {
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(acc) : "l"(a), "l"(b));
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

template <int CG, int TN>
__global__ void __launch_bounds__(kThreads, 1)
f8_kernel(const __grid_constant__ CUtensorMap mapA, const __grid_constant__ CUtensorMap mapB, const F8Params p) {
  using C = Cfg<CG, TN>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = CG == 2 ? cluster_rank() : 0;
  const uint32_t sbase = saddr(smem);
  int* tp = reinterpret_cast<int*>(smem + C::kOffTp);
  const uint32_t bar0 = sbase + C::kOffBar;
  auto full = [&](int s) { return bar0 + 8 * s; };
  auto empty = [&](int s) { return bar0 + 8 * (C::kStages + s); };
  auto acc_full = [&](int b) { return bar0 + 8 * (2 * C::kStages + b); };
  auto acc_empty = [&](int b) { return bar0 + 8 * (2 * C::kStages + C::kBufs + b); };
  const uint32_t drain = bar0 + 8 * (2 * C::kStages + 2 * C::kBufs);
  uint32_t* tm_holder = reinterpret_cast<uint32_t*>(smem + C::kOffTm);

  if (tid == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    for (int b = 0; b < C::kBufs; ++b) {
      mbar_init(acc_full(b), 1);
      mbar_init(acc_empty(b), 8 * CG);
    }
    mbar_init(drain, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) tmem_alloc<CG>(saddr(tm_holder), C::kTmemCols);
  scan_tiles(p.offsets, p.E, p.S, TN, tp, kThreads);
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  if (CG == 2) cluster_sync();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = *tm_holder;

  // an earlier launch that gave up a wait leaves its code in *err: no work then
  int total = tp[p.E] * p.n_mt;
  if (*reinterpret_cast<volatile int*>(p.err) != 0) total = 0;
  const int first = blockIdx.x / CG, stride = gridDim.x / CG;

  if (warp < kEpiWarp) {
    if (C::kSplitRegs) asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    if (warp == 0) {
      // ---------------- copies ----------------
      const bool leader = elect_one();
      Ring<C::kStages> r;
      bool ok = true;
      for (int idx = first; idx < total && ok; idx += stride) {
        const Tile t = tile_of<CG, TN>(p, tp, idx);
        const int half = (t.cols + 16 * CG - 1) / (16 * CG) * 16;
        const int m0 = (t.mt * CG + (int)rank) * 128, row = t.row0 + t.c0 + half * (int)rank;
        for (int kb = 0; kb < p.nkb; ++kb, r.next()) {
          const int s = r.s;
          if (r.used == C::kStages && !mbar_wait_warp(empty(s), r.ph ^ 1, p.err, 81)) {
            ok = false;
            break;
          }
          if (leader) {
            if (CG == 1 || rank == 0) mbar_expect_tx(full(s), CG * C::kStageBytes);
            copy_3d<CG>(sbase + s * kABytes, &mapA, kb * 128, m0, t.e, full(s));
            copy_2d<CG>(sbase + C::kOffB + s * C::kBBytes, &mapB, kb * 128, row, full(s));
          }
          __syncwarp();
        }
      }
      if (ok) {   // the last arrivals on this CTA's barriers, before it may leave
        for (int j = 0; j < r.used; ++j) mbar_wait_warp(empty(j), j < r.s ? r.ph : r.ph ^ 1, p.err, 82);
      } else if (rank == 0) {   // copies in flight
        for (int j = 0; j < r.used; ++j) drain_wait(full(j), j < r.s ? r.ph : r.ph ^ 1);
      } else {
        const unsigned long long t0 = globaltimer();   // they complete on the other CTA's barriers
        while (globaltimer() - t0 < 2000000ull) {
        }
      }
    } else if (warp == 1 && rank == 0) {
      // ---------------- MMAs ----------------
      const bool leader = elect_one();
      Ring<C::kStages> r;
      Ring<C::kBufs> ab;
      bool ok = true;
      const uint32_t id0 = (1u << 4) | ((uint32_t)(128 * CG >> 4) << 24);   // E4M3 x E4M3 -> fp32, K-major
      for (int idx = first; idx < total && ok; idx += stride) {
        const Tile t = tile_of<CG, TN>(p, tp, idx);
        const int nact = (t.cols + 16 * CG - 1) / (16 * CG) * (16 * CG);
        const uint32_t idesc = id0 | ((uint32_t)(nact >> 3) << 17);
        for (int kb = 0; kb < p.nkb; ++kb, r.next(), ab.next()) {
          const int s = r.s, buf = ab.s;
          if ((ab.used == C::kBufs && !mbar_wait_warp(acc_empty(buf), ab.ph ^ 1, p.err, 83)) ||
              !mbar_wait_warp(full(s), r.ph, p.err, 84)) {
            ok = false;
            break;
          }
          asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
          if (leader) {
            const uint64_t ad = sdesc(sbase + s * kABytes), bd = sdesc(sbase + C::kOffB + s * C::kBBytes);
            // 32 bytes along the rows each; past K the stage holds zeros
#pragma unroll
            for (int k = 0; k < 4; ++k) mma_f8<CG>(tmem + buf * TN, ad + 2 * k, bd + 2 * k, idesc, k != 0);
            commit<CG>(empty(s));
            commit<CG>(acc_full(buf));
          }
          __syncwarp();
        }
      }
      if (!ok) {   // MMAs in flight
        if (leader) commit<CG>(drain);
        __syncwarp();
        drain_wait(drain, 0);
      }
    }
  } else {
    // ---------------- promotion and store ----------------
    if (C::kSplitRegs) asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
    const int q = warp & 3, h = (warp - kEpiWarp) >> 2, et = tid - 32 * kEpiWarp;
    float* stage = reinterpret_cast<float*>(smem + C::kOffS);
    constexpr int kPer = kSG * TN / kEpiThreads > 0 ? kSG * TN / kEpiThreads : 1;   // factors per thread and group
    const int j = et & (kSG - 1);   // this thread's block within a group
    Ring<C::kBufs> ab;
    bool ok = true, left = false;
    for (int idx = first; idx < total; idx += stride) {
      const Tile t = tile_of<CG, TN>(p, tp, idx);
      const int mtile = t.mt * CG + (int)rank;   // past N's last block in a pair's second CTA: no factors, no rows
      const float* xs = p.xs + (size_t)(t.row0 + t.c0) * p.nkb;
      const float* ws = p.ws + ((size_t)t.e * p.nrb + min(mtile, p.nrb - 1)) * p.nkb;
      float f[kPer], fw;
      auto fetch = [&](int g) {   // the factors of blocks [kSG * g, ...)
        const int kb = kSG * g + j;
        fw = kb < p.nkb ? __ldg(ws + kb) : 0.f;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          const int r = (et >> 2) + i * (kEpiThreads / kSG);
          f[i] = (kb < p.nkb && r < t.cols) ? __ldg(xs + (size_t)r * p.nkb + kb) : 0.f;
        }
      };
      auto put = [&](int g) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          const int r = (et >> 2) + i * (kEpiThreads / kSG);
          if (r < TN) stage[((g & 1) * kSG + j) * C::kSPitch + r] = f[i] * fw;
        }
      };
      uint64_t acc[C::kNch][C::kCh / 2];
#pragma unroll
      for (int i = 0; i < C::kNch; ++i)
#pragma unroll
        for (int c = 0; c < C::kCh / 2; ++c) acc[i][c] = 0ull;
      fetch(0);
      // every warp is done with the last tile's factors; a warp whose wait ran
      // out still takes part in the barriers, and all of them leave at one
      if (!bar_and(1, kEpiThreads, ok)) break;
      put(0);
      bar_and(1, kEpiThreads, true);
      for (int kb = 0; kb < p.nkb; ++kb, ab.next()) {
        const int g = kb / kSG;
        if (kb % kSG == 0 && kb + kSG < p.nkb) fetch(g + 1);
        const int buf = ab.s;
        ok = ok && mbar_wait_warp(acc_full(buf), ab.ph, p.err, 85);
        if (!ok) {
          if (kb % kSG == kSG - 1 && kb + 1 < p.nkb) {
            bar_and(1, kEpiThreads, false);
            left = true;
            break;
          }
          continue;
        }
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        const uint32_t trow = tmem + buf * TN + ((uint32_t)(32 * q) << 16) + h * C::kCh;
        const float* fac = stage + ((g & 1) * kSG + kb % kSG) * C::kSPitch + h * C::kCh;
        uint32_t d[2][C::kCh];
        auto ld = [&](int i) {
          if (C::kCh == 32) tmem_ld32_nowait(trow + 2 * C::kCh * i, d[i & 1]);
          else tmem_ld16_nowait(trow + 2 * C::kCh * i, d[i & 1]);
        };
        ld(0);
#pragma unroll
        for (int i = 0; i < C::kNch; ++i) {
          tmem_ld_wait<C::kCh>(d[i & 1]);
          if (i + 1 < C::kNch) {
            ld(i + 1);
          } else {   // read: the accumulator may be written again
            asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
            if (lane == 0) {
              if (CG == 1) mbar_arrive(acc_empty(buf));
              else mbar_arrive_at(acc_empty(buf), 0);
            }
          }
#pragma unroll
          for (int c = 0; c < C::kCh / 4; ++c) {
            const ulonglong2 s = *reinterpret_cast<const ulonglong2*>(fac + 2 * C::kCh * i + 4 * c);
            fma2(acc[i][2 * c], pack2(d[i & 1][4 * c], d[i & 1][4 * c + 1]), s.x);
            fma2(acc[i][2 * c + 1], pack2(d[i & 1][4 * c + 2], d[i & 1][4 * c + 3]), s.y);
          }
        }
        if (kb % kSG == kSG - 1 && kb + 1 < p.nkb) {
          put(g + 1);   // the buffer of group g - 1, which every warp left before the last barrier
          if (!bar_and(1, kEpiThreads, true)) {
            ok = false;
            left = true;
            break;
          }
        }
      }
      if (left) break;
      if (!ok) continue;
      // column c is token row c; the warp's lanes are 32 neighbouring outputs of it
      const int m = mtile * 128 + 32 * q + lane;
      if (m < p.N) {
#pragma unroll
        for (int i = 0; i < C::kNch; ++i) {
          const int c0 = (2 * i + h) * C::kCh;
          const int el = p.out_f32 ? 4 : 2;
          const size_t pitch = (size_t)p.ld_out * el;
          uint8_t* dst = reinterpret_cast<uint8_t*>(p.out) + (size_t)(t.row0 + t.c0 + c0) * pitch + (size_t)m * el;
#pragma unroll
          for (int c = 0; c < C::kCh; ++c) {
            if (c0 + c >= t.cols) break;
            float v[2];
            unpack2(acc[i][c >> 1], v[0], v[1]);
            if (p.out_f32) *reinterpret_cast<float*>(dst) = v[c & 1];
            else *reinterpret_cast<__nv_bfloat16*>(dst) = __float2bfloat16_rn(v[c & 1]);
            dst += pitch;
            asm volatile("" : "+l"(dst));   // one running pointer, not kCh addresses in registers
          }
        }
      }
      __syncwarp();
    }
    // rows of no group
    if (p.offsets && p.zero_rest && *reinterpret_cast<volatile int*>(p.err) == 0) {
      const long t = (long)blockIdx.x * kEpiThreads + et, n = (long)gridDim.x * kEpiThreads;
      const int el = p.out_f32 ? 4 : 2;
      uint8_t* out = reinterpret_cast<uint8_t*>(p.out);
      const int2 last = group_rows(p.offsets, p.E - 1, p.S);
      zero_rows(out, 0, group_rows(p.offsets, 0, p.S).x, (size_t)p.N * el, (size_t)p.ld_out * el, t, n);
      zero_rows(out, last.x + last.y, p.S, (size_t)p.N * el, (size_t)p.ld_out * el, t, n);
    }
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  if (CG == 2) cluster_sync();   // no CTA leaves while the other may still signal it
  if (warp == 1) {
    __syncwarp();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    tmem_free<CG>(tmem, C::kTmemCols);
  }
}

template <int CG, int TN>
cudaError_t launch_t(const CUtensorMap& a, const CUtensorMap& b, const F8Params& p, long max_items, cudaStream_t st) {
  static std::atomic<uint64_t> raised{0};
  const long sms = sm_count();
  if (sms <= 0) return cudaErrorInvalidDevice;
  if (Cfg<CG, TN>::kSplitRegs) {   // the shares need the launch to hold their sum
    static const int regs = [] {
      cudaFuncAttributes fa;
      return cudaFuncGetAttributes(&fa, f8_kernel<CG, TN>) == cudaSuccess ? fa.numRegs : 0;
    }();
    if (regs < kLaunchRegs) return cudaErrorInvalidConfiguration;
  }
  const long ctas = max_items < sms / CG ? max_items * CG : sms / CG * CG;
  return launch_cluster(f8_kernel<CG, TN>, &raised, CG, (int)(ctas < CG ? CG : ctas), kThreads, Cfg<CG, TN>::kSmem, st, a, b, p);
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

  const double per = (double)g->S / g->E;
  const int tn = per <= 32 ? 32 : per <= 64 ? 64 : per <= 128 ? 128 : 256;
  constexpr int cg = 1;
  p.n_mt = (p.N + 128 * cg - 1) / (128 * cg);
  const double items = ((double)g->S / tn + p.E) * p.n_mt;
  if (items > 2.0e9) return SITU_ERR_BAD_SHAPE;
  CUtensorMap ma, mb;
  const uint64_t S = (uint64_t)g->S, N = (uint64_t)g->N, K = (uint64_t)g->K, E = (uint64_t)g->E;
  const uint64_t dw[3] = {K, N, E}, sw[2] = {K, N * K}, dx[2] = {K, S}, sx[1] = {(uint64_t)g->ldx};
  const uint32_t boxw[3] = {128, 128, 1}, boxx[2] = {128, (uint32_t)(tn / cg)};
  if (!make_map_nd(&ma, CU_TENSOR_MAP_DATA_TYPE_UINT8, g->w_q, 3, dw, sw, boxw) ||
      !make_map_nd(&mb, CU_TENSOR_MAP_DATA_TYPE_UINT8, g->x_q, 2, dx, sx, boxx))
    return SITU_ERR_CUDA;
  cudaStream_t st = (cudaStream_t)stream;
  const long cap = items > 1e6 ? 1000000 : (long)items + 1;
  const cudaError_t e = tn == 32    ? launch_t<cg, 32>(ma, mb, p, cap, st)
                        : tn == 64  ? launch_t<cg, 64>(ma, mb, p, cap, st)
                        : tn == 128 ? launch_t<cg, 128>(ma, mb, p, cap, st)
                                    : launch_t<cg, 256>(ma, mb, p, cap, st);
  return e == cudaSuccess ? SITU_OK : SITU_ERR_CUDA;
}
