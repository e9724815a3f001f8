// lora_grads.cu -- the gradients of low-rank adapters: sums over the rows of each.
//
//   dA[e][j][k] = sum_{rows i of e} v[i, j] x[i, k],   dB[e][n][j] = sum dy[i, n] u[i, j]
//
// Both are one form: 128 columns of a wide operand (x or dy) on the MMA's M side,
// the columns of a narrow one on its N side, rows along the contraction (both
// operands MN-major).  u and v come in two 16-bit terms, side by side on the N side:
// rounded to one, the gradients would be off by as much again as their own
// rounding.  In f16 the terms are those of u and v under a power of two per adapter,
// which its sums are multiplied by again: v of a fine-tuning run's first steps lies
// far below f16's smallest step.  The kernels that make v look at u as well and leave
// the adapters' largest; terms_kernel makes the terms.  Bound by the bytes of x and dy: r operations a byte.  The
// general products over groups (situ_moe_grouped_gemm) give whole tiles to CTAs, and
// four adapters of 3584 x 6144 make 56 and 96 tiles for 152 SMs.  Here the
// chunks of 64 rows of all tiles of both gradients are dealt out evenly over one CTA
// per SM; tiles that part between CTAs leave fp32 sums, which a second kernel
// adds in order (16,384 rows, rank 64: 93 us as two general products of single
// terms, 72 so, at 4.4 TB/s, the join 4 of them; tiles of 256 columns take half the
// copies of the narrow operand and leave twice the sums to join: 6 us more).
//
// A tile's last chunk has fewer than 64 rows: it comes row by row (four an
// instruction), rows past the adapter's end named out of bounds, so that the MMA
// sees zeros in both operands there: the neighbour's rows may hold infinities.
#include "lora_common.cuh"

namespace situ {
namespace lora {

namespace {

constexpr int kThreads = 256;            // copies, MMAs, two idle; four epilogue warps
constexpr int kRows = 64;                // of a stage
constexpr int kWide = 2 * kRows * 128;   // bytes of 128 columns of them
constexpr int kMaxStages = 8;
constexpr int kSmem = 212 * 1024;        // 227 KB with the scan and the static part

struct OuterParams {
  const int32_t* offsets;
  int S, n, r;
  int C[2], blocks[2];                   // of x and dy: columns, tiles of 128
  void* out[2];                          // da, db
  const uint32_t* most;                  // f16: [2][n], the bits of each adapter's largest v and u
  const float* dy_scale;
  float* parts;                          // [CTA][2][128][r]
  int stages, run;                       // run: chunks of a sum in tensor memory
  int* err;
};
// wide and narrow operand of each gradient, by 64 rows and by single ones
struct OuterMaps {
  CUtensorMap wide[2], narrow[2], wide1[2], narrow1[2];
};

// What a CTA has of one tile.
struct Piece {
  int which, e, block, from, to, chunks, row0, rows;   // chunks of the tile, the adapter's rows
  __device__ __forceinline__ bool whole() const { return from == 0 && to == chunks; }
};
struct Deal {
  const int *tp, *row;
  int n, blocks_a, blocks_b;
  long total;
  __device__ __forceinline__ Deal(const OuterParams& p, const int* tp_, const int* row_)
      : tp(tp_), row(row_), n(p.n), blocks_a(p.blocks[0]), blocks_b(p.blocks[1]), total((long)tp_[p.n] * (blocks_a + blocks_b)) {}
  // of items [i, end) the part in i's tile: first dA's tiles, by adapter, then dB's
  __device__ __forceinline__ Piece at(long i, long end) const {
    Piece t;
    const long a = (long)tp[n] * blocks_a;
    t.which = i >= a;
    const long j = t.which ? i - a : i;
    const int blocks = t.which ? blocks_b : blocks_a;
    t.e = find_group(tp, n, (int)(j / blocks));
    t.chunks = tp[t.e + 1] - tp[t.e];
    const long rem = j - (long)tp[t.e] * blocks;
    t.block = (int)(rem / t.chunks);
    t.from = (int)(rem - (long)t.block * t.chunks);
    t.to = (int)min((long)t.chunks, t.from + (end - i));
    t.row0 = row[t.e];
    t.rows = row[t.e + 1] - row[t.e];
    return t;
  }
};

// What a piece's sums count times: what dy does, and in f16 what v or u of its adapter
// was divided by.
template <int DT>
__device__ __forceinline__ float factor_of(const OuterParams& p, const Piece& t) {
  const float f = DT == SITU_DT_F16 ? exp2i(power_of(__uint_as_float(__ldcg(p.most + t.which * p.n + t.e)))) : 1.f;
  return t.which && p.dy_scale ? f * __ldg(p.dy_scale) : f;
}

// Sums of column c of a tile to the gradient, rounded: da is [j][c], db [c][j].
template <int DT>
__device__ __forceinline__ void store16(const OuterParams& p, const Piece& t, float f, int c, int j, float* v) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] *= f;
  uint16_t* out = static_cast<uint16_t*>(p.out[t.which]);
  if (t.which == 0) {
    out += ((size_t)t.e * p.r + j) * p.C[0] + c;
#pragma unroll
    for (int i = 0; i < 8; ++i) out[(size_t)i * p.C[0]] = (uint16_t)pack16<DT>(v[i], 0.f);
  } else {
    *reinterpret_cast<uint4*>(out + ((size_t)t.e * p.C[1] + c) * p.r + j) =
        make_uint4(pack16<DT>(v[0], v[1]), pack16<DT>(v[2], v[3]), pack16<DT>(v[4], v[5]), pack16<DT>(v[6], v[7]));
  }
}

template <int DT>
__global__ void __launch_bounds__(kThreads, 1)
outer_kernel(const __grid_constant__ OuterMaps m, const OuterParams p) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ int scan[kScanInts];
  __shared__ uint64_t bars[2 * kMaxStages + 5];
  __shared__ uint32_t holder[2];
  const uint32_t sbase = (saddr(smem_raw) + 1023) & ~1023u;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t bar0 = saddr(bars);
  auto full = [&](int s) { return bar0 + 8 * s; };
  auto empty = [&](int s) { return bar0 + 8 * (kMaxStages + s); };
  auto acc_full = [&](int b) { return bar0 + 8 * (2 * kMaxStages + b); };
  auto acc_empty = [&](int b) { return bar0 + 8 * (2 * kMaxStages + 2 + b); };
  const uint32_t drain = bar0 + 8 * (2 * kMaxStages + 4);
  if (tid == 0) {
    holder[1] = (uint32_t)*reinterpret_cast<volatile int*>(p.err);   // an earlier launch gave up a wait: no work then
    for (int s = 0; s < 2 * kMaxStages; ++s) mbar_init(bar0 + 8 * s, 1);
    for (int b = 0; b < 2; ++b) {
      mbar_init(acc_full(b), 1);
      mbar_init(acc_empty(b), 4);
    }
    mbar_init(drain, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) tmem_alloc<1>(saddr(holder), 512);
  scan_tiles(p.offsets, p.n, p.S, kRows, scan, scan + kMaxGroups + 1, kThreads);
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = holder[0];
  const bool dead = holder[1] != 0;
  const Deal deal(p, scan, scan + kMaxGroups + 1);
  const long i0 = first_item(blockIdx.x, deal.total, gridDim.x), i1 = first_item(blockIdx.x + 1, deal.total, gridDim.x);
  const int nboxes = (2 * p.r + 63) / 64, stage = kWide + nboxes * kRows * 128;

  if (warp == 0 && !dead) {
    // ---------------- copies ----------------
    const bool leader = elect_one();
    bool ok = true;
    // of the chunks [a, b), x or dy and v or u
    auto copy = [&](long a, long b, Turns& r, bool wide, bool narrow) {
      for (long i = a; i < b && ok;) {
        const Piece t = deal.at(i, b);
        i += t.to - t.from;
        const int c0 = t.block * 128, wboxes = c0 + 64 < p.C[t.which] ? 2 : 1;
        for (int k = t.from; k < t.to; ++k, r.next()) {
          if (r.again() && !warp_wait(empty(r.s), r.ph ^ 1, p.err, 121)) {
            ok = false;
            break;
          }
          const uint32_t to = sbase + r.s * stage;
          const int left = t.rows - k * kRows, row = t.row0 + k * kRows;
          const int fours = left >= kRows ? kRows / 4 : (left + 15) / 16 * 4;
          if (leader && wide) mbar_expect_tx(full(r.s), (wboxes + nboxes) * fours * 512);
          if (left >= kRows) {
            if (leader) {
              for (int h = 0; h < wboxes && wide; ++h) copy_2d<1>(to + h * kRows * 128, &m.wide[t.which], c0 + 64 * h, row, full(r.s));
              for (int h = 0; h < nboxes && narrow; ++h)
                copy_2d<1>(to + kWide + h * kRows * 128, &m.narrow[t.which], 64 * h, row, full(r.s));
            }
          } else {
            __syncwarp();
            const int from = wide ? 0 : wboxes, end = wboxes + (narrow ? nboxes : 0);
            for (int g = from * fours + lane; g < end * fours; g += 32) {
              const int box = g / fours, f = 4 * (g - box * fours);
              int at[4];
#pragma unroll
              for (int j = 0; j < 4; ++j) at[j] = f + j < left ? row + f + j : p.S;
              const bool x = box < wboxes;
              copy_rows4<1>(to + (x ? box : 2 + box - wboxes) * kRows * 128 + f * 128,
                            x ? &m.wide1[t.which] : &m.narrow1[t.which], x ? c0 + 64 * box : 64 * (box - wboxes), at[0], at[1],
                            at[2], at[3], full(r.s));
            }
          }
          __syncwarp();
        }
      }
    };
    // v is the predecessor's: the first round's x and dy come meanwhile
    const long first = min(i1, i0 + p.stages);
    Turns ahead(p.stages), r(p.stages);
    copy(i0, first, ahead, true, false);
    griddep_wait();
    copy(i0, first, r, false, true);
    copy(first, i1, r, true, true);
    leave(
        ok, [&] { return r.last([&](int j, uint32_t ph) { return warp_wait(empty(j), ph, p.err, 122); }); },
        [&] { r.last([&](int j, uint32_t ph) { return drain_wait(full(j), ph); }); });
  } else if (warp == 1 && !dead) {
    // ---------------- MMAs ----------------
    const bool leader = elect_one();
    const uint32_t idesc = idesc_of(DT == SITU_DT_BF16, true, true, 2 * p.r);
    Turns r(p.stages), acc(2);
    bool ok = true;
    griddep_wait();                       // bounded waits for what comes of v begin here
    for (long i = i0; i < i1 && ok;) {
      const Piece t = deal.at(i, i1);
      i += t.to - t.from;
      for (int from = t.from; from < t.to && ok; from += p.run) {
        const int to = min(t.to, from + p.run);
        if (acc.again() && !warp_wait(acc_empty(acc.s), acc.ph ^ 1, p.err, 123)) {
          ok = false;
          break;
        }
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        for (int k = from; k < to; ++k, r.next()) {
          if (!warp_wait(full(r.s), r.ph, p.err, 124)) {
            ok = false;
            break;
          }
          asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
          if (leader) {
            const uint32_t a = sbase + r.s * stage;
            const int steps = min(kRows / 16, (t.rows - k * kRows + 15) / 16);
            for (int j = 0; j < steps; ++j)
              mma_f16<1>(tmem + acc.s * 256, sdesc_mn(a, kRows * 128) + 128 * j, sdesc_mn(a + kWide, kRows * 128) + 128 * j, idesc,
                         ((k - from) | j) != 0);
            mma_commit(empty(r.s));
          }
          __syncwarp();
        }
        if (ok) {
          if (leader) mma_commit(acc_full(acc.s));
          __syncwarp();
          acc.next();
        }
      }
    }
    leave(
        ok, [&] { return r.last([&](int j, uint32_t ph) { return warp_wait(empty(j), ph, p.err, 125); }); },
        [&] {
          if (leader) mma_commit(drain);
          __syncwarp();
          drain_wait(drain, 0);
        });
  } else if (warp >= 4 && !dead) {
    // ---------------- sums to memory, a column per lane ----------------
    const int q = warp & 3;
    // adapters without rows
    for (int e = 0; e < p.n; ++e) {
      if (scan[e] != scan[e + 1]) continue;
      for (int w = 0; w < 2; ++w) {
        uint4* out = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out[w]) + (size_t)e * p.r * p.C[w]);
        const long pieces = (long)p.r * p.C[w] / 8;
        for (long i = (long)blockIdx.x * 128 + tid - 128; i < pieces; i += (long)gridDim.x * 128) out[i] = make_uint4(0, 0, 0, 0);
      }
    }
    griddep_wait();                       // `most` is the predecessors'
    Turns acc(2);
    bool ok = true;
    for (long i = i0; i < i1 && ok;) {
      const Piece t = deal.at(i, i1);
      i += t.to - t.from;
      const int c = t.block * 128 + 32 * q + lane;
      const float back = factor_of<DT>(p, t);
      float* part = p.parts + (((size_t)blockIdx.x * 2 + (t.from == 0)) * 128 + 32 * q + lane) * p.r;
      for (int from = t.from; from < t.to && ok; from += p.run, acc.next()) {
        if (!warp_wait(acc_full(acc.s), acc.ph, p.err, 126)) {
          ok = false;
          break;
        }
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        const bool earlier = from > t.from, last = from + p.run >= t.to;   // sums of this piece are in `part`; these end it
        const uint32_t sums = tmem + ((uint32_t)(32 * q) << 16) + acc.s * 256;
        for (int j = 0; j < p.r; j += 8) {                // of the first term and of the second, from whole sixteens
          uint32_t v[16], w[16];
          __syncwarp();
          tmem_ld16_nowait(sums + (j & ~15), v);
          tmem_ld16_nowait(sums + ((p.r + j) & ~15), w);
          tmem_ld_wait<16>(v);
          tmem_ld_wait<16>(w);
          if (c >= p.C[t.which]) continue;
          const bool vh = j & 8, wh = (p.r + j) & 8;
          float f[8];
#pragma unroll
          for (int x = 0; x < 8; ++x) {
            f[x] = __uint_as_float(vh ? v[8 + x] : v[x]) + __uint_as_float(wh ? w[8 + x] : w[x]);
            if (earlier) f[x] += part[j + x];
          }
          if (last && t.whole()) store16<DT>(p, t, back, c, j, f);
          else put8(part + j, f);
        }
        __syncwarp();
        asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
        mbar_arrive_if(acc_empty(acc.s), lane == 0);
      }
    }
  }
  if (dead) griddep_wait();
  griddep_launch_dependents();
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    tmem_free<1>(tmem, 512);
  }
}

// The tile that begins in CTA blockIdx.x and goes on in later ones: its sums
// added up in their order, all of a tile's loads of two parts in flight (a few at a
// time took 6 us).  A round without parts comes first, while the predecessor ends:
// it brings the instructions in.
constexpr int kJoinThreads = 512;
template <int DT>
__global__ void __launch_bounds__(kJoinThreads)
outer_join_kernel(const OuterParams p) {
  __shared__ int scan[kScanInts];
  scan_tiles(p.offsets, p.n, p.S, kRows, scan, scan + kMaxGroups + 1, kJoinThreads);
  const Deal deal(p, scan, scan + kMaxGroups + 1);
  const long G = gridDim.x, i0 = first_item(blockIdx.x, deal.total, G), i1 = first_item(blockIdx.x + 1, deal.total, G);
  if (i0 == i1) {
    griddep_wait();
    return;
  }
  // the piece that holds the CTA's last item
  const Piece t = deal.at(i1 - 1, deal.total);
  const bool mine = t.from + 1 != t.chunks && t.from < i1 - i0;   // else it ends here, or began before
  const int last = mine ? (int)cta_of(i1 - 1 + (t.chunks - t.from - 1), deal.total, G) : -1;
  for (int round = 0; round < 2; ++round) {
    if (round == 1) {
      griddep_wait();
      if (!mine || *reinterpret_cast<volatile int*>(p.err) != 0) return;   // no parts where a wait was given up
    }
    const int end = round == 1 ? last : -1;
    const float back = round == 1 ? factor_of<DT>(p, t) : 1.f;
    for (int i = threadIdx.x; i < 128 * p.r / 8; i += kJoinThreads) {
      const int c = i * 8 / p.r, j = i * 8 - c * p.r;
      const bool in = t.block * 128 + c < p.C[t.which];
      float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      for (int k0 = blockIdx.x; k0 == (int)blockIdx.x || k0 <= end; k0 += 2) {
        float4 v[2][2];
#pragma unroll
        for (int d = 0; d < 2; ++d) {
          const int k = k0 + d;
          // (more CTAs than items)
          const bool there = in && k <= end && first_item(k, deal.total, G) != first_item(k + 1, deal.total, G);
          const float4* q =
              reinterpret_cast<const float4*>(p.parts + (((size_t)k * 2 + (k == (int)blockIdx.x)) * 128 + c) * p.r + j);
          v[d][0] = there ? __ldcg(q) : make_float4(0.f, 0.f, 0.f, 0.f);
          v[d][1] = there ? __ldcg(q + 1) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll
        for (int d = 0; d < 2; ++d) {
          s[0] += v[d][0].x;
          s[1] += v[d][0].y;
          s[2] += v[d][0].z;
          s[3] += v[d][0].w;
          s[4] += v[d][1].x;
          s[5] += v[d][1].y;
          s[6] += v[d][1].z;
          s[7] += v[d][1].w;
        }
      }
      if (in && round == 1) store16<DT>(p, t, back, t.block * 128 + c, j, s);
    }
  }
}

// f16: v and u to two terms under their adapters' powers of two.  7 us of 152 (16,384
// rows at rank 64), which a launch and the adapters' search take; the look at u as a
// kernel of its own beside the shrink cost 4 to 10 more.
constexpr int kTermWarps = 8;
struct TermsParams {
  const uint16_t* u;
  float *v, *u32;
  const float* row_most;
  int S, r, n;
  const int32_t* offsets;
  const uint32_t* most;
};
__global__ void __launch_bounds__(32 * kTermWarps)
terms_kernel(const TermsParams p) {
  constexpr int kF16 = SITU_DT_F16;
  griddep_launch_dependents();
  const RowLanes k(p.r, (long)blockIdx.x * kTermWarps + (threadIdx.x >> 5));
  const int which = blockIdx.y;
  float* const to = which ? p.u32 : p.v;
  int e[kRowTurns];
  float4 v[kRowTurns];
#pragma unroll
  for (int i = 0; i < kRowTurns; ++i) {
    const long row = k.row(i, p.S);
    e[i] = row < p.S ? adapter_of(nullptr, p.offsets, p.n, (int)row) : -1;
    v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (which && row < p.S) {
      const uint2 hi = __ldg(reinterpret_cast<const uint2*>(p.u + (size_t)row * 2 * p.r + k.j));
      const uint2 lo = __ldg(reinterpret_cast<const uint2*>(p.u + ((size_t)row * 2 + 1) * p.r + k.j));
      v[i] = make_float4(lo16<kF16>(hi.x) + lo16<kF16>(lo.x), hi16<kF16>(hi.x) + hi16<kF16>(lo.x),
                         lo16<kF16>(hi.y) + lo16<kF16>(lo.y), hi16<kF16>(hi.y) + hi16<kF16>(lo.y));
    }
  }
  griddep_wait();
  uint32_t m[kRowTurns];
#pragma unroll
  for (int i = 0; i < kRowTurns; ++i) {
    const long row = k.row(i, p.S);
    m[i] = e[i] >= 0 ? __ldcg(p.most + which * p.n + e[i]) : 0;
    if (row < p.S && (which == 0 || (__float_as_uint(__ldcg(p.row_most + row)) >> 31) != 0))
      v[i] = __ldcg(reinterpret_cast<const float4*>(to + (size_t)row * p.r + k.j));
  }
  __syncwarp();                            // all of a row is read before any of it is written
#pragma unroll
  for (int i = 0; i < kRowTurns; ++i) {
    const long row = k.row(i, p.S);
    if (row >= p.S) continue;
    const float f = exp2i(-power_of(__uint_as_float(m[i])));
    uint2 hi, lo;
    two_terms<kF16>(v[i].x * f, v[i].y * f, hi.x, lo.x);
    two_terms<kF16>(v[i].z * f, v[i].w * f, hi.y, lo.y);
    uint16_t* o = reinterpret_cast<uint16_t*>(to + (size_t)row * p.r) + k.j;
    *reinterpret_cast<uint2*>(o) = hi;
    *reinterpret_cast<uint2*>(o + p.r) = lo;
  }
}

template <int DT>
cudaError_t launch_dt(const OuterMaps& m, const OuterParams& p, int smem, cudaStream_t st) {
  static std::atomic<uint64_t> raised{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (bit == 0 || !(raised.load() & bit)) {
    std::lock_guard<std::mutex> lock(attr_mutex());
    e = cudaFuncSetAttribute(outer_kernel<DT>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    raised.fetch_or(bit);
  }
  const unsigned grid = (unsigned)sm_count();
  e = launch_pdl(outer_kernel<DT>, dim3(grid), dim3(kThreads), smem, st, m, p);
  return e != cudaSuccess ? e : launch_pdl(outer_join_kernel<DT>, dim3(grid), dim3(kJoinThreads), 0, st, p);
}

}  // namespace

size_t outer_bytes(int r) { return (size_t)sm_count() * 2 * 128 * r * 4; }

situ_status launch_outer(const OuterArgs& a, cudaStream_t st) {
  OuterParams p = {};
  p.offsets = a.offsets;
  p.S = a.S;
  p.n = a.n;
  p.r = a.r;
  // The tensor cores truncate when they add, 6e-9 of a sum of one sign per element:
  // a tenth of a 16-bit result's last unit after 65,536 (bf16) and 8,192 (f16).
  p.run = (a.dtype == SITU_DT_BF16 ? 65536 : 8192) / kRows;
  p.C[0] = a.K;
  p.C[1] = a.N;
  p.blocks[0] = (a.K + 127) / 128;
  p.blocks[1] = (a.N + 127) / 128;
  p.out[0] = a.da;
  p.out[1] = a.db;
  p.parts = a.parts;
  p.err = a.err;
  p.most = a.most;
  p.dy_scale = a.dy_scale;
  const bool f16 = a.dtype == SITU_DT_F16;
  if (f16) {
    const TermsParams t = {static_cast<const uint16_t*>(a.u), static_cast<float*>(a.v), a.u32, a.row_most, a.S, a.r, a.n, a.offsets,
                           a.most};
    const long rows = kTermWarps * RowLanes::rows(a.r);   // of a block
    if (launch_pdl(terms_kernel, dim3((unsigned)((a.S + rows - 1) / rows), 2), dim3(32 * kTermWarps), 0, st, t) != cudaSuccess)
      return SITU_ERR_CUDA;
  }
  const int stage = kWide + (2 * a.r + 63) / 64 * kRows * 128;
  p.stages = (kSmem - 1024) / stage;
  if (p.stages > kMaxStages) p.stages = kMaxStages;
  const CUtensorMapDataType dt = a.dtype == SITU_DT_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  OuterMaps m;
  const void *wide[2] = {a.x, a.dy}, *narrow[2] = {a.v, f16 ? a.u32 : a.u};
  const int64_t ld[2] = {a.ldx, a.ld_dy};
  const uint32_t box[2] = {64, kRows}, one[2] = {64, 1};
  bool ok = true;
  for (int i = 0; i < 2 && ok; ++i) {
    const uint64_t dw[2] = {(uint64_t)p.C[i], (uint64_t)a.S}, sw[1] = {(uint64_t)ld[i] * 2};
    const uint64_t dn[2] = {(uint64_t)a.r * 2, (uint64_t)a.S}, sn[1] = {(uint64_t)a.r * 4};
    ok = make_map_nd(&m.wide[i], dt, wide[i], 2, dw, sw, box) && make_map_nd(&m.wide1[i], dt, wide[i], 2, dw, sw, one) &&
         make_map_nd(&m.narrow[i], dt, narrow[i], 2, dn, sn, box) && make_map_nd(&m.narrow1[i], dt, narrow[i], 2, dn, sn, one);
  }
  if (!ok) return SITU_ERR_CUDA;
  const int smem = 1024 + p.stages * stage;
  const cudaError_t e = !f16 ? launch_dt<SITU_DT_BF16>(m, p, smem, st) : launch_dt<SITU_DT_F16>(m, p, smem, st);
  return e == cudaSuccess ? SITU_OK : SITU_ERR_CUDA;
}

}  // namespace lora
}  // namespace situ
