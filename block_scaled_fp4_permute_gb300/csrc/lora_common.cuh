// lora_common.cuh -- what the adapters' kernels share (lora.cu, lora_grads.cu).
#pragma once
#include "../../include/situ_moe.h"
#include "gemm_groups.cuh"

namespace situ {
namespace lora {

using namespace gg;

constexpr int kMaxRank = 128;

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
// Of row `row`: ids' entry, or the adapter whose rows hold it; -1: none.
__device__ __forceinline__ int adapter_of(const int32_t* ids, const int32_t* offsets, int n, int row) {
  if (ids) {
    const int e = __ldcg(ids + row);
    return e >= 0 && e < n ? e : -1;
  }
  int lo = 0, hi = n + 1;          // the first entry beyond row lies in [lo, hi]
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (__ldcg(offsets + mid) > row) hi = mid;
    else lo = mid + 1;
  }
  return lo <= n ? lo - 1 : -1;
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

// D[128, N] of 16-bit operands in fp32; trans_a, trans_b: A's M, B's N elements contiguous
__device__ __forceinline__ uint32_t idesc_of(bool bf16, bool trans_a, bool trans_b, int N) {
  return (1u << 4) | (bf16 ? (1u << 7) | (1u << 10) : 0u) | (trans_a ? 1u << 15 : 0u) | (trans_b ? 1u << 16 : 0u) | ((uint32_t)(N >> 3) << 17) |
         ((uint32_t)(128 >> 4) << 24);
}

__device__ __forceinline__ void mbar_arrive_n(uint32_t a, uint32_t n) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(a), "r"(n) : "memory");
}

// Items dealt out evenly: CTA c of G takes [c T / G, (c + 1) T / G) of T, and
// item i is CTA ((i + 1) G - 1) / T's.
__host__ __device__ __forceinline__ long first_item(long c, long T, long G) { return c * T / G; }
__host__ __device__ __forceinline__ long cta_of(long i, long T, long G) { return ((i + 1) * G - 1) / T; }
// How a product's chunks (`chunks` to each of `tiles`) are dealt out: one CTA per
// SM, of at least two chunks; `most`: the parts that a tile can come in.
struct Shares {
  long ctas, least, most;
  Shares(long tiles, long chunks, long sms) {
    const long total = tiles * chunks;
    ctas = total / 2 < sms ? total / 2 : sms;
    if (ctas < 1) ctas = 1;
    least = total / ctas;
    if (least < 1) least = 1;
    most = (chunks + least - 2) / least + 1;
    if (most > chunks) most = chunks;
  }
};
// The CTAs that have a share where only `total` chunks are left (rows without an
// adapter sorted out): fewer, so that a tile still comes in no more parts.
__host__ __device__ __forceinline__ long sharers(long total, long ctas, long least) {
  const long g = total / least;
  return g < 1 ? 1 : g < ctas ? g : ctas;
}

// eight sums to memory, a whole sector a lane
__device__ __forceinline__ void put8(float* o, const float* f) {
  asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(o), "f"(f[0]), "f"(f[1]), "f"(f[2]), "f"(f[3]),
               "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7])
               : "memory");
}

inline bool bad(const void* q, uintptr_t mask) { return (reinterpret_cast<uintptr_t>(q) & mask) != 0; }
// the tensor maps take strides below 2^40 bytes
inline bool bad_ld(int64_t ld, int64_t cols, int64_t unit) { return ld < cols || ld % unit != 0 || ld >= (int64_t)1 << 38; }

// u or v of a row is kept in two terms of the operands' type, [2][r]: rounded, and
// what that leaves (an infinity leaves nothing), together 16 bits of it in bf16 and
// 22 in f16, less where f16 has no smaller steps (2^-24) or no larger values.
template <int DT>
__device__ __forceinline__ void two_terms(float a, float b, uint32_t& hi, uint32_t& lo) {
  hi = pack16<DT>(a, b);
  const float x = lo16<DT>(hi), y = hi16<DT>(hi);
  lo = pack16<DT>(fabsf(x) < INFINITY ? a - x : 0.f, fabsf(y) < INFINITY ? b - y : 0.f);
}

// The backward pass of f16 takes v and u in terms under powers of two, one per adapter,
// which its sums are multiplied by again.
// Values whose largest finite magnitude is m are divided by 2^power_of(m) first, which
// brings m to [2^14, 2^15): two terms then hold 22 bits of each, or all of it down to
// 2^-39 of m.
__device__ __forceinline__ int power_of(float m) {
  const int k = (int)(__float_as_uint(m) >> 23) - 127;   // m in [2^k, 2^(k + 1))
  return m > 0.f ? max(-100, min(120, k - 14)) : 0;
}
__device__ __forceinline__ float finite_max(float m, float v) {
  const float a = fabsf(v);
  return a < INFINITY ? fmaxf(m, a) : m;
}
// *most, the bits of a magnitude, at least m's.  Few of many rows raise it: a look
// first, where their atomics on one address would wait for each other.
__device__ __forceinline__ void raise_most(uint32_t* most, float m) {
  const uint32_t bits = __float_as_uint(m);
  if (bits > __ldcg(most)) atomicMax(most, bits);
}

// How a warp goes through rows of r fp32: four columns a lane, as many rows as
// lanes hold, kRowTurns of those together; unit: the warp's number.
constexpr int kRowTurns = 4;
struct RowLanes {
  int q, per, at, j;                     // lanes of a row, rows of a warp; the lane's row of these, its column
  long row0;
  __host__ __device__ static long rows(int r) { return kRowTurns * (32 / (r / 4)); }
  __device__ __forceinline__ RowLanes(int r, long unit) {
    const int lane = threadIdx.x & 31;
    q = r / 4;
    per = 32 / q;
    at = lane / q;
    j = 4 * (lane - at * q);
    row0 = unit * kRowTurns * per;
  }
  __device__ __forceinline__ long row(int turn, int S) const {   // S: none
    const long i = row0 + (long)turn * per + at;
    return at < per && i < S ? i : S;
  }
  // the largest of a row's lanes, in each
  __device__ __forceinline__ float largest(float m) const {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) {
      const float v = __shfl_down_sync(0xffffffffu, m, o);
      if (j / 4 + o < q) m = fmaxf(m, v);
    }
    return __shfl_sync(0xffffffffu, m, min(at * q, 31));
  }
};

// da [n, r, K] = v^T x and db [n, N, r] = dy^T u over each adapter's rows.  bf16: v
// and u [S, 2, r] in two terms.  f16: v fp32 [S, r], which is turned into such terms; u in
// them, but rows whose row_most is negative are u32's (fp32), which receives the terms
// of all; most [2][n] the bits of the adapters' largest of v and u.  parts:
// outer_bytes(r) of scratch.
struct OuterArgs {
  int dtype, S, K, N, r, n;
  const void *x, *dy, *u;
  void* v;
  float* u32;
  const float* row_most;
  const uint32_t* most;
  const float* dy_scale;                 // [1] or null: what dy counts times (v has it already)
  int64_t ldx, ld_dy;
  const int32_t* offsets;
  void *da, *db;
  float* parts;
  int32_t* err;
};
size_t outer_bytes(int r);
situ_status launch_outer(const OuterArgs& a, cudaStream_t st);

}  // namespace lora
}  // namespace situ
