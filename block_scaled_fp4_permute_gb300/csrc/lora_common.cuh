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

// Items dealt out evenly: CTA c of G takes [c T / G, (c + 1) T / G) of T, and
// item i is CTA ((i + 1) G - 1) / T's.
__host__ __device__ __forceinline__ long first_item(long c, long T, long G) { return c * T / G; }
__host__ __device__ __forceinline__ long cta_of(long i, long T, long G) { return ((i + 1) * G - 1) / T; }
// eight sums to memory, a whole sector a lane; add: to what is there
__device__ __forceinline__ void put8(float* o, const uint32_t* v, bool add) {
  float f[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(v[i]);
  if (add) {
    const float4 a = *reinterpret_cast<const float4*>(o), b = *reinterpret_cast<const float4*>(o + 4);
    f[0] += a.x;
    f[1] += a.y;
    f[2] += a.z;
    f[3] += a.w;
    f[4] += b.x;
    f[5] += b.y;
    f[6] += b.z;
    f[7] += b.w;
  }
  asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(o), "f"(f[0]), "f"(f[1]), "f"(f[2]), "f"(f[3]),
               "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7])
               : "memory");
}

inline bool bad(const void* q, uintptr_t mask) { return (reinterpret_cast<uintptr_t>(q) & mask) != 0; }
// the tensor maps take strides below 2^40 bytes
inline bool bad_ld(int64_t ld, int64_t cols, int64_t unit) { return ld < cols || ld % unit != 0 || ld >= (int64_t)1 << 38; }

// da [n, r, K] = v^T x and db [n, N, r] = dy^T u over each adapter's rows, v and
// u [S, r] of the operands' type.  parts: outer_bytes(r) of scratch.
struct OuterArgs {
  int dtype, S, K, N, r, n;
  const void *x, *dy, *v, *u;
  int64_t ldx, ld_dy;
  const int32_t* offsets;
  void *da, *db;
  float* parts;
  int32_t* err;
};
size_t outer_bytes(int r);
bool outer_takes(int dtype, int S, int K, int N);   // else the sums are too long for one in tensor memory
situ_status launch_outer(const OuterArgs& a, cudaStream_t st);

}  // namespace lora
}  // namespace situ
