// fp8_quant.cu -- quantisation to E4M3 with one fp32 scale per block of 128
// elements of a row (activations) or of 128 rows x 128 columns (weights).
//
//   scale = max(amax / 448, 2^-126),  q = E4M3(x / scale), nearest even
// in IEEE fp32 (both divisions correctly rounded), so the codes are a
// function of the inputs alone.  The floor keeps the scale of a zero or
// vanishing block a normal number.  A block with an infinity or a NaN gets a
// non-finite scale and NaN codes where x / scale is a NaN: the damage stays
// visible in what is computed from it.
//
// Bound by memory: one read of x, one byte written per element.  Each lane
// takes eight neighbouring elements (16 bytes of a 16-bit type), sixteen
// lanes a row of a block.
#include "../../include/situ_moe.h"
#include "situ_internal.h"

namespace situ {

namespace {

constexpr int kBlk = 128;
constexpr float kMinScale = 1.17549435e-38f;   // 2^-126

template <int DT>
struct In {
  static constexpr int kVec = DT == SITU_DT_F32 ? 2 : 1;   // 16-byte loads per eight elements
  uint4 v[kVec];
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < kVec; ++i) v[i] = make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void load(const void* p, size_t el) {
    const uint4* q = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p) + el * (DT == SITU_DT_F32 ? 4 : 2));
#pragma unroll
    for (int i = 0; i < kVec; ++i) v[i] = __ldg(q + i);
  }
  __device__ __forceinline__ void get(float* f) const {
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (DT == SITU_DT_F32) {
          f[4 * i + j] = __uint_as_float(w[j]);
        } else if (DT == SITU_DT_BF16) {
          f[2 * j] = bf16_lo(w[j]);
          f[2 * j + 1] = bf16_hi(w[j]);
        } else {
          f[2 * j] = f16_to_f32(w[j] & 0xFFFFu);
          f[2 * j + 1] = f16_to_f32(w[j] >> 16);
        }
      }
    }
  }
};

// the largest magnitude as a bit pattern: ordered as the values are, with
// infinity above every finite value and NaN above infinity
__device__ __forceinline__ uint32_t amax_bits(const float* f) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(f[i]) & 0x7FFFFFFFu);
  return m;
}
__device__ __forceinline__ float scale_of(uint32_t bits) {
  const float s = __fdiv_rn(__uint_as_float(bits), 448.f);
  return s < kMinScale ? kMinScale : s;   // a NaN stays
}
__device__ __forceinline__ uint2 codes(const float* f, float s) {
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) c[i] = f32x2_to_e4m3x2(__fdiv_rn(f[2 * i], s), __fdiv_rn(f[2 * i + 1], s));
  return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

// A scale per 128 columns of a row: a half warp per block, kUnroll blocks in
// flight per half warp.
constexpr int kUnroll = 4;
template <int DT>
__global__ void __launch_bounds__(256)
quant_fp8_rows_kernel(const void* __restrict__ x, long ldx, long R, int K, int nkb, uint8_t* __restrict__ q,
                      float* __restrict__ scale) {
  const long hw = ((long)blockIdx.x * 256 + threadIdx.x) >> 4;
  const int l = threadIdx.x & 15;
  const long blocks = R * nkb, b0 = hw * kUnroll;
  In<DT> in[kUnroll];
  long row[kUnroll];
  int col[kUnroll];
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const long b = b0 + u;
    row[u] = b / nkb;
    col[u] = (int)(b - row[u] * nkb) * kBlk + 8 * l;
    in[u].zero();
    if (b < blocks && col[u] < K) in[u].load(x, (size_t)row[u] * (size_t)ldx + col[u]);
  }
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    float f[8];
    in[u].get(f);
    uint32_t m = amax_bits(f);
#pragma unroll
    for (int d = 8; d >= 1; d >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, d));
    const float s = scale_of(m);
    if (b0 + u >= blocks) continue;
    if (col[u] < K) *reinterpret_cast<uint2*>(q + (size_t)row[u] * K + col[u]) = codes(f, s);
    if (l == 0) scale[b0 + u] = s;
  }
}

// A scale per 128 x 128 block: one CTA per block, held in registers between
// the maximum and the codes.
template <int DT>
__global__ void __launch_bounds__(256)
quant_fp8_tiles_kernel(const void* __restrict__ x, long ldx, long lde, int R, int K, int nrb, int nkb,
                       uint8_t* __restrict__ q, float* __restrict__ scale) {
  __shared__ uint32_t wmax[8];
  const long b = blockIdx.x;
  const int kb = (int)(b % nkb);
  const long er = b / nkb;
  const int rb = (int)(er % nrb);
  const long e = er / nrb;
  const int l = threadIdx.x & 15, r = rb * kBlk + (threadIdx.x >> 4), col = kb * kBlk + 8 * l;
  In<DT> in[8];
  uint32_t m = 0;
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    in[u].zero();
    if (r + 16 * u < R && col < K) in[u].load(x, (size_t)e * lde + (size_t)(r + 16 * u) * ldx + col);
  }
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    float f[8];
    in[u].get(f);
    m = max(m, amax_bits(f));
  }
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, d));
  if ((threadIdx.x & 31) == 0) wmax[threadIdx.x >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 8; ++w) m = max(m, wmax[w]);
  const float s = scale_of(m);
  if (threadIdx.x == 0) scale[b] = s;
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    if (r + 16 * u >= R || col >= K) continue;
    float f[8];
    in[u].get(f);
    *reinterpret_cast<uint2*>(q + ((size_t)e * R + r + 16 * u) * (size_t)K + col) = codes(f, s);
  }
}

template <int DT>
cudaError_t launch_dt(const void* x, long ldx, long lde, int E, int R, int K, int block_rows, uint8_t* q, float* scale,
                      cudaStream_t st) {
  const int nkb = (K + kBlk - 1) / kBlk;
  if (block_rows == 1) {
    const long per = 16 * kUnroll, blocks = (long)E * R * nkb;
    quant_fp8_rows_kernel<DT><<<(unsigned)((blocks + per - 1) / per), 256, 0, st>>>(x, ldx, (long)E * R, K, nkb, q, scale);
  } else {
    const int nrb = (R + kBlk - 1) / kBlk;
    quant_fp8_tiles_kernel<DT><<<(unsigned)((long)E * nrb * nkb), 256, 0, st>>>(x, ldx, lde, R, K, nrb, nkb, q, scale);
  }
  return cudaGetLastError();
}

}  // namespace
}  // namespace situ

extern "C" situ_status situ_moe_quant_fp8(const void* x, int32_t dtype, int32_t E, int32_t R, int32_t K, int64_t ldx,
                                          int32_t block_rows, uint8_t* q, float* scale, void* stream) {
  using namespace situ;
  if (dtype != SITU_DT_BF16 && dtype != SITU_DT_F16 && dtype != SITU_DT_F32) return SITU_ERR_UNSUPPORTED;
  if (block_rows != 1 && block_rows != 128) return SITU_ERR_UNSUPPORTED;
  const int64_t vec = dtype == SITU_DT_F32 ? 4 : 8;
  if (E < 0 || R < 0 || K < 8 || K % 8 != 0 || K > SITU_GEMM_MAX_DIM || ldx < K || ldx % vec != 0) return SITU_ERR_BAD_SHAPE;
  if (E > 1 && block_rows == 1 && (int64_t)E * R > SITU_GEMM_MAX_ROWS) return SITU_ERR_BAD_SHAPE;
  if ((double)E * R * ((K + 127) / 128) / (block_rows == 1 ? 64.0 : 1.0) > 2.0e9) return SITU_ERR_BAD_SHAPE;
  if (E == 0 || R == 0) return SITU_OK;
  if (!x || !q || !scale) return SITU_ERR_NULL_ARG;
  if ((reinterpret_cast<uintptr_t>(x) & 15) || (reinterpret_cast<uintptr_t>(q) & 7) ||
      (reinterpret_cast<uintptr_t>(scale) & 3))
    return SITU_ERR_MISALIGNED;
  cudaStream_t st = (cudaStream_t)stream;
  const long lde = (long)R * (long)ldx;
  const cudaError_t e =
      dtype == SITU_DT_BF16  ? launch_dt<SITU_DT_BF16>(x, (long)ldx, lde, E, R, K, block_rows, q, scale, st)
      : dtype == SITU_DT_F16 ? launch_dt<SITU_DT_F16>(x, (long)ldx, lde, E, R, K, block_rows, q, scale, st)
                             : launch_dt<SITU_DT_F32>(x, (long)ldx, lde, E, R, K, block_rows, q, scale, st);
  return e == cudaSuccess ? SITU_OK : SITU_ERR_CUDA;
}
