// fp8_quant.cu -- quantisation to E4M3 with one fp32 scale per block of 128
// elements of a row (activations) or of 128 rows x 128 columns (weights).
//
//   scale = max(amax / 448, 2^-126),  q = E4M3(x / scale), nearest even
// in IEEE fp32 (both divisions correctly rounded), so the codes are a
// function of the inputs alone.  The floor keeps the scale of a zero or
// vanishing block a normal number.  Zeros keep their sign.  A block with an
// infinity or a NaN gets a non-finite scale and NaN codes where x / scale is a
// NaN: the damage stays visible in what is computed from it.
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
  // the signs of elements 4h to 4h + 3 at the tops of four bytes
  __device__ __forceinline__ uint32_t signs(int h) const {
    const uint4& u = v[DT == SITU_DT_F32 ? h : 0];
    uint32_t w;
    if (DT == SITU_DT_F32) w = __byte_perm(__byte_perm(u.x, u.y, 0x0073), __byte_perm(u.z, u.w, 0x0073), 0x5410);
    else w = h == 0 ? __byte_perm(u.x, u.y, 0x7531) : __byte_perm(u.z, u.w, 0x7531);
    return w & 0x80808080u;
  }
  // elements 2j and 2j + 1
  __device__ __forceinline__ void pair(int j, float& a, float& b) const {
    const uint4& u = v[DT == SITU_DT_F32 ? j >> 1 : 0];
    if (DT == SITU_DT_F32) {
      a = __uint_as_float(j & 1 ? u.z : u.x);
      b = __uint_as_float(j & 1 ? u.w : u.y);
    } else {
      const uint32_t w = j == 0 ? u.x : j == 1 ? u.y : j == 2 ? u.z : u.w;
      a = DT == SITU_DT_BF16 ? bf16_lo(w) : f16_to_f32(w & 0xFFFFu);
      b = DT == SITU_DT_BF16 ? bf16_hi(w) : f16_to_f32(w >> 16);
    }
  }
};

// Magnitudes are compared as bit patterns, which are ordered as the values
// are, with infinity above every finite value and NaN above infinity: for
// 16-bit types two at a time.
template <int DT>
__device__ __forceinline__ uint32_t amax_word(uint32_t m, const uint4& v) {
  if (DT == SITU_DT_F32)
    return max(max(max(m, v.x & 0x7FFFFFFFu), max(v.y & 0x7FFFFFFFu, v.z & 0x7FFFFFFFu)), v.w & 0x7FFFFFFFu);
  return __vmaxu2(__vmaxu2(__vmaxu2(m, v.x & 0x7FFF7FFFu), __vmaxu2(v.y & 0x7FFF7FFFu, v.z & 0x7FFF7FFFu)),
                  v.w & 0x7FFF7FFFu);
}
template <int DT>
__device__ __forceinline__ uint32_t amax_join(uint32_t a, uint32_t b) {
  return DT == SITU_DT_F32 ? max(a, b) : __vmaxu2(a, b);
}
template <int DT>
__device__ __forceinline__ float amax_value(uint32_t m) {
  if (DT == SITU_DT_F32) return __uint_as_float(m);
  const uint32_t h = max(m & 0xFFFFu, m >> 16);
  return DT == SITU_DT_BF16 ? __uint_as_float(h << 16) : f16_to_f32(h);
}
// x / s correctly rounded, from r = 1 / s correctly rounded: a product, one
// residual step that makes it faithful and a second that rounds it correctly
// (Markstein, "Computation of elementary functions on the IBM RISC
// System/6000 processor", 1990).  Needs s in [2^-80, inf): the residuals of
// any quotient of at least 2^-20 are then exact, and a smaller one becomes
// the code 0 all the same.  A zero loses its sign in the residual (-0 gives
// +0 - 0): the codes take x's.  As packed pairs that is 2.5 instructions an
// element; with divisions the kernels were bound by issue slots.
__device__ __forceinline__ float quotient(float x, float s, float r) {
  float q = x * r;
  q = fmaf(fmaf(-q, s, x), r, q);
  return fmaf(fmaf(-q, s, x), r, q);
}
__device__ __forceinline__ uint64_t pair64(float a, float b) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ uint64_t fma_pair(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t mul_pair(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
// A block's scale, its negative and its reciprocal in pairs, fast = whether
// quotient() holds for it.
struct Scale {
  float s;
  bool fast;
  uint64_t ns2, r2;
};
__device__ __forceinline__ Scale scale_of(float amax) {
  Scale o;
  // 1 / 448 correctly rounded; outside these bounds the residuals may underflow or be NaN
  const float s = amax > 0x1p-90f && amax < INFINITY ? quotient(amax, 448.f, 1.f / 448.f) : __fdiv_rn(amax, 448.f);
  o.s = s < kMinScale ? kMinScale : s;   // a NaN stays
  o.fast = o.s >= 0x1p-80f && o.s < INFINITY;
  const float r = __frcp_rn(o.s);
  o.ns2 = pair64(-o.s, -o.s);
  o.r2 = pair64(r, r);
  return o;
}
// eight codes
template <int DT>
__device__ __forceinline__ uint2 codes(const In<DT>& in, const Scale& sc) {
  uint32_t c[4];
  if (sc.fast) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float a, b;
      in.pair(i, a, b);
      const uint64_t x = pair64(a, b);
      uint64_t q = mul_pair(x, sc.r2);
      q = fma_pair(fma_pair(q, sc.ns2, x), sc.r2, q);
      q = fma_pair(fma_pair(q, sc.ns2, x), sc.r2, q);
      asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(q));
      c[i] = f32x2_to_e4m3x2(a, b);
    }
    return make_uint2(c[0] | (c[1] << 16) | in.signs(0), c[2] | (c[3] << 16) | in.signs(1));
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float a, b;
      in.pair(i, a, b);
      c[i] = f32x2_to_e4m3x2(__fdiv_rn(a, sc.s), __fdiv_rn(b, sc.s));
    }
  }
  return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

// A scale per 128 columns of a row: eight lanes per block, each with eight
// elements of its first half and eight of its second, kUnroll blocks in
// flight per lane.
constexpr int kUnroll = 2;
template <int DT>
__global__ void __launch_bounds__(256)
quant_fp8_rows_kernel(const void* __restrict__ x, long ldx, long R, int K, int nkb, uint8_t* __restrict__ q,
                      float* __restrict__ scale) {
  const int l = threadIdx.x & 7;
  const long blocks = R * nkb, b0 = (((long)blockIdx.x * 256 + threadIdx.x) >> 3) * kUnroll;
  // one division for the first block's row, 32 bits wide where that holds it
  const long row0 = blocks <= 0xFFFFFFFFl ? (long)((uint32_t)b0 / (uint32_t)nkb) : b0 / nkb;
  long row[kUnroll];
  int col[kUnroll];
  In<DT> in[kUnroll][2];
  long r = row0;
  int kb = (int)(b0 - row0 * nkb);
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    row[u] = r;
    col[u] = kb * kBlk + 8 * l;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      in[u][h].zero();
      if (r < R && col[u] + 64 * h < K) in[u][h].load(x, (size_t)r * (size_t)ldx + col[u] + 64 * h);
    }
    if (++kb == nkb) {
      kb = 0;
      ++r;
    }
  }
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 2 * In<DT>::kVec; ++i) m = amax_word<DT>(m, in[u][i / In<DT>::kVec].v[i % In<DT>::kVec]);
#pragma unroll
    for (int d = 4; d >= 1; d >>= 1) m = amax_join<DT>(m, __shfl_xor_sync(0xffffffffu, m, d));
    const Scale sc = scale_of(amax_value<DT>(m));
    if (row[u] >= R) continue;
#pragma unroll
    for (int h = 0; h < 2; ++h)
      if (col[u] + 64 * h < K)
        *reinterpret_cast<uint2*>(q + (size_t)row[u] * K + col[u] + 64 * h) = codes<DT>(in[u][h], sc);
    if (l == 0) scale[b0 + u] = sc.s;
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
  for (int u = 0; u < 8; ++u)
#pragma unroll
    for (int i = 0; i < In<DT>::kVec; ++i) m = amax_word<DT>(m, in[u].v[i]);
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) m = amax_join<DT>(m, __shfl_xor_sync(0xffffffffu, m, d));
  if ((threadIdx.x & 31) == 0) wmax[threadIdx.x >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 8; ++w) m = amax_join<DT>(m, wmax[w]);
  const Scale sc = scale_of(amax_value<DT>(m));
  if (threadIdx.x == 0) scale[b] = sc.s;
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    if (r + 16 * u >= R || col >= K) continue;
    *reinterpret_cast<uint2*>(q + ((size_t)e * R + r + 16 * u) * (size_t)K + col) = codes<DT>(in[u], sc);
  }
}

template <int DT>
cudaError_t launch_dt(const void* x, long ldx, long lde, int E, int R, int K, int block_rows, uint8_t* q, float* scale,
                      cudaStream_t st) {
  const int nkb = (K + kBlk - 1) / kBlk;
  if (block_rows == 1) {
    const long per = 32 * kUnroll, blocks = (long)E * R * nkb;
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
