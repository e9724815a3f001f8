// gated.cu -- the gated activation on the 16-bit products' gate and up
// columns, with its input kept in 8 bits (MXFP8: E4M3 codes, one power of two
// per 32 columns), its backward pass from those, and the same 8 bits for any
// 16-bit activations.
//
//   SITU          h = [b tanh(g/b) sigmoid(g)] [bl tanh(u/bl)]
//   SWIGLU_BIAS   h = g sigmoid(a g) (u + c)
// With E0 = e^-g, E1 = e^(-2g/b), E2 = e^(-2u/bl) and d_i = 1 + E_i,
//   sigmoid(g) = 1/d0,  tanh(g/b) = (1 - E1)/d1,  its derivative by g times b = 4 E1/d1^2,
//   d/dg [b tanh(g/b) sigmoid(g)] = 1/d0 (4 E1/d1^2 + b tanh(g/b) E0/d0):
// no difference of nearly equal numbers, and one reciprocal, of d0 d1 d2, for
// all three.  Exponents are clamped at 25 (SWIGLU_BIAS: 80), where the factors
// are at their limits to 1.4e-11, so that the product stays finite; NaN passes.
//
// Bound by memory: per pair of gate and up, the forward reads 4 bytes and
// writes 2 (h) and 2 1/16 (the kept form); the backward reads 2 1/16 and 2 (dh)
// and writes 4 and, with h, 2 more.  Power-of-two scales make what is restored
// exact in 16 bits, so that the gradients' 16-bit products take it as it is.
//
// Four neighbouring lanes hold a block of 32 columns, eight each (16 bytes of a
// 16-bit type); a thread takes kRows rows, all loads first.
#include "../../include/situ_moe.h"
#include "situ_internal.h"

namespace situ {

namespace {

constexpr int kRows = 2;   // rows of a thread

struct GatedParams {
  const void* x;
  long ldx;
  const float *p0, *p1;
  const int32_t* offsets;
  int S, I, E;
  void* h;
  long ldh;
  uint8_t *q, *scale;
  const void* dh;
  long ld_dh;
  void* dx;
  long ld_dx;
};

template <int DT>
__device__ __forceinline__ uint32_t pack16(float a, float b) {
  return DT == SITU_DT_BF16 ? f32x2_to_bf16x2(a, b) : pack_f16x2(a, b);
}
template <int DT>
__device__ __forceinline__ void unpack16(uint32_t w, float& a, float& b) {
  a = DT == SITU_DT_BF16 ? bf16_lo(w) : f16_to_f32(w & 0xFFFFu);
  b = DT == SITU_DT_BF16 ? bf16_hi(w) : f16_to_f32(w >> 16);
}
template <int DT>
__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
  unpack16<DT>(v.x, f[0], f[1]);
  unpack16<DT>(v.y, f[2], f[3]);
  unpack16<DT>(v.z, f[4], f[5]);
  unpack16<DT>(v.w, f[6], f[7]);
}
template <int DT>
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack16<DT>(f[0], f[1]), pack16<DT>(f[2], f[3]), pack16<DT>(f[4], f[5]), pack16<DT>(f[6], f[7]));
}

__device__ __forceinline__ uint4 ld16(const void* p, size_t el) {
  return __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + el));
}
__device__ __forceinline__ void st16(void* p, size_t el, const uint4& v) {
  *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + el) = v;
}

// The expert whose rows hold row r: -1 for none.
__device__ __forceinline__ int expert_of(const int32_t* offsets, int E, int r) {
  if (!offsets) return 0;
  int lo = 0, hi = E + 1;             // the first entry beyond r lies in [lo, hi]
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(offsets + mid) > r) hi = mid;
    else lo = mid + 1;
  }
  return lo <= E ? lo - 1 : -1;       // 0: before the first expert's rows
}

// Eight elements of a block of 32 to codes, and the block's scale byte.  The
// magnitudes' bit patterns are ordered as the values are, infinity and NaN
// above all.
template <int DT>
__device__ __forceinline__ uint2 save8(const uint4& v, const float (&f)[8], uint32_t& byte) {
  constexpr uint32_t kM = 0x7FFF7FFFu, kInf = DT == SITU_DT_BF16 ? 0x7F80u : 0x7C00u;
  uint32_t m = __vmaxu2(__vmaxu2(v.x & kM, v.y & kM), __vmaxu2(v.z & kM, v.w & kM));
  m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 1));
  m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 2));
  m = max(m & 0xFFFFu, m >> 16);
  const int e = mxfp8_exponent(DT == SITU_DT_BF16 ? __uint_as_float(m << 16) : f16_to_f32(m));
  byte = (uint32_t)(e + 127);
  if (m >= kInf) {
    byte = 255u;
    return make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu);
  }
  const float s = __uint_as_float((uint32_t)(127 - e) << 23);   // e in [-127, 120]
  return make_uint2(f32x2_to_e4m3x2(f[0] * s, f[1] * s) | (f32x2_to_e4m3x2(f[2] * s, f[3] * s) << 16),
                    f32x2_to_e4m3x2(f[4] * s, f[5] * s) | (f32x2_to_e4m3x2(f[6] * s, f[7] * s) << 16));
}

__device__ __forceinline__ float scale_value(uint32_t b) {
  return __uint_as_float(b == 0 ? 0x00400000u : b == 255 ? 0x7FC00000u : b << 23);
}
__device__ __forceinline__ void restore8(const uint2& q, float s, float (&f)[8]) {
  e4m3x2_to_f32x2(q.x & 0xFFFFu, f[0], f[1]);
  e4m3x2_to_f32x2(q.x >> 16, f[2], f[3]);
  e4m3x2_to_f32x2(q.y & 0xFFFFu, f[4], f[5]);
  e4m3x2_to_f32x2(q.y >> 16, f[6], f[7]);
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] *= s;
}

__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float rcp_approx(float a) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(a));
  return r;
}
__device__ __forceinline__ float exp25(float z) { return exp2_approx(min_nan(z, 25.f * kLog2e)); }

// The activation of one row's expert and its derivatives.
template <int ACT>
struct Act {
  float b, bl, k0, k1;   // SITU: caps and -2 log2(e) / cap, 0 without one; SWIGLU_BIAS: b = a, bl = c
  __device__ __forceinline__ Act(float p0, float p1) : b(p0), bl(p1), k0(0.f), k1(0.f) {
    if (ACT == SITU_ACT_FN_SITU) {
      k0 = situ_cap_k(p0);
      k1 = situ_cap_k(p1);
    }
  }
  __device__ __forceinline__ float swiglu_exp(float g) const {
    return exp2_approx(max_nan(min_nan(-kLog2e * b * g, 80.f * kLog2e), -80.f * kLog2e));
  }
  __device__ __forceinline__ float value(float g, float u) const {
    if (ACT == SITU_ACT_FN_SWIGLU_BIAS) return g * (u + bl) * rcp_approx(1.f + swiglu_exp(g));
    const float e0 = exp25(-kLog2e * g), e1 = exp25(k0 * g), e2 = exp25(k1 * u);
    const float ng = k0 < 0.f ? b * (1.f - e1) : g, dg = k0 < 0.f ? 1.f + e1 : 1.f;
    const float nu = k1 < 0.f ? bl * (1.f - e2) : u, du = k1 < 0.f ? 1.f + e2 : 1.f;
    return ng * nu * rcp_approx((1.f + e0) * dg * du);
  }
  // h and its derivatives by g and u
  __device__ __forceinline__ float all(float g, float u, float& hg, float& hu) const {
    if (ACT == SITU_ACT_FN_SWIGLU_BIAS) {
      const float e0 = swiglu_exp(g), s = rcp_approx(1.f + e0), up = u + bl;
      hu = g * s;
      hg = s * fmaf(b * hu, e0, 1.f) * up;
      return hu * up;
    }
    const float e0 = exp25(-kLog2e * g), e1 = exp25(k0 * g), e2 = exp25(k1 * u);
    const float d0 = 1.f + e0, d1 = 1.f + e1, d2 = 1.f + e2;
    const float d12 = d1 * d2, r = rcp_approx(d0 * d12);
    const float r0 = r * d12, r12 = r * d0, r1 = r12 * d2, r2 = r12 * d1;
    const float t = k0 < 0.f ? b * (1.f - e1) * r1 : g, dt = k0 < 0.f ? 4.f * e1 * r1 * r1 : 1.f;
    const float up = k1 < 0.f ? bl * (1.f - e2) * r2 : u, dup = k1 < 0.f ? 4.f * e2 * r2 * r2 : 1.f;
    const float gate = t * r0;
    hg = r0 * fmaf(gate, e0, dt) * up;
    hu = gate * dup;
    return gate * up;
  }
};

// A thread's place: columns c .. c + 7 of rows row0 + blockDim.y j.
struct Place {
  int c;
  long row0;
  __device__ __forceinline__ Place()
      : c((int)(blockIdx.y * blockDim.x + threadIdx.x) * 8),
        row0((long)blockIdx.x * blockDim.y * kRows + threadIdx.y) {}
  __device__ __forceinline__ long row(int j) const { return row0 + (long)j * blockDim.y; }
};

template <int DT, int ACT, bool SAVE>
__global__ void __launch_bounds__(512)
gated_kernel(GatedParams p) {
  const Place at;
  const int nb = (p.I + 31) / 32;
  uint4 g[kRows], u[kRows];
  int e[kRows];
#pragma unroll
  for (int j = 0; j < kRows; ++j) {
    const long r = at.row(j);
    g[j] = u[j] = make_uint4(0, 0, 0, 0);
    e[j] = -1;
    if (r < p.S && at.c < p.I) {
      e[j] = expert_of(p.offsets, p.E, (int)r);
      if (e[j] >= 0) {
        g[j] = ld16(p.x, (size_t)r * p.ldx + at.c);
        u[j] = ld16(p.x, (size_t)r * p.ldx + p.I + at.c);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < kRows; ++j) {
    const long r = at.row(j);
    const bool have = r < p.S && at.c < p.I;
    float fg[8], fu[8];
    unpack8<DT>(g[j], fg);
    unpack8<DT>(u[j], fu);
    if (SAVE) {
      uint32_t bg, bu;
      const uint2 qg = save8<DT>(g[j], fg, bg), qu = save8<DT>(u[j], fu, bu);
      if (have) {
        uint8_t* q = p.q + (size_t)r * 2 * p.I + at.c;
        *reinterpret_cast<uint2*>(q) = qg;
        *reinterpret_cast<uint2*>(q + p.I) = qu;
        if ((threadIdx.x & 3) == 0) {
          uint8_t* s = p.scale + (size_t)r * 2 * nb + at.c / 32;
          s[0] = (uint8_t)bg;
          s[nb] = (uint8_t)bu;
        }
      }
    }
    if (!have) continue;
    float h[8];
    if (e[j] >= 0) {
      const Act<ACT> act(__ldg(p.p0 + e[j]), __ldg(p.p1 + e[j]));
#pragma unroll
      for (int i = 0; i < 8; ++i) h[i] = act.value(fg[i], fu[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) h[i] = 0.f;
    }
    st16(p.h, (size_t)r * p.ldh + at.c, pack8<DT>(h));
  }
}

template <int DT, int ACT, bool H>
__global__ void __launch_bounds__(512)
gated_back_kernel(GatedParams p) {
  const Place at;
  const int nb = (p.I + 31) / 32;
  if (at.c >= p.I) return;
  uint2 qg[kRows], qu[kRows];
  uint32_t bg[kRows], bu[kRows];
  uint4 dh[kRows];
  int e[kRows];
#pragma unroll
  for (int j = 0; j < kRows; ++j) {
    const long r = at.row(j);
    e[j] = r < p.S ? expert_of(p.offsets, p.E, (int)r) : -1;
    if (e[j] < 0) continue;
    const uint8_t* q = p.q + (size_t)r * 2 * p.I + at.c;
    const uint8_t* s = p.scale + (size_t)r * 2 * nb + at.c / 32;
    qg[j] = __ldg(reinterpret_cast<const uint2*>(q));
    qu[j] = __ldg(reinterpret_cast<const uint2*>(q + p.I));
    bg[j] = __ldg(s);
    bu[j] = __ldg(s + nb);
    dh[j] = ld16(p.dh, (size_t)r * p.ld_dh + at.c);
  }
#pragma unroll
  for (int j = 0; j < kRows; ++j) {
    const long r = at.row(j);
    if (r >= p.S) continue;
    uint4 og = make_uint4(0, 0, 0, 0), ou = og, oh = og;
    if (e[j] >= 0) {
      float fg[8], fu[8], d[8], h[8];
      restore8(qg[j], scale_value(bg[j]), fg);
      restore8(qu[j], scale_value(bu[j]), fu);
      unpack8<DT>(dh[j], d);
      const Act<ACT> act(__ldg(p.p0 + e[j]), __ldg(p.p1 + e[j]));
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float hg, hu;
        h[i] = act.all(fg[i], fu[i], hg, hu);
        fg[i] = d[i] * hg;
        fu[i] = d[i] * hu;
      }
      og = pack8<DT>(fg);
      ou = pack8<DT>(fu);
      if (H) oh = pack8<DT>(h);
    }
    st16(p.dx, (size_t)r * p.ld_dx + at.c, og);
    st16(p.dx, (size_t)r * p.ld_dx + p.I + at.c, ou);
    if (H) st16(p.h, (size_t)r * p.ldh + at.c, oh);
  }
}

template <int DT>
__global__ void __launch_bounds__(512)
save_kernel(const void* x, long ldx, int S, int K, uint8_t* q, uint8_t* scale) {
  const Place at;
  uint4 v[kRows];
#pragma unroll
  for (int j = 0; j < kRows; ++j)
    v[j] = at.row(j) < S && at.c < K ? ld16(x, (size_t)at.row(j) * ldx + at.c) : make_uint4(0, 0, 0, 0);
#pragma unroll
  for (int j = 0; j < kRows; ++j) {
    float f[8];
    unpack8<DT>(v[j], f);
    uint32_t b;
    const uint2 c = save8<DT>(v[j], f, b);
    if (at.row(j) >= S || at.c >= K) continue;
    *reinterpret_cast<uint2*>(q + (size_t)at.row(j) * K + at.c) = c;
    if ((threadIdx.x & 3) == 0) scale[(size_t)at.row(j) * ((K + 31) / 32) + at.c / 32] = (uint8_t)b;
  }
}

// Values past a 16-bit type's range become its largest.
template <int DT>
__global__ void __launch_bounds__(512)
restore_kernel(const uint8_t* q, const uint8_t* scale, int S, int K, void* x, long ldx) {
  const Place at;
  if (at.c >= K) return;
  constexpr float kMost = DT == SITU_DT_BF16 ? 3.38953139e38f : 65504.f;
  uint2 c[kRows];
  uint32_t b[kRows];
#pragma unroll
  for (int j = 0; j < kRows; ++j)
    if (at.row(j) < S) {
      c[j] = __ldg(reinterpret_cast<const uint2*>(q + (size_t)at.row(j) * K + at.c));
      b[j] = __ldg(scale + (size_t)at.row(j) * ((K + 31) / 32) + at.c / 32);
    }
#pragma unroll
  for (int j = 0; j < kRows; ++j) {
    if (at.row(j) >= S) continue;
    float f[8];
    restore8(c[j], scale_value(b[j]), f);
    const size_t el = (size_t)at.row(j) * ldx + at.c;
    if (DT == SITU_DT_F32) {
      float4* o = reinterpret_cast<float4*>(static_cast<float*>(x) + el);
      o[0] = make_float4(f[0], f[1], f[2], f[3]);
      o[1] = make_float4(f[4], f[5], f[6], f[7]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = max_nan(min_nan(f[i], kMost), -kMost);
      st16(x, el, pack8<DT>(f));
    }
  }
}

// A block's threads: x over 8-column pieces of a row (a multiple of four, so
// that a block of 32 columns never parts), y over rows, whole warps in all.
struct Shape {
  dim3 grid, block;
};
Shape shape_of(int S, int K) {
  const int pieces = (K + 31) / 32 * 4;
  int x, y, parts = 1;
  if (pieces <= 64) {
    x = pieces;
    y = 8;
  } else {
    parts = (pieces + 255) / 256;
    x = ((pieces + parts - 1) / parts + 31) / 32 * 32;
    y = x > 128 ? 1 : 2;
  }
  const long per = (long)y * kRows;
  return {dim3((unsigned)((S + per - 1) / per), (unsigned)parts), dim3((unsigned)x, (unsigned)y)};
}

bool bad(const void* q, uintptr_t mask) { return (reinterpret_cast<uintptr_t>(q) & mask) != 0; }
bool bad_ld(int64_t ld, int64_t cols, int64_t unit) { return ld < cols || ld % unit != 0 || ld > (int64_t)1 << 39; }
bool bad_rows(int S, int K) { return S < 0 || S > SITU_GEMM_MAX_ROWS || K < 8 || K % 8 != 0 || K > SITU_GEMM_MAX_DIM; }

situ_status done() { return cudaGetLastError() == cudaSuccess ? SITU_OK : SITU_ERR_CUDA; }

situ_status check_gated(const situ_gated_args* a) {
  if ((a->dtype != SITU_DT_BF16 && a->dtype != SITU_DT_F16) ||
      (a->activation != SITU_ACT_FN_SITU && a->activation != SITU_ACT_FN_SWIGLU_BIAS))
    return SITU_ERR_UNSUPPORTED;
  if (bad_rows(a->S, a->I) || a->E < 1 || a->E > SITU_MAX_LOCAL_EXPERTS || (!a->offsets && a->E != 1))
    return SITU_ERR_BAD_SHAPE;
  return SITU_OK;
}

GatedParams params_of(const situ_gated_args* a) {
  GatedParams p;
  p.x = a->gate_up;
  p.ldx = (long)a->ld_gate_up;
  p.p0 = a->p0;
  p.p1 = a->p1;
  p.offsets = a->offsets;
  p.S = a->S;
  p.I = a->I;
  p.E = a->E;
  p.h = a->h;
  p.ldh = (long)a->ldh;
  p.q = a->q;
  p.scale = a->scale;
  p.dh = a->dh;
  p.ld_dh = (long)a->ld_dh;
  p.dx = a->dgate_up;
  p.ld_dx = (long)a->ld_dgate_up;
  return p;
}

}  // namespace
}  // namespace situ

extern "C" situ_status situ_moe_gated(const situ_gated_args* a, void* stream) {
  using namespace situ;
  if (!a) return SITU_ERR_NULL_ARG;
  const situ_status s = check_gated(a);
  if (s != SITU_OK) return s;
  if (bad_ld(a->ld_gate_up, 2 * (int64_t)a->I, 8) || bad_ld(a->ldh, a->I, 8)) return SITU_ERR_BAD_SHAPE;
  if (a->S == 0) return SITU_OK;
  if (!a->gate_up || !a->p0 || !a->p1 || !a->h || !a->q != !a->scale) return SITU_ERR_NULL_ARG;
  if (bad(a->gate_up, 15) || bad(a->h, 15) || bad(a->q, 7) || bad(a->p0, 3) || bad(a->p1, 3) || bad(a->offsets, 3))
    return SITU_ERR_MISALIGNED;
  const GatedParams p = params_of(a);
  const Shape sh = shape_of(a->S, a->I);
  cudaStream_t st = (cudaStream_t)stream;
  auto launch = [&](auto k) { k<<<sh.grid, sh.block, 0, st>>>(p); };
  auto by_save = [&](auto yes, auto no) { a->q ? launch(yes) : launch(no); };
  constexpr int kS = SITU_ACT_FN_SITU, kW = SITU_ACT_FN_SWIGLU_BIAS, kB = SITU_DT_BF16, kF = SITU_DT_F16;
  if (a->dtype == kB)
    a->activation == kS ? by_save(gated_kernel<kB, kS, true>, gated_kernel<kB, kS, false>)
                        : by_save(gated_kernel<kB, kW, true>, gated_kernel<kB, kW, false>);
  else
    a->activation == kS ? by_save(gated_kernel<kF, kS, true>, gated_kernel<kF, kS, false>)
                        : by_save(gated_kernel<kF, kW, true>, gated_kernel<kF, kW, false>);
  return done();
}

extern "C" situ_status situ_moe_gated_backward(const situ_gated_args* a, void* stream) {
  using namespace situ;
  if (!a) return SITU_ERR_NULL_ARG;
  const situ_status s = check_gated(a);
  if (s != SITU_OK) return s;
  if (bad_ld(a->ld_dh, a->I, 8) || bad_ld(a->ld_dgate_up, 2 * (int64_t)a->I, 8) || (a->h && bad_ld(a->ldh, a->I, 8)))
    return SITU_ERR_BAD_SHAPE;
  if (a->S == 0) return SITU_OK;
  if (!a->q || !a->scale || !a->p0 || !a->p1 || !a->dh || !a->dgate_up) return SITU_ERR_NULL_ARG;
  if (bad(a->dh, 15) || bad(a->dgate_up, 15) || bad(a->h, 15) || bad(a->q, 7) || bad(a->p0, 3) || bad(a->p1, 3) ||
      bad(a->offsets, 3))
    return SITU_ERR_MISALIGNED;
  const GatedParams p = params_of(a);
  const Shape sh = shape_of(a->S, a->I);
  cudaStream_t st = (cudaStream_t)stream;
  auto launch = [&](auto k) { k<<<sh.grid, sh.block, 0, st>>>(p); };
  auto by_h = [&](auto yes, auto no) { a->h ? launch(yes) : launch(no); };
  constexpr int kS = SITU_ACT_FN_SITU, kW = SITU_ACT_FN_SWIGLU_BIAS, kB = SITU_DT_BF16, kF = SITU_DT_F16;
  if (a->dtype == kB)
    a->activation == kS ? by_h(gated_back_kernel<kB, kS, true>, gated_back_kernel<kB, kS, false>)
                        : by_h(gated_back_kernel<kB, kW, true>, gated_back_kernel<kB, kW, false>);
  else
    a->activation == kS ? by_h(gated_back_kernel<kF, kS, true>, gated_back_kernel<kF, kS, false>)
                        : by_h(gated_back_kernel<kF, kW, true>, gated_back_kernel<kF, kW, false>);
  return done();
}

extern "C" situ_status situ_moe_save_mxfp8(const void* x, int32_t dtype, int32_t S, int32_t K, int64_t ldx, uint8_t* q,
                                           uint8_t* scale, void* stream) {
  using namespace situ;
  if (dtype != SITU_DT_BF16 && dtype != SITU_DT_F16) return SITU_ERR_UNSUPPORTED;
  if (bad_rows(S, K) || bad_ld(ldx, K, 8)) return SITU_ERR_BAD_SHAPE;
  if (S == 0) return SITU_OK;
  if (!x || !q || !scale) return SITU_ERR_NULL_ARG;
  if (bad(x, 15) || bad(q, 7)) return SITU_ERR_MISALIGNED;
  const Shape sh = shape_of(S, K);
  auto launch = [&](auto k) { k<<<sh.grid, sh.block, 0, (cudaStream_t)stream>>>(x, (long)ldx, S, K, q, scale); };
  dtype == SITU_DT_BF16 ? launch(save_kernel<SITU_DT_BF16>) : launch(save_kernel<SITU_DT_F16>);
  return done();
}

extern "C" situ_status situ_moe_restore_mxfp8(const uint8_t* q, const uint8_t* scale, int32_t dtype, int32_t S, int32_t K,
                                              void* x, int64_t ldx, void* stream) {
  using namespace situ;
  if (dtype != SITU_DT_BF16 && dtype != SITU_DT_F16 && dtype != SITU_DT_F32) return SITU_ERR_UNSUPPORTED;
  if (bad_rows(S, K) || bad_ld(ldx, K, dtype == SITU_DT_F32 ? 4 : 8)) return SITU_ERR_BAD_SHAPE;
  if (S == 0) return SITU_OK;
  if (!x || !q || !scale) return SITU_ERR_NULL_ARG;
  if (bad(x, 15) || bad(q, 7)) return SITU_ERR_MISALIGNED;
  const Shape sh = shape_of(S, K);
  auto launch = [&](auto k) { k<<<sh.grid, sh.block, 0, (cudaStream_t)stream>>>(q, scale, S, K, x, (long)ldx); };
  dtype == SITU_DT_BF16 ? launch(restore_kernel<SITU_DT_BF16>)
                        : dtype == SITU_DT_F16 ? launch(restore_kernel<SITU_DT_F16>) : launch(restore_kernel<SITU_DT_F32>);
  return done();
}
