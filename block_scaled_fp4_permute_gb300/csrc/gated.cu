// gated.cu -- the gated activation on the 16-bit products' gate and up
// columns, with its input kept in 8 bits (MXFP8: E4M3 codes, one power of two
// per 32 columns), its backward pass from those, and the same 8 bits for any
// 16-bit activations.
//
//   SITU          h = [b tanh(g/b) sigmoid(g)] [bl tanh(u/bl)]
//   SWIGLU_BIAS   h = g sigmoid(a g) (u + c)
// With E0 = e^-g, E1 = e^(-2g/b), E2 = e^(-2u/bl) and d_i = 1 + E_i,
//   sigmoid(g) = 1/d0,  tanh(g/b) = (1 - E1)/d1,  its derivative by g times b = 4 E1/d1^2,
//   d/dg [b tanh(g/b) sigmoid(g)] = 1/d0 (4 E1/d1^2 + b tanh(g/b) E0/d0)
// and one reciprocal, of d0 d1 d2, for all three.  1 - E1 is a difference of nearly
// equal numbers where g is small beside b.  So the factor is g tanh(y)/y with
// y = max(|g/b|, 2^-7.5): tanh(y)/y is off by y^2/3 < 2^-16.5 below that, and the
// difference by 2^-15.5 at most above (its derivative's 1 - tanh^2 by 2^-15).  A result
// is rounded once, whatever the cap.
// Where the product could overflow, each factor has a reciprocal of its own: E1 and E2
// are taken of magnitudes, and a sigmoid below 2^-126 is zero.  NaN passes.
//
// Bound by memory: per pair of gate and up, the forward reads 4 bytes and
// writes 2 (h) and 2 1/16 (the kept form); the backward reads 2 1/16 and 2 (dh)
// and writes 4 and, with h, 2 more.  Power-of-two scales make what is restored
// exact in 16 bits, so that the gradients' 16-bit products take it as it is.
// Measured (bf16, 32,768 rows of 2,048, 32 experts): forward 101 us (5.4 TB/s),
// backward 123 (5.5), held by issue slots as much as by memory (with the factors as
// they stand above, 91 and 115; SWIGLU_BIAS 83 and 109).
//
// Two neighbouring lanes hold a block of 32 columns, 16 each: the row's expert
// and its constants are then a small part of a thread's work (with eight columns
// a lane they were a third of it).  A lane's columns are every other eight, so
// that each store instruction of a pair fills a 32-byte sector; codes change
// hands first, to go in 16 bytes.
#include "../../include/situ_moe.h"
#include "situ_internal.h"

namespace situ {

namespace {

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
  int wide;   // codes of 16 columns are 16-byte aligned
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
// pairs of fp32: one instruction, and one issue slot, for two operations
struct F2 {
  uint64_t v;
};
__device__ __forceinline__ F2 f2(float a, float b) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ F2 f2(float a) { return f2(a, a); }
__device__ __forceinline__ float2 both(F2 a) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a.v));
  return r;
}
__device__ __forceinline__ F2 operator*(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 operator+(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 operator-(F2 a, F2 b) {
  F2 r;
  asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
__device__ __forceinline__ F2 exp2_pair(F2 z) {
  const float2 a = both(z);
  return f2(exp2_approx(a.x), exp2_approx(a.y));
}
__device__ __forceinline__ F2 rcp_pair(F2 z) {
  const float2 a = both(z);
  return f2(rcp_approx(a.x), rcp_approx(a.y));
}

// The expert whose rows hold row r: -1 for none.  `together`: the warp's lanes
// ask for one row.
__device__ __forceinline__ int expert_of(const int32_t* offsets, int E, int r, bool together) {
  if (!offsets) return 0;
  int lo = 0, n = E + 1;              // the first entry beyond r lies in [lo, lo + n]
  if (together) {
    while (n > 0) {                   // a 32nd of what is left each time
      const int step = (n + 31) >> 5, at = lo + (int)(threadIdx.x & 31) * step;
      const int below = __popc(__ballot_sync(0xffffffffu, at < lo + n && __ldg(offsets + at) <= r));
      if (below == 0) break;
      const int from = lo + (below - 1) * step + 1;
      n = min(step - 1, lo + n - from);
      lo = from;
    }
  } else {
    while (n > 0) {
      const int half = n >> 1;
      if (__ldg(offsets + lo + half) <= r) {
        lo += half + 1;
        n -= half + 1;
      } else {
        n = half;
      }
    }
  }
  return lo <= E ? lo - 1 : -1;       // 0: before the first expert's rows
}

// A lane's 16 columns of a row: eight, and the eight 16 further.
struct Line {
  uint4 v[2];
};
__device__ __forceinline__ Line load_line(const void* p, size_t el, bool first, bool second) {
  Line l;
  l.v[0] = first ? ld16(p, el) : make_uint4(0, 0, 0, 0);
  l.v[1] = second ? ld16(p, el + 16) : make_uint4(0, 0, 0, 0);
  return l;
}
__device__ __forceinline__ void store_line(void* p, size_t el, const uint4 (&v)[2], bool first, bool second) {
  if (first) st16(p, el, v[0]);
  if (second) st16(p, el + 16, v[1]);
}
// their codes
__device__ __forceinline__ uint4 load_codes(const uint8_t* q, bool first, bool second) {
  const uint2 a = first ? __ldg(reinterpret_cast<const uint2*>(q)) : make_uint2(0, 0);
  const uint2 b = second ? __ldg(reinterpret_cast<const uint2*>(q + 16)) : make_uint2(0, 0);
  return make_uint4(a.x, a.y, b.x, b.y);
}
// wide (the same for both lanes of a pair): the block is whole and 16-byte
// aligned; by whole warps
__device__ __forceinline__ void store_codes(uint8_t* q, const uint4& c, bool first, bool second, bool wide) {
  const bool odd = threadIdx.x & 1;
  const uint32_t x = __shfl_xor_sync(0xffffffffu, odd ? c.x : c.z, 1), y = __shfl_xor_sync(0xffffffffu, odd ? c.y : c.w, 1);
  if (wide) {
    if (first) *reinterpret_cast<uint4*>(q + (odd ? 8 : 0)) = odd ? make_uint4(x, y, c.z, c.w) : make_uint4(c.x, c.y, x, y);
    return;
  }
  if (first) *reinterpret_cast<uint2*>(q) = make_uint2(c.x, c.y);
  if (second) *reinterpret_cast<uint2*>(q + 16) = make_uint2(c.z, c.w);
}
// the largest magnitude of 16 codes, whose bits are ordered as the values are
__device__ __forceinline__ float amax_code(const uint4& c) {
  constexpr uint32_t kM = 0x007F007Fu;
  uint32_t m = __vmaxu2(__vmaxu2(c.x & kM, c.y & kM), __vmaxu2(c.z & kM, c.w & kM));
  m = __vmaxu2(m, __vmaxu2(__vmaxu2((c.x >> 8) & kM, (c.y >> 8) & kM), __vmaxu2((c.z >> 8) & kM, (c.w >> 8) & kM)));
  return e4m3_code_to_f32(max(m & 0xFFFFu, m >> 16));
}

// The larger magnitudes of two pairs, under signs that say nothing; NaN if either
// is.
template <int DT>
__device__ __forceinline__ uint32_t max_mag(uint32_t a, uint32_t b) {
  uint32_t r;
  if (DT == SITU_DT_BF16) asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  else asm("max.NaN.xorsign.abs.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// The largest of 16 magnitudes, two at a time (a NaN's bits are above an
// infinity's), and as a value.
template <int DT>
__device__ __forceinline__ uint32_t amax_bits(const Line& l) {
  const uint32_t a = max_mag<DT>(max_mag<DT>(l.v[0].x, l.v[0].y), max_mag<DT>(l.v[0].z, l.v[0].w));
  const uint32_t b = max_mag<DT>(max_mag<DT>(l.v[1].x, l.v[1].y), max_mag<DT>(l.v[1].z, l.v[1].w));
  return max_mag<DT>(a, b) & 0x7FFF7FFFu;
}
template <int DT>
__device__ __forceinline__ float amax_value(uint32_t m) {
  m = max(m & 0xFFFFu, m >> 16);
  return DT == SITU_DT_BF16 ? __uint_as_float(m << 16) : f16_to_f32(m);
}

// A block's scale byte, from its lanes' maxima, and what its elements are
// multiplied by: NaN for a block with an infinity or a NaN, so that every code is
// one.
struct Kept {
  uint32_t byte;
  float factor;
};
template <int DT>
__device__ __forceinline__ Kept kept_of(uint32_t m) {
  constexpr uint32_t kInf = DT == SITU_DT_BF16 ? 0x7F80u : 0x7C00u;
  m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 1));
  const int e = mxfp8_exponent(amax_value<DT>(m));              // in [-127, 120]
  const bool lost = max(m & 0xFFFFu, m >> 16) >= kInf;
  return {lost ? 255u : (uint32_t)(e + 127), lost ? __uint_as_float(0x7FFFFFFFu) : __uint_as_float((uint32_t)(127 - e) << 23)};
}
__device__ __forceinline__ uint2 save8(const float (&f)[8], float s, bool lost) {
  const F2 t = f2(s);
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 v = both(f2(f[2 * i], f[2 * i + 1]) * t);
    c[i] = f32x2_to_e4m3x2(v.x, v.y);
  }
  if (lost) return make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu);        // whatever the NaNs' signs
  return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

__device__ __forceinline__ float scale_value(uint32_t b) {
  return __uint_as_float(b == 0 ? 0x00400000u : b == 255 ? 0x7FC00000u : b << 23);
}
__device__ __forceinline__ void restore8(uint32_t lo, uint32_t hi, float s, float (&f)[8]) {
  e4m3x2_to_f32x2(lo & 0xFFFFu, f[0], f[1]);
  e4m3x2_to_f32x2(lo >> 16, f[2], f[3]);
  e4m3x2_to_f32x2(hi & 0xFFFFu, f[4], f[5]);
  e4m3x2_to_f32x2(hi >> 16, f[6], f[7]);
  const F2 t = f2(s);
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    const float2 v = both(f2(f[i], f[i + 1]) * t);
    f[i] = v.x;
    f[i + 1] = v.y;
  }
}

constexpr float kSmall = 1.f / 181;      // 2^-7.5 of a cap, below which its factor counts as the argument

// b tanh(x / b) and its derivative; k = -2 log2(e) / b, 0 without a cap
struct Tanh {
  float t, dt;
  __device__ __forceinline__ Tanh(float x, float b, float k) : t(x), dt(1.f) {
    if (k < 0.f) {
      const float e = exp2_approx(-fabsf(k * x)), r = rcp_approx(1.f + e);
      if (!(fabsf(x) < kSmall * b)) t = copysignf(b * (1.f - e) * r, x);
      dt = 4.f * e * r * r;
    }
  }
};
// sigmoid(v) and, from v brought into where that is no subnormal, sigmoid(-v)
__device__ __forceinline__ float sigmoid(float v) { return rcp_approx(1.f + exp2_approx(-kLog2e * v)); }
struct Sigmoid {
  float v, s, c;
  __device__ __forceinline__ explicit Sigmoid(float a) {
    constexpr float kMost = 87.f;
    v = max_nan(min_nan(a, kMost), -kMost);
    const float e = exp2_approx(-kLog2e * v), r = rcp_approx(1.f + e);
    s = a < -kMost ? 0.f : r;
    c = e * r;
  }
};

// The activation of one row's expert and its derivatives.
template <int ACT>
struct Act {
  float b, bl, k0, k1;   // SITU: caps and -2 log2(e) / cap, 0 without one; SWIGLU_BIAS: b = a, bl = c
  __device__ __forceinline__ Act(float p0, float p1) : b(p0), bl(p1), k0(0.f), k1(0.f) {
    if (ACT == SITU_ACT_FN_SITU) {
      constexpr float kLeast = -3e38f;         // finite beside caps below fp32's normal numbers
      k0 = p0 > 0.f ? fmaxf(-2.f * kLog2e * rcp_approx(p0), kLeast) : 0.f;
      k1 = p1 > 0.f ? fmaxf(-2.f * kLog2e * rcp_approx(p1), kLeast) : 0.f;
    }
  }
  __device__ __forceinline__ float value(float g, float u) const {
    if (ACT == SITU_ACT_FN_SWIGLU_BIAS) return g * sigmoid(b * g) * (u + bl);
    return Tanh(g, b, k0).t * sigmoid(g) * Tanh(u, bl, k1).t;
  }
  // h and its derivatives by g and u
  __device__ __forceinline__ float all(float g, float u, float& hg, float& hu) const {
    if (ACT == SITU_ACT_FN_SWIGLU_BIAS) {
      const float up = u + bl;
      const Sigmoid s(b * g);
      hu = g * s.s;
      hg = s.s * fmaf(s.v, s.c, 1.f) * up;
      return hu * up;
    }
    const Tanh t(g, b, k0), up(u, bl, k1);
    const Sigmoid s(g);
    const float gate = t.t * s.s;
    hg = s.s * fmaf(t.t, s.c, t.dt) * up.t;
    hu = gate * up.dt;
    return gate * up.t;
  }
};

// SITU with both caps, on pairs, where no exponential or product of them can
// overflow: the exponents' sum is below 120 for the thread's largest gate and up (so
// there is no NaN or infinity among them).  One at a time the kernels
// were bound by issue slots (52 instructions a pair: forward 141 us).
struct Situ2 {
  F2 k, k0, k1;
  float most_g, most_u;   // exponents per unit of |g| and |u|
  bool capped;
  __device__ __forceinline__ explicit Situ2(const Act<SITU_ACT_FN_SITU>& a)
      : k(f2(-kLog2e)), k0(f2(a.k0)), k1(f2(a.k1)),
        most_g(kLog2e - a.k0), most_u(-a.k1), capped(a.k0 < 0.f && a.k1 < 0.f) {}
  __device__ __forceinline__ bool fits(float amax_g, float amax_u) const {
    return capped && amax_g * most_g + amax_u * most_u < 120.f;   // false for NaN
  }
  // cap tanh(x / cap) = x (1 - E) / (y (1 + E)), y = max(|x / cap|, kSmall), E = e^-2y: z = -2 y log2(e) takes y's
  // place, with the constants that leaves in the sigmoid's denominator
  __device__ __forceinline__ F2 value(F2 g, F2 u) const {
    const F2 one = f2(1.f), c = f2(0.25f / (kLog2e * kLog2e)), z1 = away(g * k0), z2 = away(u * k1);
    const F2 e0 = exp2_pair(g * k), e1 = exp2_pair(z1), e2 = exp2_pair(z2);
    return (g * (one - e1)) * (u * (one - e2)) * rcp_pair(fma2(e0, c, c) * fma2(e1, z1, z1) * fma2(e2, z2, z2));
  }
  static __device__ __forceinline__ F2 away(F2 z) {
    const float2 a = both(z);
    constexpr float kMost = -2.f * kLog2e * kSmall;
    return f2(fminf(-fabsf(a.x), kMost), fminf(-fabsf(a.y), kMost));
  }
  // h, and its derivatives by g and, a 16th of it, by u: gate is a quarter here, up four times
  __device__ __forceinline__ F2 all(F2 g, F2 u, F2& hg, F2& hu16) const {
    constexpr float kC = -2.f * kLog2e;      // z / y
    const F2 one = f2(1.f), z1 = away(g * k0), z2 = away(u * k1);
    const F2 e0 = exp2_pair(g * k), e1 = exp2_pair(z1), e2 = exp2_pair(z2);
    const F2 d0 = e0 + one, d1 = fma2(e1, z1, z1), d2 = fma2(e2, z2, z2), d12 = d1 * d2, r = rcp_pair(d0 * d12);
    const F2 r0 = r * d12, r12 = r * d0, r1 = r12 * d2, r2 = r12 * d1, q1 = z1 * r1, q2 = z2 * r2;
    const F2 dt = (e1 * q1) * q1, dup = (e2 * q2) * q2;   // a quarter each
    const F2 gate = (g * fma2(e1, f2(-.25f * kC), f2(.25f * kC))) * r1 * r0, up = (u * fma2(e2, f2(-4.f * kC), f2(4.f * kC))) * r2;
    hg = r0 * fma2(gate, e0, dt) * up;
    hu16 = gate * dup;
    return gate * up;
  }
};
// A thread's place: columns c .. c + 7 and c + 16 .. c + 23 of row r, in a block
// of 32 columns.
struct Place {
  int block, c;
  long r;
  bool together;   // a warp holds one row
  __device__ __forceinline__ explicit Place(int rows = 1)
      : block((int)(blockIdx.y * blockDim.x + threadIdx.x) / 2), c(block * 32 + 8 * (int)(threadIdx.x & 1)),
        r((long)blockIdx.x * blockDim.y * rows + threadIdx.y), together((blockDim.x & 31) == 0) {}
  __device__ __forceinline__ bool whole(int K) const { return block * 32 + 32 <= K; }
};

template <int DT, int ACT, bool SAVE>
__global__ void __launch_bounds__(256, ACT == SITU_ACT_FN_SITU ? 5 : 6)   // 101 us with 48 registers, 104 with 64 and, spilling, with 40
gated_kernel(GatedParams p) {
  const Place at;
  const bool first = at.r < p.S && at.c < p.I, second = at.r < p.S && at.c + 16 < p.I;
  const int e = at.r < p.S ? expert_of(p.offsets, p.E, (int)at.r, at.together) : -1;
  const size_t el = (size_t)at.r * p.ldx + at.c;
  const Line g = load_line(p.x, el, first && e >= 0, second && e >= 0);
  const Line u = load_line(p.x, el + p.I, first && e >= 0, second && e >= 0);
  const uint32_t mg = amax_bits<DT>(g), mu = amax_bits<DT>(u);
  Kept kg, ku;
  if (SAVE) {
    kg = kept_of<DT>(mg);
    ku = kept_of<DT>(mu);
  }
  const Act<ACT> act(e >= 0 ? __ldg(p.p0 + e) : 1.f, e >= 0 ? __ldg(p.p1 + e) : 1.f);
  bool fits = false;
  if constexpr (ACT == SITU_ACT_FN_SITU) fits = Situ2(act).fits(amax_value<DT>(mg), amax_value<DT>(mu));
  uint4 qg, qu, h[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    float fg[8], fu[8], v[8];
    unpack8<DT>(g.v[k], fg);
    unpack8<DT>(u.v[k], fu);
    if (SAVE) {
      const uint2 a = save8(fg, kg.factor, kg.byte == 255u), b = save8(fu, ku.factor, ku.byte == 255u);
      (k ? qg.z : qg.x) = a.x;
      (k ? qg.w : qg.y) = a.y;
      (k ? qu.z : qu.x) = b.x;
      (k ? qu.w : qu.y) = b.y;
    }
    if (fits) {
      if constexpr (ACT == SITU_ACT_FN_SITU) {
        const Situ2 a(act);
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
          const float2 t = both(a.value(f2(fg[i], fg[i + 1]), f2(fu[i], fu[i + 1])));
          v[i] = t.x;
          v[i + 1] = t.y;
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = act.value(fg[i], fu[i]);
    }
    h[k] = pack8<DT>(v);
  }
  if (e < 0) h[0] = h[1] = make_uint4(0, 0, 0, 0);
  if (SAVE) {
    uint8_t* q = p.q + (size_t)at.r * 2 * p.I + at.c;
    const bool wide = p.wide && at.whole(p.I);
    store_codes(q, qg, first, second, wide);
    store_codes(q + p.I, qu, first, second, wide);
    if (first && (threadIdx.x & 1) == 0) {
      const int nb = (p.I + 31) / 32;
      uint8_t* s = p.scale + (size_t)at.r * 2 * nb + at.block;
      s[0] = (uint8_t)kg.byte;
      s[nb] = (uint8_t)ku.byte;
    }
  }
  store_line(p.h, (size_t)at.r * p.ldh + at.c, h, first, second);
}

template <int DT, int ACT, bool H>
__global__ void __launch_bounds__(256, 4)   // 123 us with 64 registers, 152 with 48, which spill
gated_back_kernel(GatedParams p) {
  const Place at;
  const int e = at.r < p.S ? expert_of(p.offsets, p.E, (int)at.r, at.together) : -1;
  if (at.r >= p.S || at.c >= p.I) return;
  const bool second = at.c + 16 < p.I;
  uint4 og[2], ou[2], oh[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) og[k] = ou[k] = oh[k] = make_uint4(0, 0, 0, 0);
  if (e >= 0) {
    const int nb = (p.I + 31) / 32;
    const uint8_t* q = p.q + (size_t)at.r * 2 * p.I + at.c;
    const uint8_t* s = p.scale + (size_t)at.r * 2 * nb + at.block;
    const uint4 qg = load_codes(q, true, second), qu = load_codes(q + p.I, true, second);
    const uint32_t bg = __ldg(s), bu = __ldg(s + nb);
    const Line d = load_line(p.dh, (size_t)at.r * p.ld_dh + at.c, true, second);
    const Act<ACT> act(__ldg(p.p0 + e), __ldg(p.p1 + e));
    const float sg = scale_value(bg), su = scale_value(bu);
    bool fits = false;
    if constexpr (ACT == SITU_ACT_FN_SITU) {
      const Situ2 a(act);
      fits = a.fits(448.f * sg, 448.f * su) || a.fits(amax_code(qg) * sg, amax_code(qu) * su);   // a code is 448 at most
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      float fg[8], fu[8], df[8], h[8];
      restore8(k ? qg.z : qg.x, k ? qg.w : qg.y, sg, fg);
      restore8(k ? qu.z : qu.x, k ? qu.w : qu.y, su, fu);
      unpack8<DT>(d.v[k], df);
      if (fits) {
        if constexpr (ACT == SITU_ACT_FN_SITU) {
          const Situ2 a(act);
          const F2 sixteen = f2(16.f);
#pragma unroll
          for (int i = 0; i < 8; i += 2) {
            F2 hg, hu;
            const F2 dd = f2(df[i], df[i + 1]);
            const float2 v = both(a.all(f2(fg[i], fg[i + 1]), f2(fu[i], fu[i + 1]), hg, hu));
            const float2 x = both(dd * hg), y = both((dd * sixteen) * hu);
            h[i] = v.x;
            h[i + 1] = v.y;
            fg[i] = x.x;
            fg[i + 1] = x.y;
            fu[i] = y.x;
            fu[i + 1] = y.y;
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float hg, hu;
          h[i] = act.all(fg[i], fu[i], hg, hu);
          fg[i] = df[i] * hg;
          fu[i] = df[i] * hu;
        }
      }
      og[k] = pack8<DT>(fg);
      ou[k] = pack8<DT>(fu);
      if (H) oh[k] = pack8<DT>(h);
    }
  }
  store_line(p.dx, (size_t)at.r * p.ld_dx + at.c, og, true, second);
  store_line(p.dx, (size_t)at.r * p.ld_dx + p.I + at.c, ou, true, second);
  if (H) store_line(p.h, (size_t)at.r * p.ldh + at.c, oh, true, second);
}

// The copies take kCopyRows rows a thread, all loads first (32,768 x 3,584 bf16:
// saved in 53 us, restored in 51, 6.7 and 6.9 TB/s).
constexpr int kCopyRows = 2;

template <int DT>
__global__ void __launch_bounds__(512)
save_kernel(const void* x, long ldx, int S, int K, uint8_t* q, uint8_t* scale, int wide) {
  const Place at(kCopyRows);
  Line l[kCopyRows];
#pragma unroll
  for (int j = 0; j < kCopyRows; ++j) {
    const long r = at.r + (long)j * blockDim.y;
    l[j] = load_line(x, (size_t)r * ldx + at.c, at.c < K && r < S, at.c + 16 < K && r < S);
  }
#pragma unroll
  for (int j = 0; j < kCopyRows; ++j) {
    const long r = at.r + (long)j * blockDim.y;
    const bool first = at.c < K && r < S, second = at.c + 16 < K && r < S;
    const Kept k = kept_of<DT>(amax_bits<DT>(l[j]));
    float f[8];
    unpack8<DT>(l[j].v[0], f);
    const uint2 a = save8(f, k.factor, k.byte == 255u);
    unpack8<DT>(l[j].v[1], f);
    const uint2 b = save8(f, k.factor, k.byte == 255u);
    store_codes(q + (size_t)r * K + at.c, make_uint4(a.x, a.y, b.x, b.y), first, second, wide && at.whole(K));
    if (first && (threadIdx.x & 1) == 0) scale[(size_t)r * ((K + 31) / 32) + at.block] = (uint8_t)k.byte;
  }
}

// Values past a 16-bit type's range become its largest.
template <int DT>
__global__ void __launch_bounds__(512)
restore_kernel(const uint8_t* q, const uint8_t* scale, int S, int K, void* x, long ldx) {
  const Place at(kCopyRows);
  if (at.c >= K) return;
  constexpr float kMost = DT == SITU_DT_BF16 ? 3.38953139e38f : 65504.f;
  const bool second = at.c + 16 < K;
  uint4 c[kCopyRows];
  uint32_t b[kCopyRows];
#pragma unroll
  for (int j = 0; j < kCopyRows; ++j) {
    const long r = at.r + (long)j * blockDim.y;
    if (r < S) {
      c[j] = load_codes(q + (size_t)r * K + at.c, true, second);
      b[j] = __ldg(scale + (size_t)r * ((K + 31) / 32) + at.block);
    }
  }
#pragma unroll
  for (int j = 0; j < kCopyRows; ++j) {
    const long r = at.r + (long)j * blockDim.y;
    if (r >= S) continue;
    const float s = scale_value(b[j]);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if (k && !second) break;
      float f[8];
      restore8(k ? c[j].z : c[j].x, k ? c[j].w : c[j].y, s, f);
      const size_t el = (size_t)r * ldx + at.c + 16 * k;
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
}

// A block's threads: x over half blocks of 32 columns, y over rows, whole warps in all.
struct Shape {
  dim3 grid, block;
};
Shape shape_of(int S, int K, int rows = 1) {   // rows of a thread
  const int pieces = (K + 31) / 32 * 2;
  int x, y, parts = 1;
  if (pieces <= 16) {
    x = pieces;
    y = 16;
  } else if (pieces <= 32) {
    x = (pieces + 3) / 4 * 4;
    y = 8;
  } else {
    parts = (pieces + 255) / 256;
    x = ((pieces + parts - 1) / parts + 31) / 32 * 32;
    y = x > 128 ? 1 : x > 64 ? 2 : 4;
  }
  const long per = (long)y * rows;
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
  p.wide = a->I % 16 == 0 && !bad(a->q, 15);
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
  const Shape sh = shape_of(S, K, kCopyRows);
  auto launch = [&](auto k) { k<<<sh.grid, sh.block, 0, (cudaStream_t)stream>>>(x, (long)ldx, S, K, q, scale, K % 16 == 0 && !bad(q, 15)); };
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
  const Shape sh = shape_of(S, K, kCopyRows);
  auto launch = [&](auto k) { k<<<sh.grid, sh.block, 0, (cudaStream_t)stream>>>(q, scale, S, K, x, (long)ldx); };
  dtype == SITU_DT_BF16 ? launch(restore_kernel<SITU_DT_BF16>)
                        : dtype == SITU_DT_F16 ? launch(restore_kernel<SITU_DT_F16>) : launch(restore_kernel<SITU_DT_F32>);
  return done();
}
