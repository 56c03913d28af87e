// Per-block NVFP4 quantization arithmetic shared by the quantize kernel and
// the GEMM that quantizes its activation operand itself.  Both must encode
// bit for bit alike, so both call quantize_block().
//
// Format [picx.dev summary of "Why Gated DeltaNet Survives 4-Bit
// Quantization", "Background"]: E2M1 values, one E4M3 scale per 16-element
// block set from blockmax/6, one FP32 scale per tensor.  Per block:
//   amax_b = max|x|, t = (amax_b/6)*g, s = E4M3_rn_sat(t),
//   s == 0 -> signed-zero codes, else r = g/e4m3(s), code = E2M1_rn_sat(x*r).
// All FP32 steps use explicitly rounded intrinsics (no contraction), and the
// FP8/FP4 encodings use the hardware cvt.rn.satfinite conversions.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cstdint>

namespace nvfp4 {

// Unsigned division by an invariant divisor d (Granlund and Montgomery,
// "Division by invariant integers using multiplication", 1994, unsigned
// case): with l = ceil(log2 d) and m = floor(2^32 (2^l - d) / d) + 1,
// n / d == (mulhi(n, m) + n) >> l for every 32-bit n.
struct DivU32 {
  uint32_t m, l;
};

__device__ __forceinline__ uint32_t div_u32(uint32_t n, DivU32 d) {
  const uint32_t t = __umulhi(n, d.m);
  return (uint32_t)(((uint64_t)t + n) >> d.l);
}

// Host side: the (m, l) pair for divisor d >= 1.
inline DivU32 make_div(uint32_t d) {
  uint32_t l = 0;
  while ((1ull << l) < d) ++l;
  DivU32 r;
  r.l = l;
  r.m = (uint32_t)((((1ull << l) - d) << 32) / d + 1);
  return r;
}


// ----------------------------------------------------------------- encoders

__device__ __forceinline__ uint32_t cvt_e4m3(float t) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(t), "f"(t));
  return r & 0xFFu;
}

__device__ __forceinline__ float e4m3_to_f32(uint32_t s) {
  uint32_t h2;
  const uint16_t in = (uint16_t)(s & 0xFF);
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(in));
  return __half2float(__ushort_as_half((unsigned short)(h2 & 0xFFFF)));
}

// Eight floats -> eight E2M1 codes, element 0 in the low nibble of the low byte.
__device__ __forceinline__ uint32_t cvt_e2m1x8(const float (&y)[8]) {
  uint32_t out;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(out)
      : "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]), "f"(y[4]), "f"(y[5]), "f"(y[6]), "f"(y[7]));
  return out;
}

__device__ __forceinline__ uint32_t cvt_e2m1x2(float lo, float hi) {
  uint32_t out;
  asm("{\n\t.reg .b8 b0;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.u32.u8 %0, b0;\n\t}"
      : "=r"(out)
      : "f"(lo), "f"(hi));
  return out;
}

// Offset of scale j of row r in the tensor-core scale layout.
__device__ __forceinline__ int64_t tc_scale_offset(int64_t r, int64_t j, int64_t kc) {
  return ((r >> 7) * kc + (j >> 2)) * 512 + (r & 31) * 16 + ((r >> 5) & 3) * 4 + (j & 3);
}

// One thread owns one 16-element block: 32 (bf16) or 64 (f32) contiguous
// bytes in, 8 bytes of codes and one scale byte out; a warp reads 1 KB
// (bf16) and writes 256 contiguous bytes of codes.
template <bool kF32>
struct Block16 {
  uint4 v[kF32 ? 4 : 2];
};

// The 16 elements at p (16-byte aligned), for data that several CTAs read.
template <bool kF32>
__device__ __forceinline__ void load_block_at(const void* p, Block16<kF32>& B) {
  const uint4* q = reinterpret_cast<const uint4*>(p);
#pragma unroll
  for (int i = 0; i < (kF32 ? 4 : 2); ++i) B.v[i] = q[i];
}

// The same through 32-byte loads and stores, one whole DRAM sector a lane
// (16-byte ones at this stride use half of each sector they touch, twice).
// `wide`: the address is 32-byte aligned; else 16-byte pieces.
__device__ __forceinline__ void ld_32b(const void* p, uint4& a, uint4& b, bool wide) {
  if (wide) {
    asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(a.x), "=r"(a.y), "=r"(a.z), "=r"(a.w), "=r"(b.x), "=r"(b.y), "=r"(b.z), "=r"(b.w)
                 : "l"(p)
                 : "memory");
  } else {
    a = *reinterpret_cast<const uint4*>(p);
    b = *(reinterpret_cast<const uint4*>(p) + 1);
  }
}

__device__ __forceinline__ void st_32b(void* p, const uint4& a, const uint4& b, bool wide) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(a.x), "r"(a.y), "r"(a.z),
                 "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
                 : "memory");
  } else {
    *reinterpret_cast<uint4*>(p) = a;
    *(reinterpret_cast<uint4*>(p) + 1) = b;
  }
}

template <bool kF32>
__device__ __forceinline__ void load_block_wide(const void* p, Block16<kF32>& B, bool wide) {
#pragma unroll
  for (int i = 0; i < (kF32 ? 2 : 1); ++i)
    ld_32b(reinterpret_cast<const uint8_t*>(p) + 32 * i, B.v[2 * i], B.v[2 * i + 1], wide);
}

template <bool kF32>
__device__ __forceinline__ void load_block(const void* x, uint32_t b, Block16<kF32>& B) {
  const uint4* p = reinterpret_cast<const uint4*>(x) + (size_t)b * (kF32 ? 4 : 2);
#pragma unroll
  for (int i = 0; i < (kF32 ? 4 : 2); ++i) B.v[i] = __ldcs(p + i);
}

// Largest magnitude of the block.  bf16: clear both sign bits of each packed
// pair and take the unsigned 16-bit maximum (non-negative bf16 bit patterns
// order like their values; inputs are finite), then widen exactly to f32.
template <bool kF32>
__device__ __forceinline__ float block_amax(const Block16<kF32>& B) {
  if constexpr (kF32) {
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      m = fmaxf(m, fabsf(__uint_as_float(B.v[i].x)));
      m = fmaxf(m, fabsf(__uint_as_float(B.v[i].y)));
      m = fmaxf(m, fabsf(__uint_as_float(B.v[i].z)));
      m = fmaxf(m, fabsf(__uint_as_float(B.v[i].w)));
    }
    return m;
  } else {
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      w = __vmaxu2(w, B.v[i].x & 0x7FFF7FFFu);
      w = __vmaxu2(w, B.v[i].y & 0x7FFF7FFFu);
      w = __vmaxu2(w, B.v[i].z & 0x7FFF7FFFu);
      w = __vmaxu2(w, B.v[i].w & 0x7FFF7FFFu);
    }
    const uint32_t m16 = max(w >> 16, w & 0xFFFFu);
    return __uint_as_float(m16 << 16);
  }
}

template <bool kF32>
__device__ __forceinline__ void block_floats(const Block16<kF32>& B, float (&f)[16]) {
  if constexpr (kF32) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[4 * i + 0] = __uint_as_float(B.v[i].x);
      f[4 * i + 1] = __uint_as_float(B.v[i].y);
      f[4 * i + 2] = __uint_as_float(B.v[i].z);
      f[4 * i + 3] = __uint_as_float(B.v[i].w);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t w[4] = {B.v[i].x, B.v[i].y, B.v[i].z, B.v[i].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        f[8 * i + 2 * k] = __uint_as_float(w[k] << 16);              // bf16 -> f32 is exact
        f[8 * i + 2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
      }
    }
  }
}

// rtab entry for scale byte s: g / e4m3(s) for s in 1..126, 0 otherwise.
__device__ __forceinline__ float recip_entry(float g, uint32_t s) {
  return (s >= 1 && s <= 126) ? __fdiv_rn(g, e4m3_to_f32(s)) : 0.0f;
}

// One 16-element block: returns the scale byte and the 16 codes (lo: elements
// 0-7, hi: elements 8-15, element 0 in the low nibble).  rtab as above.
template <bool kF32>
__device__ __forceinline__ uint32_t quantize_block(const Block16<kF32>& B, float g, const float* rtab,
                                                   uint32_t& lo, uint32_t& hi, float* amax_out = nullptr) {
  const float amax = block_amax<kF32>(B);
  if (amax_out) *amax_out = amax;
  const float q = __fdiv_rn(amax, 6.0f);
  const float t = __fmul_rn(q, g);
  const uint32_t s = cvt_e4m3(t);
  float f[16];
  block_floats<kF32>(B, f);
  if (s == 0) {
    lo = hi = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      lo |= ((__float_as_uint(f[i]) >> 31) << 3) << (4 * i);
      hi |= ((__float_as_uint(f[8 + i]) >> 31) << 3) << (4 * i);
    }
  } else {
    const float r = rtab[s];
    float y0[8], y1[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      y0[i] = __fmul_rn(f[i], r);
      y1[i] = __fmul_rn(f[8 + i], r);
    }
    lo = cvt_e2m1x8(y0);
    hi = cvt_e2m1x8(y1);
  }
  return s;
}

// The same block from FP32 values, for kernels that quantize what they just
// computed or use one global scale a group: amax must be the largest
// magnitude of f.  Bit for bit what quantize_block writes for the same values
// and scale, with the two divisions replaced:
//   amax / 6   by a product with 1/6 and one fused correction (division by a
//              constant; Brisebarre, Muller and Raina, "Accelerating correctly
//              rounded floating-point division when the divisor is known in
//              advance", 2004), checked against the division for every
//              mantissa; below 2^-100, where the correction could underflow,
//              it stays a division;
//   g / s      by q[m] 2^-e for s = (1 + m/8) 2^e, with the eight quotients
//              q[m] = g / (1 + m/8) taken once per scale: a power of two
//              scales a rounded quotient exactly while nothing is subnormal
//              (g >= 2^-100).
constexpr float kTinyAmax = 7.888609052210118e-31f;   // 2^-100

// Quotient m of a global scale's table of eight.
__device__ __forceinline__ float scale_quotient(float g, int m) { return __fdiv_rn(g, 1.0f + (float)m * 0.125f); }

__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 r;
  asm("{\n\t.reg .b64 x, y, z;\n\t"
      "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "mul.rn.f32x2 z, x, y;\n\t"
      "mov.b64 {%0, %1}, z;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}

__device__ __forceinline__ uint32_t quantize_values(const float (&f)[16], float amax, float g, const float* quot,
                                                    uint32_t& lo, uint32_t& hi) {
  constexpr float kSixth = 1.0f / 6.0f;
  const float q0 = __fmul_rn(amax, kSixth);
  float q = __fmaf_rn(__fmaf_rn(-6.0f, q0, amax), kSixth, q0);
  if (amax < kTinyAmax) q = __fdiv_rn(amax, 6.0f);
  const uint32_t s = cvt_e4m3(__fmul_rn(q, g));
  const uint32_t bits = __float_as_uint(e4m3_to_f32(s));
  float r = __fmul_rn(quot[(bits >> 20) & 7], __uint_as_float((254u << 23) - (bits & 0x7F800000u)));
  if (g < kTinyAmax) r = __fdiv_rn(g, __uint_as_float(bits));
  if (s == 0) r = 0.0f;                    // codes are signed zeros
  const float2 r2 = make_float2(r, r);
  float y0[8], y1[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 u = mul2(make_float2(f[2 * i], f[2 * i + 1]), r2);
    const float2 v = mul2(make_float2(f[8 + 2 * i], f[9 + 2 * i]), r2);
    y0[2 * i] = u.x;
    y0[2 * i + 1] = u.y;
    y1[2 * i] = v.x;
    y1[2 * i + 1] = v.y;
  }
  lo = cvt_e2m1x8(y0);
  hi = cvt_e2m1x8(y1);
  return s;
}

// x * sigmoid(x): exp to 2 ulp, an approximate quotient of 2 (flushed to zero
// beyond 2^126: the limit's own value).
__device__ __forceinline__ float silu(float x) { return __fdividef(x, 1.0f + expf(-x)); }

// f_i *= num_i / (1 + exp(-x_i)): a sigmoid (num = 1) or SiLU (num = x) gate
// of a block.  The special-function unit is what gates cost (a warp's exp or
// reciprocal holds it for 8 cycles), so two quotients share a reciprocal,
// 1 / a = b * (1 / (a b)), which holds while the product stays finite: for
// x >= -43 throughout the block.  exp to 2 ulp, reciprocal 1 ulp, a few
// products.  (The block norm gains by it, 30.7 to 28.3 us for gated heads of
// 4096 x 4096 and 98 to 80 us for a gated 1003 x 17408; the quantizer's SwiGLU,
// which has more other work a load, took 23 instead of 21 us and uses silu().)
template <bool kSilu>
__device__ __forceinline__ void apply_gate(const float (&x)[16], float (&f)[16]) {
  float low = x[0];
#pragma unroll
  for (int i = 1; i < 16; ++i) low = fminf(low, x[i]);
  if (low >= -43.0f) {
#pragma unroll
    for (int i = 0; i < 16; i += 2) {
      const float a = 1.0f + expf(-x[i]), b = 1.0f + expf(-x[i + 1]);
      const float r = __fdividef(1.0f, __fmul_rn(a, b));
      f[i] *= kSilu ? x[i] * (b * r) : b * r;
      f[i + 1] *= kSilu ? x[i + 1] * (a * r) : a * r;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i)
      f[i] *= __fdividef(kSilu ? x[i] : 1.0f, 1.0f + expf(-x[i]));
  }
}

}  // namespace nvfp4
