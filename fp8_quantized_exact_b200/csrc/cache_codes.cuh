// Conversions and packed FP32 arithmetic shared by the cache's kernels.
#pragma once
#include "sage_common.cuh"

namespace sage {
namespace cattn {

// Row of an 8-key block of an MMA operand -> key.  Keys of neighbouring rows
// differ in bits 0 and 2, so the 16-byte shared-memory accesses of two rows fall
// on different banks under both swizzles (64- and 128-byte rows).
__device__ __forceinline__ int key_of(int n) { return (n >> 1) ^ ((n & 1) ? 5 : 0); }

// Four codes -> bytes 0 and 2, and bytes 1 and 3, as FP16 pairs (exact).
template <int F>
__device__ __forceinline__ void codes_to_f16(uint32_t w, uint32_t& even, uint32_t& odd) {
  if (F == SAGE_CACHE_INT8) {
    // 0x6400 | (code + 128) is 1024 + 128 + code in FP16
    const uint32_t e = (w & 0x00FF00FFu) ^ 0x64806480u, o = ((w >> 8) & 0x00FF00FFu) ^ 0x64806480u;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(even) : "r"(e), "r"(0x64806480u));
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(odd) : "r"(o), "r"(0x64806480u));
  } else {
    const uint32_t p = __byte_perm(w, 0, 0x3120);
    asm("{.reg .b16 lo, hi; mov.b32 {lo, hi}, %2; cvt.rn.f16x2.e4m3x2 %0, lo; cvt.rn.f16x2.e4m3x2 %1, hi;}"
        : "=r"(even), "=r"(odd)
        : "r"(p));
  }
}

// Unused slots hold any bytes: E4M3 NaN codes become 0 (their weight is 0).
template <int F>
__device__ __forceinline__ uint32_t no_nan(uint32_t w) {
  return F == SAGE_CACHE_E4M3 ? w & ~__vcmpeq4(w & 0x7F7F7F7Fu, 0x7F7F7F7Fu) : w;
}

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Two FP32 values in one 64-bit register.
__device__ __forceinline__ uint64_t pair(float x, float y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ float2 unpair(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// Byte offset of 16-byte chunk `chunk` of row `key` of a tile of D-byte rows
// that TMA wrote with the D-byte swizzle.
template <int D>
__device__ __forceinline__ uint32_t swizzled(int key, int chunk) {
  return key * D + ((D == 128 ? chunk ^ (key & 7) : chunk ^ ((key >> 1) & 3)) << 4);
}

// The power of two by which a Q row is divided before it becomes FP16 (from the
// largest magnitude's BF16 bits): its largest value then is below 2^14, and its
// BF16 values are exact in FP16 down to 2^-27 of the largest.
__device__ __forceinline__ int q_exponent(uint32_t top) {
  return (top == 0 || top >= 0x7F80u) ? 0 : max((int)(top >> 7) - 127 - 13, -110);
}
// 2^-eq, by which a Q row is multiplied.  A row with an infinity or a NaN becomes NaN in every channel, so that all its scores
// are: infinities would pass for a row that sees nothing where they all are negative.
__device__ __forceinline__ float q_down(uint32_t top, int eq) {
  return __int_as_float(top >= 0x7F80u ? 0x7FC00000 : (127 - eq) << 23);
}
// The factor of the row's scores, which hold sm_scale log2 e already (it goes to the key's scale): a power of two, so that
// x f - c is the difference of two scores without a rounding of either product.  With sm_scale in f the fused x f - c
// kept what rounding had taken from c, which passes 2^16 from scores of 2^40 on.
__device__ __forceinline__ float q_factor(int eq) { return __int_as_float((127 + eq) << 23); }

// A row's weights p v-scale 2^-E are FP16 in the MMAs, which holds 11 bits from 2^-14 to 2^16 and ever fewer down to 2^-25.
// Where that range lies is what the row's offset c decides: p = 2^(s - c), V scales times 2^-E are at most 1, and c follows
// the largest weight, not the largest score: a key of nearly all the probability and next to no value, or of a huge
// V scale and no probability, leaves the others their bits.  Weights down to 2^-21 of the largest that the row met keep
// 11 bits; the others are off by at most 2^-32 of the largest.  p itself is FP32 and may be large.
constexpr float kHead = 8.0f;   // when c is set, the tile's largest weight is in (2^(kHead - 1), 2^kHead]
constexpr float kLimit = 15.0f;  // scores that pass c by more raise it (log2)
constexpr float kLow = 76.0f;    // p stays at or below 2^(kLow + kHead), however small the weights beside it are (an lse of such a
                                 // row is off by up to 2^-18, FP32's step of its s - c)
constexpr float kMass = 100.0f;  // a row's sum stays below 2^kMass when c is lowered because E grew

// c for a tile whose largest score is `top` and whose largest score plus log2 of its V scale is `weight` (rounded up): an
// integer, so that factors between offsets are powers of two; rounded up, so that large scores, which leave no room
// for the small terms, put c at `top` at most.
__device__ __forceinline__ float tile_offset(float top, float weight, int E) {
  return ceilf(__fadd_ru(fminf(fmaxf(__fadd_ru(weight, -(float)E), __fadd_ru(top, -kLow)), top), -kHead));
}
// c when E grows by `de`: what keeps the unit of the weights' sums, 2^(c + E), as long as the row's sum, `mass` so far, has room.
__device__ __forceinline__ float kept_offset(float c, int de, float mass) {
  const float room = fmaxf(kMass - (float)((__float_as_int(mass) >> 23) - 126), 0.0f);
  return __fadd_ru(c, -fminf((float)de, room));
}

// A row's sum l with its offset c as c' and l' in [2^-bias, 2^(1-bias)), and g = l' / l: l may be large, and the row's
// weighted sum is l times a mean of values.  What is joined has a bias: up to 12 parts of a CTA and then up to 148 of a
// unit stay below the largest value in all (12 * 148 * 2^(1 - kPartBias) < 1).  l is below 2^113 by the limits above (2^28
// keys), so g is a normal number.
struct Mass {
  float c, l, g;
};
constexpr int kPartBias = 12;
__device__ __forceinline__ Mass normalised(float c, float l, int bias) {
  const int k = l > 0.0f && l < 0x1p127f ? (__float_as_int(l) >> 23) - 127 + bias : 0;  // zero, infinity and NaN stay
  if (k == 0) return {c, l, 1.0f};
  const float c2 = c + (float)k;  // rounded where c passes 2^24: the factor is of what it became
  float g;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(g) : "f"(c - c2));
  return {c2, l * g, g};
}

}  // namespace cattn
}  // namespace sage
