// moe_exact.h — arithmetic of the kernels whose results are exact by an argument about their bits:
// plain C++, so that the host can try it at every value it depends on.
#pragma once

#include <cmath>
#include <cstdint>
#include <cstring>
#include <initializer_list>

#ifdef __CUDACC__
#define MOE_HD __host__ __device__ __forceinline__
#else
#define MOE_HD inline
#endif

namespace moe {

// -x / s in fp32 as a division rounds it, for many x of 16-bit types and one s = rn(a / 448), a of
// the same type and at least |x|: a product with the reciprocal, and one correction by what the
// product leaves over.  Codes where x / s is halfway between two e4m3 values would else go by the
// reciprocal's rounding (4 in 10^4 of bf16 rows).  What is left over has bits 58 places below s, so
// where s is tiny x is scaled up as it is (UP; never so in fp16, whose s is from 2^-33 on or a zero
// block's).  Where x / s is below 2^-11, a code of zero, it may be off.
// Negated, a zero keeps its sign without an operation for it: a sum of two zeros is +0 unless both
// are -0.  Two values an instruction (by one: 8192 x 4096 18.9 us).
struct Quotient {
  float minus_inv, s;
  bool tiny;
  MOE_HD explicit Quotient(float scale) {
    tiny = scale < 0x1p-80f;
    s = tiny ? scale * 0x1p64f : scale;
#ifdef __CUDA_ARCH__
    minus_inv = -__frcp_rn(s);
#else
    minus_inv = -(1.0f / s);
#endif
    if (s == INFINITY) s = 0.0f;  // (finite x: zero, as the reciprocal is; infinite: not a number)
  }
  MOE_HD void divide2(float& x, float& y) const {
#ifdef __CUDA_ARCH__
    asm("{\n\t.reg .b64 v, i, s, q, r;\n\tmov.b64 v, {%0, %1};\n\tmov.b64 i, {%2, %2};\n\tmov.b64 s, {%3, %3};\n\t"
        "mul.rn.f32x2 q, v, i;\n\tfma.rn.f32x2 r, q, s, v;\n\tfma.rn.f32x2 q, r, i, q;\n\tmov.b64 {%0, %1}, q;\n\t}"
        : "+f"(x), "+f"(y)
        : "f"(minus_inv), "f"(s));
#else
    for (float* v : {&x, &y}) {
      const float q = *v * minus_inv;
      *v = fmaf(fmaf(q, s, *v), minus_inv, q);
    }
#endif
  }
  template <bool UP, int N>
  MOE_HD void divide(float (&x)[N]) const {
#pragma unroll
    for (int j = 0; j < N; j += 2) {
      if (UP) x[j] *= 0x1p64f, x[j + 1] *= 0x1p64f;
      divide2(x[j], x[j + 1]);
    }
  }
};

// Two scales of a block's sum p of e4m3 products are applied as their product where that is a normal
// number, else one after the other, the larger first where neither is zero: |p| is 0 or from 2^-18 to
// 2^25, so p times the larger has all its bits unless the whole is infinite or zero in fp32 itself.
MOE_HD bool normal(float s) {
  uint32_t b;
#ifdef __CUDA_ARCH__
  b = __float_as_uint(s);
#else
  std::memcpy(&b, &s, 4);
#endif
  return 2u * b - 0x01000000u < 0xfe000000u;
}
constexpr float kNearScale = 0x1p-63f;  // two scales from this to below its reciprocal have a normal product
MOE_HD float add_scaled(float sum, float p, float a, float b) {
  if (normal(a * b) || a == 0.0f || b == 0.0f) return fmaf(p, a * b, sum);
  const bool swap = fabsf(a) < fabsf(b);
  return fmaf(p * (swap ? b : a), swap ? a : b, sum);
}

// Sums of the draw's weights in 32-bit words, kWordBits of every weight in each: a CTA may have every
// token of the longest row, all in one sum.
constexpr int kMaxLogits = 393216;  // of a row
constexpr int kWeightBits = 45;     // a weight is below 2^this, so a row's sum below 2^64
constexpr int kWordBits = 12, kWords = 4;
static_assert(kWords * kWordBits >= kWeightBits, "every bit of a weight is in a word");
static_assert(static_cast<uint64_t>(kMaxLogits) * ((1u << kWordBits) - 1) <= UINT32_MAX, "a word holds a row's sum");
static_assert(kMaxLogits <= UINT64_MAX >> kWeightBits, "64 bits hold a row's sum");
MOE_HD uint32_t word_of(uint64_t weight, int j) {
  return static_cast<uint32_t>(weight >> (kWordBits * j)) & ((1u << kWordBits) - 1u);
}
MOE_HD uint64_t of_word(uint32_t sum, int j) { return static_cast<uint64_t>(sum) << (kWordBits * j); }

// Ranges of order keys (order_key() of a value, -0 as 0) are divided by 512: the shift that does so,
// and the part of a key in [lo, hi], from hi downwards.  Always below 512; comparing values in place
// of keys lets a +0 into a range that ends at the key of -0.
MOE_HD int part_shift(uint32_t lo, uint32_t hi) {
#ifdef __CUDA_ARCH__
  const int bits = 32 - __clz(static_cast<int>(hi - lo));
#else
  const int bits = hi == lo ? 0 : 32 - __builtin_clz(hi - lo);
#endif
  return bits > 9 ? bits - 9 : 0;
}
MOE_HD bool in_range(uint32_t key, uint32_t lo, uint32_t hi) { return key - lo <= hi - lo; }
MOE_HD uint32_t part_of(uint32_t key, uint32_t hi, int shift) { return (hi - key) >> shift; }

}  // namespace moe
