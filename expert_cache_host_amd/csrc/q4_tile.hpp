// Device helpers for 4-bit codes on the matrix cores, shared by the
// matrix-vector product and the cache's attention.
//
// v_mfma_f32_16x16x32_f16: lane l = (n = l % 16, g = l / 16) holds 8 halves of
// row n of A (column n of B), K slots 8 g .. 8 g + 7; of C it holds column n and
// rows 4 g + i.  A block of 32 codes is 4 words; word g decodes to the elements
// 4 g .. 4 g + 3 and 4 g + 16 .. 4 g + 19, in the order unit_order() says, so a
// lane's K slots are one word and the other operand is laid out to match.
#pragma once
#include <hip/hip_runtime.h>

#include <cstdint>

namespace moe {

typedef _Float16 half2_t __attribute__((ext_vector_type(2)));
typedef _Float16 half8_t __attribute__((ext_vector_type(8)));
typedef float floatx4 __attribute__((ext_vector_type(4)));

// The constants of the decoding, held in registers: with literals the compiler
// takes an and and an or where v_and_or_b32 does both.
struct CodeBits {
  uint32_t lo = 0x000f000fu, hi = 0x00f000f0u, one = 0x64006400u;
  __device__ __forceinline__ CodeBits() {
    asm("" : "+s"(lo));
    asm("" : "+s"(hi));
    asm("" : "+v"(one));
  }
  // Two codes minus 8 from the low nibbles of a word's halves: or-ing a nibble
  // into binary16 1024 gives 1024 + q; both steps are exact.
  __device__ __forceinline__ half2_t low(uint32_t w) const {
    const half2_t v = __builtin_bit_cast(half2_t, (w & lo) | one);
    return v - half2_t{(_Float16)1032.f, (_Float16)1032.f};
  }
  // The same from the second nibbles: 1024 + 16 q, so (1024 + 16 q) / 16 - 72 = q - 8.
  __device__ __forceinline__ half2_t high(uint32_t w) const {
    const half2_t v = __builtin_bit_cast(half2_t, (w & hi) | one);
    return __builtin_elementwise_fma(v, half2_t{(_Float16)0.0625f, (_Float16)0.0625f},
                                     half2_t{(_Float16)-72.f, (_Float16)-72.f});
  }
};

__device__ __forceinline__ half8_t join8(half2_t a, half2_t b, half2_t c, half2_t d) {
  return half8_t{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// The eight values q - 8 of a word: elements (0, 2, 16, 18, 1, 3, 17, 19) + 4 g
// of its block when the word is word g.
__device__ __forceinline__ half8_t decode_word(const CodeBits &c, uint32_t w) {
  return join8(c.low(w), c.high(w), c.low(w >> 8), c.high(w >> 8));
}

// Codes as the matrix cores can take them without any arithmetic: a nibble q in
// the low bits of a half is the subnormal q 2^-24, one in the next four bits 16 q
// 2^-24, and the products of subnormals are exact.  The second nibbles' factor
// 16 is for the other operand or the result to take away, as are the 2^-24 and
// the codes' offset of 8.
struct RawCodes {
  static __device__ __forceinline__ uint32_t low(uint32_t w) { return w & 0x000f000fu; }
  static __device__ __forceinline__ uint32_t high(uint32_t w) { return w & 0x00f000f0u; }
  static __device__ __forceinline__ half8_t join(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    return __builtin_bit_cast(half8_t, make_uint4(a, b, c, d));
  }
  // A word in decode_word's order; K slots 2, 3, 6 and 7 hold 16 times the code.
  static __device__ __forceinline__ half8_t word(uint32_t w) {
    return join(low(w), high(w), low(w >> 8), high(w >> 8));
  }
  // -8 as a word's slots would hold it.
  static __device__ __forceinline__ half8_t minus_eight() {
    return join(0x80088008u, 0x80808080u, 0x80088008u, 0x80808080u);
  }
  // What slot j of the other operand is multiplied by.
  static __device__ __forceinline__ constexpr float slot(int j) { return j & 2 ? 0.0625f : 1.f; }
};

// Puts x[4 g .. 4 g + 3] (a) and x[4 g + 16 .. 4 g + 19] (b) into decode_word's order.
__device__ __forceinline__ void unit_order(const float4 a, const float4 b, float (&v)[8]) {
  v[0] = a.x, v[1] = a.z, v[2] = b.x, v[3] = b.z;
  v[4] = a.y, v[5] = a.w, v[6] = b.y, v[7] = b.w;
}

// 4 x 4 transpose of words over the wave's four 16-lane rows: row g holds words
// 0..3 of item g before, word g of items 0..3 after.
__device__ __forceinline__ uint4 transpose_rows(uint4 v) {
  const auto a = __builtin_amdgcn_permlane32_swap(v.x, v.z, false, false);
  const auto b = __builtin_amdgcn_permlane32_swap(v.y, v.w, false, false);
  const auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
  const auto d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
  return make_uint4(c[0], c[1], d[0], d[1]);
}

// Every row's word, in all rows: row g holds s_g before, (s_0 .. s_3) after.
__device__ __forceinline__ uint4 gather_rows(uint32_t s) {
  const auto a = __builtin_amdgcn_permlane32_swap(s, s, false, false);
  const auto b = __builtin_amdgcn_permlane16_swap(a[0], a[0], false, false);
  const auto c = __builtin_amdgcn_permlane16_swap(a[1], a[1], false, false);
  return make_uint4(b[0], b[1], c[0], c[1]);
}

// Largest value over the four 16-lane rows, per lane n.
__device__ __forceinline__ uint32_t rows_max_u32(uint32_t v) {
  const auto a = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  const uint32_t m = max(a[0], a[1]);
  const auto b = __builtin_amdgcn_permlane16_swap(m, m, false, false);
  return max(b[0], b[1]);
}

// Largest value over the wave: DPP within rows of 16 lanes, then across them.
__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
  v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, true));   // quad_perm [1,0,3,2]
  v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, true));   // quad_perm [2,3,0,1]
  v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x141, 0xF, 0xF, true));  // row_half_mirror
  v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x140, 0xF, 0xF, true));  // row_mirror
  return rows_max_u32(v);
}

// Between LDS writes of a wave's lanes and its other lanes' reads of them, or such
// reads and the next writes over them: LDS serves a wave's accesses in order, and
// this holds the compiler to their order, whatever types they are made through.
__device__ __forceinline__ void wave_lds_order() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Exponent e for which |v| * 2^-e lies below 2^14 for every v whose magnitude
// bits are at most `bits` (the bits of the largest, as an integer), kept where
// 2^e and 2^-e are normal floats.  Infinities and NaN clamp at the top.
__device__ __forceinline__ int scale_exp(uint32_t bits) {
  return min(max((int)(bits >> 23) - 127 - 13, -126), 126);
}
__device__ __forceinline__ float exp2_int(int e) {
  return __builtin_bit_cast(float, (uint32_t)(e + 127) << 23);
}

// Binary16 parts of v: hi + lo keeps 2^-22 of v down to 2^-25 of the unit; an
// infinity stays one in hi alone.
__device__ __forceinline__ void split_half(float v, _Float16 &hi, _Float16 &lo) {
  hi = (_Float16)v;
  const float h = (float)hi;
  lo = (_Float16)(h == v ? 0.f : v - h);
}

}  // namespace moe
