// group.cuh -- 4-bit weights with group scales: the packed word and its 16-bit element types.
//
// A weight value is s (q - z): q the 4-bit code, s a 16-bit scale and z a zero point of 0..15 (8 where none is
// stored), both one per group of 32, 64 or 128 consecutive columns.  s (q - z) has at most 11 + 4 significant bits,
// so fp32 holds it exactly.  Eight codes of a row share a little-endian 32-bit word: code j sits in nibble j / 2 of
// the low half (j even) or of the high half (j odd), so
//   (word >> 4 i) & 0x000f000f
// is the pair (code 2i, code 2i + 1), each in the low bits of one 16-bit half: with the bits of 128 (bf16) or 1024
// (fp16) or-ed in, the half is 128 + code (1024 + code) exactly, and one packed subtraction of 128 + z leaves the
// integer q - z as an exact 16-bit float.
#pragma once
#include <cuda_fp16.h>

#include "nf4_common.cuh"

namespace nf4 {

template <bool kHalf>
struct GroupType {  // bf16
  using T = __nv_bfloat16;
  static constexpr uint32_t kBias = 0x43004300u;  // 128, 128
  static constexpr float kBiasF = 128.0f;
  static __device__ __forceinline__ float to_f32(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }
  // round to nearest even; values beyond the largest finite one stay at it (scales only)
  static __device__ __forceinline__ uint16_t scale_bits(float v) {
    return __bfloat16_as_ushort(__float2bfloat16_rn(fminf(v, 3.3895313892515355e38f)));
  }
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) { return pack_bf16x2(lo, hi); }
  static __device__ __forceinline__ uint32_t sub2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
  }
  // d = A B + c
  static __device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                             uint32_t b0, uint32_t b1, float c0, float c1, float c2, float c3) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
  }
};

template <>
struct GroupType<true> {  // fp16
  using T = __half;
  static constexpr uint32_t kBias = 0x64006400u;  // 1024, 1024
  static constexpr float kBiasF = 1024.0f;
  static __device__ __forceinline__ float to_f32(uint16_t v) { return __half2float(__ushort_as_half(v)); }
  static __device__ __forceinline__ uint16_t scale_bits(float v) {
    return __half_as_ushort(__float2half_rn(fminf(v, 65504.0f)));
  }
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    uint32_t d;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
  }
  static __device__ __forceinline__ uint32_t sub2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
  }
  static __device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                             uint32_t b0, uint32_t b1, float c0, float c1, float c2, float c3) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
  }
};

}  // namespace nf4
