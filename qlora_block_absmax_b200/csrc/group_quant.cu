// group_quant.cu -- weights of uniform 4-bit codes with group scales: quantization and expansion.
//
// Quantization of one group of G consecutive columns (G = 32, 64 or 128), every step rounded once in fp32:
//   with zero points   lo = min(0, min w), hi = max(0, max w), s = T((hi - lo) / 15), z = clamp(rint(-lo / s), 0, 15)
//   symmetric          s = T(max |w| / 7), z = 8
//   q = clamp(rint(w / s) + z, 0, 15),  rint to the nearest even integer, s == 0: q = z (z = 0 with zero points)
// where T rounds to the scales' 16-bit type.  Expansion: T'(s (q - z)), the product exact in fp32.
//
// One lane holds two packed words (16 codes), G / 16 lanes share a group and find its range with shuffles.  The kernel's
// bound is its instructions, so little is divided and nothing goes through the conversion units (a quarter of the rate of
// the others): the quotients are products with an approximate 1 / s, rounded by adding 1.5 * 2^23.  Such a product is off
// by at most 1.5 * 2^-23 of its size, 2.9e-6 where |w / s| <= 16, and the fp32 quotient by 2^-24, 4.8e-7 below 16; a
// product within 4e-6 of a rounding border b (an integer and a half) is settled exactly, so every code is the one the
// division gives:
//   fp32 source    by the division itself (2 in 10^5 values)
//   16-bit source  w and b s have at most 11 and 16 significant bits, so where they differ, they do by 2^-16 of their
//                  size, 7.6e-6 at the least border: w / s = b, and the even neighbour is the code.  (w = s / 2 is common among
//                  bf16 weights: most warps meet a tie.)
// 4096x4096 bf16 with zero points took 23.4 us with IEEE quotients, rintf and float-to-integer conversions on one word
// per lane, 19.6 us with the division in every tie.
//
// Expansion: one word per lane, so that a warp's stores are contiguous; bound by HBM.
#include "group.cuh"
#include "internal.h"

namespace nf4 {
namespace {

constexpr int kThreads = 256;
constexpr float kRound = 12582912.0f;  // 1.5 * 2^23: adding it rounds to the nearest integer, ties to even
constexpr float kNear = 0.499996f;     // |t - rint(t)| beyond this: t may stand for a value on the other side of a border

// t = w / s but for an error below 4e-6, q = rint(t): rint of the exact quotient where a near one is a tie
__device__ __forceinline__ float settle_tie(float t, float q) {
  const float d = t - q;
  // q's parity is the last mantissa bit of 1.5 * 2^23 + q
  const bool odd = __float_as_uint(__fadd_rn(q, kRound)) & 1u;
  return fabsf(d) > kNear && odd ? q + copysignf(1.0f, d) : q;
}

template <int kSrc>  // 0 fp32, 1 bf16, 2 fp16
__device__ __forceinline__ void load16(const void* src, int64_t pair, float (&v)[16]) {
  if constexpr (kSrc == 0) {
    const float4* p = reinterpret_cast<const float4*>(src) + pair * 4;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 a = __ldcs(p + i);
      v[4 * i] = a.x;
      v[4 * i + 1] = a.y;
      v[4 * i + 2] = a.z;
      v[4 * i + 3] = a.w;
    }
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint4 a = __ldcs(reinterpret_cast<const uint4*>(src) + pair * 2 + h);
      const uint32_t r[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[8 * h + 2 * i] = GroupType<kSrc == 2>::to_f32((uint16_t)(r[i] & 0xffffu));
        v[8 * h + 2 * i + 1] = GroupType<kSrc == 2>::to_f32((uint16_t)(r[i] >> 16));
      }
    }
  }
}

__device__ __forceinline__ float rcp_approx(float x) {
  float d;
  asm("rcp.approx.f32 %0, %1;" : "=f"(d) : "f"(x));
  return d;
}

// kL = G / 16 lanes per group; kHalf: fp16 scales (else bf16); kZeros: zero points
template <int kSrc, int kL, bool kHalf, bool kZeros>
__global__ void __launch_bounds__(kThreads)
    quantize_groups_kernel(const void* __restrict__ src, int64_t pairs, uint2* __restrict__ packed,
                           uint16_t* __restrict__ scale, uint8_t* __restrict__ zero) {
  using G = GroupType<kHalf>;
  pdl_launch_dependents();
  pdl_wait();
  const int64_t stride = (int64_t)gridDim.x * kThreads;
  // the loop bound is that of the warp's first lane, so the shuffles always see all 32 lanes; a group lies within
  // one warp and is present in whole or not at all (pairs is a multiple of kL)
  const int lane = threadIdx.x & 31;
  for (int64_t p0 = (int64_t)blockIdx.x * kThreads + (threadIdx.x - lane); p0 < pairs; p0 += stride) {
    const int64_t pair = p0 + lane;
    const bool valid = pair < pairs;
    float v[16];
    if (valid) {
      load16<kSrc>(src, pair, v);
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = 0.0f;
    }
    float lo = 0.0f, hi = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      if constexpr (kZeros) lo = fminf(lo, v[i]);
      hi = fmaxf(hi, kZeros ? v[i] : fabsf(v[i]));
    }
#pragma unroll
    for (int d = 1; d < kL; d <<= 1) {
      if constexpr (kZeros) lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, d));
      hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, d));
    }
    const uint16_t sbits = G::scale_bits(kZeros ? __fdiv_rn(__fsub_rn(hi, lo), 15.0f) : __fdiv_rn(hi, 7.0f));
    const float s = G::to_f32(sbits);
    float z = kZeros ? 0.0f : 8.0f;
    uint32_t out[2] = {0, 0};
    if (s > 0.0f) {
      const float inv = rcp_approx(s);
      float q[16], far = 0.0f, qz = 0.0f;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float t = v[i] * inv;
        q[i] = __fsub_rn(__fadd_rn(t, kRound), kRound);
        far = fmaxf(far, fabsf(t - q[i]));
      }
      if constexpr (kZeros) {
        const float t = -lo * inv;
        qz = __fsub_rn(__fadd_rn(t, kRound), kRound);
        far = fmaxf(far, fabsf(t - qz));
      }
      // near a border, or a scale so small that 1 / s is not an ordinary number
      if (kSrc != 0 && far > kNear && s >= 1e-30f) {
#pragma unroll
        for (int i = 0; i < 16; ++i) q[i] = settle_tie(v[i] * inv, q[i]);
        if constexpr (kZeros) qz = settle_tie(-lo * inv, qz);
      } else if (!(far <= kNear) || s < 1e-30f) {
#pragma unroll
        for (int i = 0; i < 16; ++i) q[i] = rintf(__fdiv_rn(v[i], s));
        if constexpr (kZeros) qz = rintf(__fdiv_rn(-lo, s));
      }
      if constexpr (kZeros) z = fminf(qz, 15.0f);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        // 2^23 + code: the code in the low mantissa bits
        const float c = __fadd_rn(fminf(fmaxf(__fadd_rn(q[i], z), 0.0f), 15.0f), 8388608.0f);
        out[i >> 3] |= (__float_as_uint(c) & 15u) << (4 * ((i & 7) >> 1) + 16 * (i & 1));
      }
    } else {
      out[0] = out[1] = (uint32_t)z * 0x11111111u;
    }
    if (valid) {
      packed[pair] = make_uint2(out[0], out[1]);
      if ((lane & (kL - 1)) == 0) {
        const int64_t g = pair / kL;
        scale[g] = sbits;
        if constexpr (kZeros) zero[g] = (uint8_t)z;
      }
    }
  }
}

// kOut: 0 fp32, 1 bf16, 2 fp16; shift: log2(G / 8), words per group
template <int kOut, bool kHalf>
__global__ void __launch_bounds__(kThreads)
    dequantize_groups_kernel(const uint32_t* __restrict__ packed, const uint16_t* __restrict__ scale,
                             const uint8_t* __restrict__ zero, int64_t words, int shift, void* __restrict__ out) {
  pdl_launch_dependents();
  pdl_wait();
  const int64_t stride = (int64_t)gridDim.x * kThreads;
  for (int64_t word = (int64_t)blockIdx.x * kThreads + threadIdx.x; word < words; word += stride) {
    const uint32_t w = __ldcs(packed + word);
    const int64_t g = word >> shift;
    const float s = GroupType<kHalf>::to_f32(__ldg(scale + g));
    const float z = 8388608.0f + (zero != nullptr ? (float)__ldg(zero + g) : 8.0f);
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t c = (w >> (4 * (i >> 1) + 16 * (i & 1))) & 15u;
      v[i] = __fmul_rn(__fsub_rn(__uint_as_float(0x4b000000u | c), z), s);  // 2^23 + c, exact
    }
    if constexpr (kOut == 0) {
      float4* p = reinterpret_cast<float4*>(out) + word * 2;
      __stcs(p, make_float4(v[0], v[1], v[2], v[3]));
      __stcs(p + 1, make_float4(v[4], v[5], v[6], v[7]));
    } else {
      using G = GroupType<kOut == 2>;
      __stcs(reinterpret_cast<uint4*>(out) + word,
             make_uint4(G::pack(v[0], v[1]), G::pack(v[2], v[3]), G::pack(v[4], v[5]), G::pack(v[6], v[7])));
    }
  }
}

unsigned grid_for(int64_t items, int num_sms) {
  const int64_t need = (items + kThreads - 1) / kThreads, most = (int64_t)num_sms * 8;
  return (unsigned)(need < most ? need : most);
}

template <int kSrc, int kL, bool kHalf>
cudaError_t launch_quant(const void* src, int64_t pairs, const GroupWeight& g, cudaStream_t stream, int num_sms) {
  auto* packed = reinterpret_cast<uint2*>(const_cast<uint8_t*>(g.packed));
  auto* scale = const_cast<uint16_t*>(static_cast<const uint16_t*>(g.scale));
  auto* zero = const_cast<uint8_t*>(g.zero);
  const dim3 grid(grid_for(pairs, num_sms));
  const cudaError_t e =
      zero != nullptr ? launch_pdl(quantize_groups_kernel<kSrc, kL, kHalf, true>, grid, dim3(kThreads), 0, stream, src,
                                   pairs, packed, scale, zero)
                      : launch_pdl(quantize_groups_kernel<kSrc, kL, kHalf, false>, grid, dim3(kThreads), 0, stream,
                                   src, pairs, packed, scale, zero);
  count_launches(1);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <int kSrc, int kL>
cudaError_t launch_quant_scale(const void* src, int64_t pairs, const GroupWeight& g, cudaStream_t stream,
                               int num_sms) {
  return g.half ? launch_quant<kSrc, kL, true>(src, pairs, g, stream, num_sms)
                : launch_quant<kSrc, kL, false>(src, pairs, g, stream, num_sms);
}

template <int kSrc>
cudaError_t launch_quant_group(const void* src, int64_t pairs, const GroupWeight& g, cudaStream_t stream,
                               int num_sms) {
  if (g.group == 32) return launch_quant_scale<kSrc, 2>(src, pairs, g, stream, num_sms);
  if (g.group == 64) return launch_quant_scale<kSrc, 4>(src, pairs, g, stream, num_sms);
  return launch_quant_scale<kSrc, 8>(src, pairs, g, stream, num_sms);
}

template <int kOut>
cudaError_t launch_dequant(const GroupWeight& g, void* out, cudaStream_t stream, int num_sms) {
  const int64_t words = g.rows * g.cols / 8;
  const int shift = g.group == 32 ? 2 : g.group == 64 ? 3 : 4;
  const auto* packed = reinterpret_cast<const uint32_t*>(g.packed);
  const auto* scale = static_cast<const uint16_t*>(g.scale);
  const dim3 grid(grid_for(words, num_sms));
  const cudaError_t e = g.half ? launch_pdl(dequantize_groups_kernel<kOut, true>, grid, dim3(kThreads), 0, stream,
                                            packed, scale, g.zero, words, shift, out)
                               : launch_pdl(dequantize_groups_kernel<kOut, false>, grid, dim3(kThreads), 0, stream,
                                            packed, scale, g.zero, words, shift, out);
  count_launches(1);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_quantize_groups(const void* src, int src_dtype, const GroupWeight& g, cudaStream_t stream,
                                   int num_sms) {
  const int64_t pairs = g.rows * g.cols / 16;
  if (src_dtype == 0) return launch_quant_group<0>(src, pairs, g, stream, num_sms);
  if (src_dtype == 1) return launch_quant_group<1>(src, pairs, g, stream, num_sms);
  return launch_quant_group<2>(src, pairs, g, stream, num_sms);
}

cudaError_t launch_dequantize_groups(const GroupWeight& g, void* out, int out_dtype, cudaStream_t stream,
                                     int num_sms) {
  if (out_dtype == 0) return launch_dequant<0>(g, out, stream, num_sms);
  if (out_dtype == 1) return launch_dequant<1>(g, out, stream, num_sms);
  return launch_dequant<2>(g, out, stream, num_sms);
}

}  // namespace nf4
