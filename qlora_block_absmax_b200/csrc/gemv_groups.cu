// gemv_groups.cu -- decode product (batch 1..8) with 4-bit codes and group scales.
//
//   y[b, n] = T( sum_g s[n, g] * sum_{k in g} (q[n, k] - z[n, g]) x[b, k] )
// The inner sums run on mma.sync m16n8k16 with the weights as A (16 rows) and the activations as B (batch on N): the
// operand q - z is an integer of at most 4 bits, exact in either 16-bit type, and each product with x is exact in
// fp32; the scale is applied to the group's fp32 sum.  No weight is rounded.
//
// One CTA = one 16-row tile, its warps taking 128-column steps in turn.  Lane (g, t) = (lane / 4, lane % 4) holds the
// words of rows g and g + 8.  An MMA reduces over the four lanes t, so all four have to hold the same group: at a
// group of 128 each lane takes four consecutive words of the step, at 64 two and two, at 32 single words four apart.
// The order of k inside an MMA is free as long as both operands use the same one: a word's pairs (0,1), (2,3) feed one
// MMA and (4,5), (6,7) the next, against 16 contiguous bytes of x.
// The warps' sums are added in a fixed order, so results are deterministic.
#include "group.cuh"
#include "internal.h"

namespace nf4 {
namespace {

constexpr int kWarps = 4;
constexpr int kStep = 128;  // columns per warp step

// word of slot i (0..3) and lane t within a step, by group size
template <int kGroup>
__device__ __forceinline__ int slot_word(int i, int t) {
  return kGroup == 128 ? 4 * t + i : kGroup == 64 ? 8 * (i >> 1) + 2 * t + (i & 1) : 4 * i + t;
}

template <int kGroup>
struct Step {
  static constexpr int kSub = kStep / kGroup;  // groups per step
  uint32_t w[2][4];       // words of rows g, g + 8
  uint16_t s[2][kSub];    // scales
  uint8_t z[2][kSub];     // zero points
};

template <int kGroup, bool kZeros>
__device__ __forceinline__ void load_step(Step<kGroup>& d, const uint8_t* __restrict__ packed,
                                          const uint16_t* __restrict__ scale, const uint8_t* __restrict__ zero,
                                          const int64_t (&row)[2], int64_t cols, int64_t st, int t) {
  constexpr int kSub = Step<kGroup>::kSub;
  const int64_t groups = cols / kGroup;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint8_t* p = packed + row[h] * (cols / 2) + st * (kStep / 2);
#pragma unroll
    for (int j = 0; j < kSub; ++j) {
      const bool ok = st * kSub + j < groups;  // the last step may be short by whole groups
      if constexpr (kGroup == 128) {
        const uint4 v = ok ? __ldcs(reinterpret_cast<const uint4*>(p) + t) : make_uint4(0, 0, 0, 0);
        d.w[h][0] = v.x;
        d.w[h][1] = v.y;
        d.w[h][2] = v.z;
        d.w[h][3] = v.w;
      } else if constexpr (kGroup == 64) {
        const uint2 v = ok ? __ldcs(reinterpret_cast<const uint2*>(p) + 4 * j + t) : make_uint2(0, 0);
        d.w[h][2 * j] = v.x;
        d.w[h][2 * j + 1] = v.y;
      } else {
        d.w[h][j] = ok ? __ldcs(reinterpret_cast<const uint32_t*>(p) + 4 * j + t) : 0u;
      }
      const int64_t gi = row[h] * groups + st * kSub + j;
      d.s[h][j] = ok ? __ldg(scale + gi) : (uint16_t)0;
      d.z[h][j] = kZeros && ok ? __ldg(zero + gi) : (uint8_t)8;
    }
  }
}

template <bool kHalf, int kGroup, bool kZeros>
__global__ void __launch_bounds__(kWarps * 32)
    gemv_groups_kernel(const uint8_t* __restrict__ packed, const uint16_t* __restrict__ scale,
                       const uint8_t* __restrict__ zero, int64_t rows, int64_t cols, const uint16_t* __restrict__ x,
                       int batch, uint16_t* __restrict__ y) {
  using G = GroupType<kHalf>;
  constexpr int kSub = Step<kGroup>::kSub, kSlots = 4 / kSub;  // word slots per group
  __shared__ float red[kWarps][16][8];
  pdl_launch_dependents();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int64_t r0 = (int64_t)blockIdx.x * 16 + g;
  // rows past the last one read it again; they are not written
  const int64_t row[2] = {r0 < rows ? r0 : rows - 1, r0 + 8 < rows ? r0 + 8 : rows - 1};
  const int64_t nsteps = (cols + kStep - 1) / kStep;
  const uint16_t* xr = x + (int64_t)g * cols;
  float acc[4] = {0.f, 0.f, 0.f, 0.f};
  Step<kGroup> cur, nxt;
  if (warp < nsteps) load_step<kGroup, kZeros>(cur, packed, scale, zero, row, cols, warp, t);
  for (int64_t st = warp; st < nsteps; st += kWarps) {
    if (st + kWarps < nsteps) load_step<kGroup, kZeros>(nxt, packed, scale, zero, row, cols, st + kWarps, t);
#pragma unroll
    for (int j = 0; j < kSub; ++j) {
      const uint32_t z0 = G::pack(G::kBiasF + (float)cur.z[0][j], G::kBiasF + (float)cur.z[0][j]);
      const uint32_t z1 = G::pack(G::kBiasF + (float)cur.z[1][j], G::kBiasF + (float)cur.z[1][j]);
      float part[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = j * kSlots; i < (j + 1) * kSlots; ++i) {
        const int64_t k = st * kStep + 8 * slot_word<kGroup>(i, t);
        uint4 xv = make_uint4(0, 0, 0, 0);
        if (g < batch && k < cols) xv = __ldg(reinterpret_cast<const uint4*>(xr + k));
        uint32_t a[2][4];
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          a[0][p] = G::sub2(((cur.w[0][i] >> (4 * p)) & 0x000f000fu) | G::kBias, z0);
          a[1][p] = G::sub2(((cur.w[1][i] >> (4 * p)) & 0x000f000fu) | G::kBias, z1);
        }
        G::mma(part, a[0][0], a[1][0], a[0][1], a[1][1], xv.x, xv.y);
        G::mma(part, a[0][2], a[1][2], a[0][3], a[1][3], xv.z, xv.w);
      }
      const float s0 = G::to_f32(cur.s[0][j]), s1 = G::to_f32(cur.s[1][j]);
      acc[0] = fmaf(s0, part[0], acc[0]);
      acc[1] = fmaf(s0, part[1], acc[1]);
      acc[2] = fmaf(s1, part[2], acc[2]);
      acc[3] = fmaf(s1, part[3], acc[3]);
    }
    cur = nxt;
  }
  // accumulator fragment: (row g, batch 2t), (g, 2t + 1), (g + 8, 2t), (g + 8, 2t + 1)
  red[warp][g][2 * t] = acc[0];
  red[warp][g][2 * t + 1] = acc[1];
  red[warp][g + 8][2 * t] = acc[2];
  red[warp][g + 8][2 * t + 1] = acc[3];
  __syncthreads();
  const int r = threadIdx.x & 15, b = threadIdx.x >> 4;
  const int64_t n = (int64_t)blockIdx.x * 16 + r;
  if (b < batch && n < rows) {
    float sum = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) sum += red[w][r][b];
    y[(int64_t)b * rows + n] = (uint16_t)(G::pack(sum, 0.0f) & 0xffffu);
  }
}
static_assert(kWarps * 32 == 16 * 8, "one thread per output of the tile");

template <bool kHalf, int kGroup>
cudaError_t launch(const GroupWeight& w, const void* x, int batch, void* y, cudaStream_t stream) {
  const dim3 grid((unsigned)((w.rows + 15) / 16)), block(kWarps * 32);
  const auto* scale = static_cast<const uint16_t*>(w.scale);
  const auto* xs = static_cast<const uint16_t*>(x);
  auto* ys = static_cast<uint16_t*>(y);
  const cudaError_t e =
      w.zero != nullptr ? launch_pdl(gemv_groups_kernel<kHalf, kGroup, true>, grid, block, 0, stream, w.packed, scale,
                                     w.zero, w.rows, w.cols, xs, batch, ys)
                        : launch_pdl(gemv_groups_kernel<kHalf, kGroup, false>, grid, block, 0, stream, w.packed, scale,
                                     w.zero, w.rows, w.cols, xs, batch, ys);
  count_launches(1);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <bool kHalf>
cudaError_t launch_group_size(const GroupWeight& w, const void* x, int batch, void* y, cudaStream_t stream) {
  if (w.group == 32) return launch<kHalf, 32>(w, x, batch, y, stream);
  if (w.group == 64) return launch<kHalf, 64>(w, x, batch, y, stream);
  return launch<kHalf, 128>(w, x, batch, y, stream);
}

}  // namespace

cudaError_t launch_gemv_groups(const GroupWeight& w, const void* x, int batch, void* y, cudaStream_t stream,
                               int num_sms) {
  (void)num_sms;
  if ((w.rows + 15) / 16 > INT32_MAX) return cudaErrorInvalidValue;
  return w.half ? launch_group_size<true>(w, x, batch, y, stream) : launch_group_size<false>(w, x, batch, y, stream);
}

}  // namespace nf4
