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
//
// The kernel lives on bytes in flight: each warp keeps two steps of codes (1 KB each) loading in registers, and the
// scales of the tile's 16 rows -- contiguous in memory -- come as one coalesced copy into shared memory, already
// widened to (fp32 scale, packed bias + zero point), 256 groups at a time.
// The warps' sums are added in a fixed order, so results are deterministic.
//
// Measured (cold weights): 14336x4096 batch 1, groups of 128 12.1 us (2.5 TB/s, 39 % of the measured copy bandwidth);
// the loads alone take 7.3 us of it.  No pipe is full (57344x4096: ALU 54 %, L1 59 %, issue 58 %): a step's loads, the
// extraction of its codes (7 ALU operations and 4 packed subtractions per word) and its MMAs wait for one another.
// 4096x14336 fp16 11.3 us, 14336x4096 batch 8 in groups of 64 15.5 us, 32003x4128 in groups of 32 36 us; 1024x4096 4.1 us,
// most of it launch and latency.
#include "group.cuh"
#include "internal.h"

namespace nf4 {
namespace {

constexpr int kStep = 128;    // columns per warp step
constexpr int kChunk = 256;   // groups of scales in shared memory at a time

// (v & 0x000f000f) | bias in one LOP3
__device__ __forceinline__ uint32_t nibbles_or(uint32_t v, uint32_t bias) {
  uint32_t d;
  asm("lop3.b32 %0, %1, 0x000f000f, %2, 0xea;" : "=r"(d) : "r"(v), "r"(bias));
  return d;
}

// word of slot i (0..3) and lane t within a step, by group size
template <int kGroup>
__device__ __forceinline__ int slot_word(int i, int t) {
  return kGroup == 128 ? 4 * t + i : kGroup == 64 ? 8 * (i >> 1) + 2 * t + (i & 1) : 4 * i + t;
}

// codes of rows g and g + 8; `left`: columns from the step's first one to the row's end
template <int kGroup>
__device__ __forceinline__ void load_step(uint32_t (&w)[2][4], const uint8_t* __restrict__ p0,
                                          const uint8_t* __restrict__ p1, int left, int t) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint8_t* p = h ? p1 : p0;
    if constexpr (kGroup == 128) {
      const uint4 v = __ldcs(reinterpret_cast<const uint4*>(p) + t);
      w[h][0] = v.x;
      w[h][1] = v.y;
      w[h][2] = v.z;
      w[h][3] = v.w;
    } else if constexpr (kGroup == 64) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint2 v = 64 * j < left ? __ldcs(reinterpret_cast<const uint2*>(p) + 4 * j + t) : make_uint2(0, 0);
        w[h][2 * j] = v.x;
        w[h][2 * j + 1] = v.y;
      }
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        w[h][j] = 32 * j < left ? __ldcs(reinterpret_cast<const uint32_t*>(p) + 4 * j + t) : 0u;
    }
  }
}

template <bool kHalf, int kGroup, bool kZeros, int kWarps>
__global__ void __launch_bounds__(kWarps * 32)
    gemv_groups_kernel(const uint8_t* __restrict__ packed, const uint16_t* __restrict__ scale,
                       const uint8_t* __restrict__ zero, int64_t rows, int64_t cols, const uint16_t* __restrict__ x,
                       int batch, uint16_t* __restrict__ y, int pitch) {
  using G = GroupType<kHalf>;
  constexpr int kSub = kStep / kGroup, kSlots = 4 / kSub;  // groups per step, word slots per group
  __shared__ float red[kWarps][16][8];
  extern __shared__ float2 meta[];  // [16][pitch]: fp32 scale, packed bias + zero point
  pdl_launch_dependents();
  pdl_wait();
  uint32_t bias;  // kept in a register: as a constant beside the mask it would cost a second instruction per use
  asm volatile("mov.b32 %0, %1;" : "=r"(bias) : "n"(G::kBias));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int64_t tile = (int64_t)blockIdx.x * 16;
  const int64_t r0 = tile + g;
  // rows past the last one read it again; they are not written
  const int64_t ra = r0 < rows ? r0 : rows - 1, rb = r0 + 8 < rows ? r0 + 8 : rows - 1;
  const int groups = (int)(cols / kGroup);
  // A warp takes two neighbouring steps at a time (128 bytes of a row, a whole cache line), the warps in turn.  Its
  // pointers move on by a constant from pair to pair.
  constexpr int kPair = 2 * kStep, kTurn = kWarps * kPair;  // columns per pair, per turn of all warps
  const uint8_t* p0 = packed + ra * (cols / 2) + warp * (kPair / 2);
  const uint8_t* p1 = packed + rb * (cols / 2) + warp * (kPair / 2);
  int left = (int)cols - warp * kPair;  // columns from the pair's first one to the row's end (of the pair loaded next)
  // lanes past the batch read its last row again: their columns of the product are not written
  const uint16_t* xr = x + (int64_t)(g < batch ? g : batch - 1) * cols + 8 * slot_word<kGroup>(0, t) + warp * kPair;
  uint32_t buf[2][2][4];
  auto load = [&](int d) {
    if (d * kStep < left) load_step<kGroup>(buf[d], p0 + d * (kStep / 2), p1 + d * (kStep / 2), left - d * kStep, t);
  };
  load(0);
  load(1);

  float acc[4] = {0.f, 0.f, 0.f, 0.f};
  constexpr int kPerChunk = kChunk / (2 * kSub) / kWarps;  // pairs per warp and chunk of scales
  static_assert(kPerChunk > 0, "chunk");
  for (int c = 0; c < groups; c += kChunk) {
    const int gn = groups - c < kChunk ? groups - c : kChunk;
    if (c > 0) __syncthreads();
    for (int i = threadIdx.x; i < 16 * gn; i += kWarps * 32) {
      const int r = i / gn, j = i - r * gn;
      const int64_t at = (tile + r < rows ? tile + r : rows - 1) * groups + c + j;
      const float z = G::kBiasF + (kZeros ? (float)__ldg(zero + at) : 8.0f);
      meta[r * pitch + j] = make_float2(G::to_f32(__ldg(scale + at)), __uint_as_float(G::pack(z, z)));
    }
    __syncthreads();
    const float2* mp = meta + g * pitch + warp * (2 * kSub);
    int gl = gn - warp * (2 * kSub);  // groups of the chunk from the pair's first one on
#pragma unroll 1
    for (int q = 0; q < kPerChunk && gl > 0; ++q) {
      p0 += kTurn / 2;
      p1 += kTurn / 2;
      left -= kTurn;
#pragma unroll
      for (int d = 0; d < 2; ++d) {
        if (d * kSub < gl) {
#pragma unroll
          for (int j = 0; j < kSub; ++j) {
            if (kSub > 1 && d * kSub + j >= gl) break;  // the last step may be short by whole groups
            const float2 m0 = mp[d * kSub + j], m1 = mp[8 * pitch + d * kSub + j];
            const uint32_t z0 = __float_as_uint(m0.y), z1 = __float_as_uint(m1.y);
            float part[4];
#pragma unroll
            for (int s = j * kSlots; s < (j + 1) * kSlots; ++s) {
              const uint4 xv = __ldg(reinterpret_cast<const uint4*>(xr + d * kStep + 8 * slot_word<kGroup>(s, 0)));
              uint32_t a[2][4];
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const uint32_t w = buf[d][h][s], z = h ? z1 : z0;
#pragma unroll
                for (int p = 0; p < 4; ++p) a[h][p] = G::sub2(nibbles_or(w >> (4 * p), bias), z);
              }
              if (s == j * kSlots)
                G::mma(part, a[0][0], a[1][0], a[0][1], a[1][1], xv.x, xv.y, 0.f, 0.f, 0.f, 0.f);
              else
                G::mma(part, a[0][0], a[1][0], a[0][1], a[1][1], xv.x, xv.y, part[0], part[1], part[2], part[3]);
              G::mma(part, a[0][2], a[1][2], a[0][3], a[1][3], xv.z, xv.w, part[0], part[1], part[2], part[3]);
            }
            acc[0] = fmaf(m0.x, part[0], acc[0]);
            acc[1] = fmaf(m0.x, part[1], acc[1]);
            acc[2] = fmaf(m1.x, part[2], acc[2]);
            acc[3] = fmaf(m1.x, part[3], acc[3]);
          }
        }
        load(d);
      }
      xr += kTurn;
      mp += kWarps * 2 * kSub;
      gl -= kWarps * 2 * kSub;
    }
  }
  // accumulator fragment: (row g, batch 2t), (g, 2t + 1), (g + 8, 2t), (g + 8, 2t + 1)
  red[warp][g][2 * t] = acc[0];
  red[warp][g][2 * t + 1] = acc[1];
  red[warp][g + 8][2 * t] = acc[2];
  red[warp][g + 8][2 * t + 1] = acc[3];
  __syncthreads();
  const int r = threadIdx.x & 15, b = threadIdx.x >> 4;
  if (b < batch && tile + r < rows) {
    float sum = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) sum += red[w][r][b];
    y[(int64_t)b * rows + tile + r] = (uint16_t)(G::pack(sum, 0.0f) & 0xffffu);
  }
}

template <bool kHalf, int kGroup, int kWarps>
cudaError_t launch_shape(const GroupWeight& w, const void* x, int batch, void* y, cudaStream_t stream) {
  static_assert(kWarps * 32 >= 16 * 8, "a thread per output of the tile");
  const dim3 grid((unsigned)((w.rows + 15) / 16)), block(kWarps * 32);
  const auto* scale = static_cast<const uint16_t*>(w.scale);
  const auto* xs = static_cast<const uint16_t*>(x);
  auto* ys = static_cast<uint16_t*>(y);
  const int64_t groups = w.cols / kGroup;
  // an odd pitch spreads the eight rows that a warp reads at once over the banks
  const int pitch = (int)(groups < kChunk ? groups : kChunk) | 1;
  const size_t smem = (size_t)16 * pitch * sizeof(float2);
  const cudaError_t e =
      w.zero != nullptr
          ? launch_pdl(gemv_groups_kernel<kHalf, kGroup, true, kWarps>, grid, block, smem, stream, w.packed,
                       scale, w.zero, w.rows, w.cols, xs, batch, ys, pitch)
          : launch_pdl(gemv_groups_kernel<kHalf, kGroup, false, kWarps>, grid, block, smem, stream, w.packed,
                       scale, w.zero, w.rows, w.cols, xs, batch, ys, pitch);
  count_launches(1);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <bool kHalf, int kGroup>
cudaError_t launch(const GroupWeight& w, const void* x, int batch, void* y, cudaStream_t stream, int num_sms) {
  // Few tiles: sixteen warps share a tile's columns (4096x14336 batch 1: 11.6 us against 14.0 with eight).  Many: eight,
  // so that more tiles are under way on an SM (14336x4096 batch 1: 12.6 us against 13.8, batch 8 in groups of 64: 15.9
  // against 18.2).
  return (w.rows + 15) / 16 <= 2 * (int64_t)num_sms ? launch_shape<kHalf, kGroup, 16>(w, x, batch, y, stream)
                                                    : launch_shape<kHalf, kGroup, 8>(w, x, batch, y, stream);
}

template <bool kHalf>
cudaError_t launch_group_size(const GroupWeight& w, const void* x, int batch, void* y, cudaStream_t stream,
                              int num_sms) {
  if (w.group == 32) return launch<kHalf, 32>(w, x, batch, y, stream, num_sms);
  if (w.group == 64) return launch<kHalf, 64>(w, x, batch, y, stream, num_sms);
  return launch<kHalf, 128>(w, x, batch, y, stream, num_sms);
}

}  // namespace

cudaError_t launch_gemv_groups(const GroupWeight& w, const void* x, int batch, void* y, cudaStream_t stream,
                               int num_sms) {
  if ((w.rows + 15) / 16 > INT32_MAX) return cudaErrorInvalidValue;
  return w.half ? launch_group_size<true>(w, x, batch, y, stream, num_sms)
                : launch_group_size<false>(w, x, batch, y, stream, num_sms);
}

}  // namespace nf4
