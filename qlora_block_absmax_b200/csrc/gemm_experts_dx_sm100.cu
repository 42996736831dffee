// gemm_experts_dx_sm100.cu -- input gradient of the expert products, on tcgen05 tensor cores.
//
//   dX[t, k] = bf16_rn( sum_n dY[t, n] * Wc[e * N + n, k] )   for offsets[e] <= t < offsets[e + 1]
// with the same Wc as the forward product (gemm_experts_sm100.cu), accumulated in fp32: the loss gradient passing
// through frozen 4-bit experts on its way to the adapters and the layers below ("bitsandbytes",
// ozercemkelahmet.com/tools, "Strengths and limitations").
//
// The packed weight is read as it lies: a stage is 64 weight rows n (the reduction) x 128 columns k (the output tile).
// Producer thread (r, h) decodes one level-1 block, row r, columns 64 h .., and writes it as one 128-byte row of an
// MN-major, 128-byte-swizzled shared-memory tile, so the MMA reads Wc^T without a transpose pass:
//   A = Wc^T tile [128 k (UMMA M, MN-major)] x [64 n], B = dY tile [up to TM rows] x [64 n] (TMA), D in TMEM.
// Two accumulators: one tile's epilogue runs beside the next tile's MMAs.  Warp roles as in the forward product.
#include <cuda.h>

#include <atomic>

#include "experts.cuh"

namespace nf4 {
namespace {

using namespace experts;

constexpr int kTileR = 64;  // weight rows (reduction) per stage
constexpr int kGroups = 4;
constexpr int kWHalf = kTileR * 32;  // one level-1 block of codes per row
constexpr int kWBytes = 2 * kWHalf;  // packed codes of a stage: two blocks per row
constexpr int kABytes = kTileR * kTileN * 2;
constexpr int kProdWarp0 = kEpiWarps;
constexpr int kTmaWarp = kProdWarp0 + 4 * kGroups;
constexpr int kMmaWarp = kTmaWarp + 1;
constexpr int kTmaWWarp = kTmaWarp + 2;
constexpr int kThreads = (kTmaWWarp + 1) * 32;

// A-tile layout (MN-major, 128-byte swizzle): reduction row r, column e (k) at
//   (r / 8) * kKGroup + (e / 64) * kMnAtom + (r % 8) * 128 + (((e % 64) / 8) ^ (r % 8)) * 16 + (e % 8) * 2
constexpr uint32_t kMnAtom = 1024;
constexpr uint32_t kKGroup = 2048;

// TM: widest activation tile, 256, or 64 for few rows per expert (smaller stages leave room for a deeper code ring)
template <int TM>
struct Cfg {
  static constexpr int kStages = TM == 256 ? 4 : 6;    // operand ring: dY tile + decoded tile
  static constexpr int kWStages = TM == 256 ? 4 : 12;  // packed codes
  static constexpr int kBBytes = TM * kTileR * 2;
  static constexpr int kRingBytes = kStages * (kBBytes + kABytes) + kWStages * kWBytes;
  static constexpr int kTmemCols = 2 * TM;  // two accumulators
  // as in the forward product: the operand ring empties in order, code loads may land out of order
  static_assert(kStages >= kGroups && kWStages % kGroups == 0, "rings and producer groups");
};

template <int TM>
struct Smem {
  uint64_t wfull[Cfg<TM>::kWStages];
  uint64_t wempty[Cfg<TM>::kWStages];
  uint64_t full[Cfg<TM>::kStages];
  uint64_t empty[Cfg<TM>::kStages];
  uint64_t acc_full[2], acc_empty[2];
  uint32_t tmem_base;
  int abort;
  float unit_lut[256];
  Schedule sc;
};

template <int TM>
constexpr size_t smem_bytes() {
  return (size_t)Cfg<TM>::kRingBytes + kEpiWarps * kOutBytes + sizeof(Smem<TM>) + 1024;
}
static_assert(smem_bytes<256>() <= 232448 && smem_bytes<64>() <= 232448, "shared memory per CTA");

template <bool kDQ, int kBook, int TM>
__global__ void __launch_bounds__(kThreads, 1)
    gemm_experts_dx_kernel(Scales s, const int* __restrict__ offsets, int experts, int rows, int cols, int m_total,
                        const __grid_constant__ CUtensorMap ymap64, const __grid_constant__ CUtensorMap ymap16,
                        const __grid_constant__ CUtensorMap wmap, __nv_bfloat16* __restrict__ dx, unsigned* err) {
  using C = Cfg<TM>;
  constexpr int kStages = C::kStages, kWStages = C::kWStages;
  extern __shared__ uint8_t smem_raw[];
  pdl_launch_dependents();
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw);
  const uint32_t b_smem0 = base, a_smem0 = b_smem0 + kStages * C::kBBytes, w_smem0 = a_smem0 + kStages * kABytes;
  uint8_t* a_gen0 = gbase + kStages * C::kBBytes;
  const uint8_t* w_gen0 = a_gen0 + kStages * kABytes;
  uint8_t* out_stage = gbase + C::kRingBytes;
  auto* sm = reinterpret_cast<Smem<TM>*>(out_stage + kEpiWarps * kOutBytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kWStages; ++i) {
      mbar_init(&sm->wfull[i], 1);
      mbar_init(&sm->wempty[i], 4);
    }
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&sm->full[i], 1 + 4);
      mbar_init(&sm->empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm->acc_full[i], 1);
      mbar_init(&sm->acc_empty[i], kEpiWarps);
    }
    sm->abort = 0;
    fence_mbar_init();
  }
  if (kDQ && threadIdx.x < 256) sm->unit_lut[threadIdx.x] = dq_unit(threadIdx.x, s.dq_code);
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&sm->tmem_base)),
                 "r"(C::kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  pdl_wait();
  build_schedule<TM>(&sm->sc, offsets, experts, m_total, cols / kTileN);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm->tmem_base;
  const int units = sm->sc.first[experts], kps = rows / kTileR;

  if (warp >= kProdWarp0 && warp < kTmaWarp) {
    // ------------------------------------------------ producers
    const int group = (warp - kProdWarp0) >> 2;
    const int p = ((warp - kProdWarp0) & 3) * 32 + lane;
    const int r = p & (kTileR - 1), h = p >> 6;  // weight row within the stage, 64-column half of the output tile
    const int64_t rb = cols / kBlock;
    // this thread's 128-byte row of the A tile
    const uint32_t a_row = (uint32_t)(r >> 3) * kKGroup + (uint32_t)h * kMnAtom + (uint32_t)(r & 7) * 128u;
    const float mu = kDQ ? __ldg(s.mean) : 0.0f;
    const DecodeMul dm = decode_mul();
    uint32_t it = group;
    int u = blockIdx.x, ks = group;
    int64_t block0 = 0;  // level-1 block of this thread in the unit's first stage
    auto settle = [&]() {  // move (u, ks) to the unit that holds the stage
      while (ks >= kps && u < units) {
        ks -= kps;
        u += gridDim.x;
      }
      if (u < units) {
        const Unit t = unit_at<TM>(&sm->sc, experts, u);
        block0 = ((int64_t)t.expert * rows + r) * rb + t.n0 / kBlock + h;
      }
    };
    settle();
    uint32_t code = 0;  // the stage's scale, loaded one of this group's stages ahead
    float scale = 0.0f;
    auto load_scale = [&]() {
      if (u >= units) return;
      const int64_t b = block0 + (int64_t)ks * kTileR * rb;
      if (kDQ) {
        code = __ldg(s.q + b);
        scale = __ldg(s.scale + b / kDqBlock);
      } else {
        scale = __ldg(s.absmax + b);
      }
    };
    load_scale();
    while (u < units) {
      const int ws = it % kWStages, as = it % kStages;
      const uint32_t wph = (it / kWStages) & 1, aph = (it / kStages) & 1;
      const float a = kDQ ? dq_absmax(sm->unit_lut[code], scale, mu) : scale;
      ks += kGroups;
      if (ks >= kps) settle();
      load_scale();
      if (!wait_or_abort(&sm->wfull[ws], wph, sm, err)) break;
      const uint4* wsrc = reinterpret_cast<const uint4*>(w_gen0 + ws * kWBytes + h * kWHalf + r * 32);
      const uint4 w0 = wsrc[0], w1 = wsrc[1];
      fence_proxy_async_smem();  // the slot is refilled by TMA after these reads
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm->wempty[ws]);
      const Table T = make_table<kBook>(a);
      const uint32_t words[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
      uint32_t q[32];  // columns 2j, 2j + 1 of the row as bf16x2
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        uint32_t d[4];
        decode_word(words[c], T, d, dm);
        q[4 * c] = d[0];
        q[4 * c + 1] = d[1];
        q[4 * c + 2] = d[2];
        q[4 * c + 3] = d[3];
      }
      if (!wait_or_abort(&sm->empty[as], aph ^ 1, sm, err)) break;  // the MMAs left this slot
      uint8_t* arow = a_gen0 + as * kABytes + a_row;
#pragma unroll
      for (int c = 0; c < 8; ++c)
        *reinterpret_cast<uint4*>(arow + ((uint32_t)(c ^ (r & 7)) << 4)) =
            make_uint4(q[4 * c], q[4 * c + 1], q[4 * c + 2], q[4 * c + 3]);
      fence_proxy_async_smem();  // generic-proxy writes, read by the tensor cores (async proxy)
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm->full[as]);
      it += kGroups;
    }
  } else if (warp == kTmaWarp) {
    // ------------------------------------------------ TMA: dY tiles
    if (lane == 0) {
      uint32_t it = 0;
      bool ok = true;
      for (int u = blockIdx.x; u < units && ok; u += gridDim.x) {
        const Unit t = unit_at<TM>(&sm->sc, experts, u);
        for (int ks = 0; ks < kps; ++ks, ++it) {
          const int as = it % kStages;
          ok = wait_or_abort(&sm->empty[as], ((it / kStages) & 1) ^ 1, sm, err);
          if (!ok) break;
          mbar_expect_tx(&sm->full[as], (uint32_t)t.width * kTileR * 2);
          load_rows(b_smem0 + as * C::kBBytes, &ymap64, &ymap16, ks * kTileR, t.m0, t.width, &sm->full[as]);
        }
      }
      for (uint32_t j = (it > kStages ? it - kStages : 0); j < it; ++j)  // drain the copies still in flight
        if (!mbar_wait_bounded(&sm->full[j % kStages], (j / kStages) & 1, err)) break;
    }
  } else if (warp == kTmaWWarp) {
    // ------------------------------------------------ TMA: packed codes
    if (lane == 0) {
      uint32_t it = 0;
      bool ok = true;
      for (int u = blockIdx.x; u < units && ok; u += gridDim.x) {
        const Unit t = unit_at<TM>(&sm->sc, experts, u);
        const int n = t.expert * rows;
        for (int ks = 0; ks < kps; ++ks, ++it) {
          const int ws = it % kWStages;
          ok = wait_or_abort(&sm->wempty[ws], ((it / kWStages) & 1) ^ 1, sm, err);
          if (!ok) break;
          mbar_expect_tx(&sm->wfull[ws], kWBytes);
          // columns n0 .. n0 + 63 and n0 + 64 .. n0 + 127 of 64 rows (32 bytes each)
          tma_load_2d(w_smem0 + ws * kWBytes, &wmap, t.n0 / 2, n + ks * kTileR, &sm->wfull[ws]);
          tma_load_2d(w_smem0 + ws * kWBytes + kWHalf, &wmap, t.n0 / 2 + 32, n + ks * kTileR, &sm->wfull[ws]);
        }
      }
      for (uint32_t j = (it > kWStages ? it - kWStages : 0); j < it; ++j)
        if (!mbar_wait_bounded(&sm->wfull[j % kWStages], (j / kWStages) & 1, err)) break;
    }
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------ MMA issuer
    if (lane == 0) {
      uint32_t it = 0, ucount = 0;
      bool ok = true;
      for (int u = blockIdx.x; u < units && ok; u += gridDim.x, ++ucount) {
        const uint32_t idesc = instr_desc(kTileN, unit_at<TM>(&sm->sc, experts, u).width, /*a_mn=*/true);
        const int acc = ucount & 1;
        ok = wait_or_abort(&sm->acc_empty[acc], ((ucount >> 1) & 1) ^ 1, sm, err);
        if (!ok) break;
        tc_fence_after();
        for (int ks = 0; ks < kps; ++ks, ++it) {
          const int as = it % kStages;
          ok = wait_or_abort(&sm->full[as], (it / kStages) & 1, sm, err);
          if (!ok) break;
          tc_fence_after();
          const uint32_t a_addr = a_smem0 + as * kABytes, b_addr = b_smem0 + as * C::kBBytes;
#pragma unroll
          for (int kk = 0; kk < kTileR / 16; ++kk)
            tc_mma_ss(tmem + acc * TM, smem_desc_mn_sw128(a_addr + kk * 2 * kKGroup, kMnAtom, kKGroup),
                      smem_desc_sw128(b_addr + kk * 32), idesc, (ks | kk) != 0);
          tc_commit(&sm->empty[as]);
        }
        if (ok) tc_commit(&sm->acc_full[acc]);
      }
    }
  } else if (warp < kEpiWarps) {
    // ------------------------------------------------ epilogue
    uint32_t ucount = 0;
    for (int u = blockIdx.x; u < units; u += gridDim.x, ++ucount) {
      const Unit t = unit_at<TM>(&sm->sc, experts, u);
      const int acc = ucount & 1;
      if (!wait_or_abort(&sm->acc_full[acc], (ucount >> 1) & 1, sm, err)) break;
      tc_fence_after();
      store_unit(t.n0, t.m0, t.m1, t.width, tmem + ((uint32_t)(warp * 32) << 16) + acc * TM, out_stage, dx, cols,
                 [&]() { mbar_arrive(&sm->acc_empty[acc]); });
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(C::kTmemCols) : "memory");
  }
}

template <bool kDQ, int kBook, int TM>
cudaError_t launch(const ExpertsCall& c, const CUtensorMap& y64, const CUtensorMap& y16, const CUtensorMap& wmap,
                   int grid, unsigned* err, cudaStream_t stream) {
  constexpr size_t smem = smem_bytes<TM>();
  static std::atomic<uint64_t> attr_done{0};  // shared-memory opt-in, once per device
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!(attr_done.load() & (1ull << dev))) {
    const cudaError_t e = cudaFuncSetAttribute(gemm_experts_dx_kernel<kDQ, kBook, TM>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    attr_done.fetch_or(1ull << dev);
  }
  const cudaError_t e =
      launch_pdl(gemm_experts_dx_kernel<kDQ, kBook, TM>, dim3(grid), dim3(kThreads), smem, stream, c.scales, c.offsets,
                 c.experts, (int)c.rows, (int)c.cols, (int)c.m, y64, y16, wmap, static_cast<__nv_bfloat16*>(c.out), err);
  count_launches(1);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <int TM>
cudaError_t launch_form(const ExpertsCall& c, const CUtensorMap& y64, const CUtensorMap& y16, const CUtensorMap& wmap,
                        int grid, unsigned* err, cudaStream_t stream) {
  const bool dq = c.scales.absmax == nullptr;
  if (dq)
    return c.scales.book ? launch<true, 1, TM>(c, y64, y16, wmap, grid, err, stream)
                         : launch<true, 0, TM>(c, y64, y16, wmap, grid, err, stream);
  return c.scales.book ? launch<false, 1, TM>(c, y64, y16, wmap, grid, err, stream)
                       : launch<false, 0, TM>(c, y64, y16, wmap, grid, err, stream);
}

}  // namespace

cudaError_t launch_gemm_experts_dx(const ExpertsCall& c, unsigned* err, cudaStream_t stream, int num_sms) {
  CUtensorMap y64, y16, wmap;
  if (!make_map(&y64, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, c.in, c.rows, c.m, kTileR, 64, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !make_map(&y16, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, c.in, c.rows, c.m, kTileR, 16, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !make_map(&wmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, c.packed, c.cols / 2, c.rows * c.experts, 32, kTileR,
                CU_TENSOR_MAP_SWIZZLE_NONE))
    return cudaErrorNotSupported;
  // no more units than the row tiles that m rows can make, each with all column tiles
  const bool wide = c.m > 64 * (int64_t)c.experts;
  const int64_t tm = wide ? 256 : 64;
  const int64_t tiles = (c.m < c.experts ? c.m : c.experts) + c.m / tm;
  const int64_t units = tiles * (c.cols / kTileN);
  const int grid = (int)(units < num_sms ? units : num_sms);
  return wide ? launch_form<256>(c, y64, y16, wmap, grid, err, stream)
              : launch_form<64>(c, y64, y16, wmap, grid, err, stream);
}

}  // namespace nf4
