// gemm_experts_sm100.cu -- the 4-bit matmul grouped by expert, on tcgen05 tensor cores.
//
//   Y[t, n] = bf16_rn( sum_k Wc[e * N + n, k] * X[t, k] )   for offsets[e] <= t < offsets[e + 1]
// with Wc = bf16_rn(RN(code * a)) as in the library's other products ("bitsandbytes", ozercemkelahmet.com/tools, "How
// it works" Step 5), accumulated in fp32: the linear layers of a mixture-of-experts block whose experts are 4-bit
// weights, each row going through the expert that its router chose.
//
// A work unit is a tile of 128 weight rows (UMMA M) x up to TM activation rows (UMMA N, the tile's own width) over the
// whole reduction, 128 columns (two level-1 blocks per weight row) per stage.  The weight tile is decoded by producer warps into TMEM (operand A), the
// activation tile comes by TMA (operand B), D[n, t] accumulates in TMEM.  Warp roles of the one persistent CTA per SM:
//   warps 0-3    epilogue
//   then 4 G     producers in G groups, each taking every G-th stage: thread p decodes row p of the stage's tile
//   next         TMA: activation tiles
//   next         TMEM allocator and MMA issuer (one thread)
//   last         TMA: packed codes
#include <cuda.h>

#include <atomic>

#include "experts.cuh"

namespace nf4 {
namespace {

using namespace experts;

// Reduction per stage.  The issuing thread pays about 350 cycles per stage for its barrier test, fences and commit
// besides some 50 per MMA; at 64 columns (four MMAs) that came to 600 cycles per stage, above the time in which the
// producers decode one.
constexpr int kTileK = 128;
constexpr int kHalfK = 64;  // one level-1 block per weight row, one 128-byte swizzle atom of activations
constexpr int kGroups = 4;
constexpr int kWBytes = kTileN * kTileK / 2;  // packed codes of a stage
constexpr int kProdWarp0 = kEpiWarps;
constexpr int kTmaWarp = kProdWarp0 + 4 * kGroups;
constexpr int kMmaWarp = kTmaWarp + 1;
constexpr int kTmaWWarp = kTmaWarp + 2;
constexpr int kThreads = (kTmaWWarp + 1) * 32;

// TM: widest activation tile, 128, or 64 for few rows per expert (smaller stages leave room for a deeper code ring)
template <int TM>
struct Cfg {
  static constexpr int kStages = TM == 128 ? 4 : 6;    // operand ring: activation tile + 64 TMEM columns of weights
  static constexpr int kWStages = TM == 128 ? 8 : 12;  // packed codes
  static constexpr int kAccs = 2;                      // accumulators: an epilogue runs beside the next tile
  static constexpr int kHalfB = TM * kHalfK * 2;
  static constexpr int kBBytes = 2 * kHalfB;
  static constexpr int kRingBytes = kStages * kBBytes + kWStages * kWBytes;
  static constexpr int kACol0 = kAccs * TM;  // first TMEM column of the decoded tiles
  static constexpr int kTmemCols = 512;
  static_assert(kACol0 + kStages * kTileK / 2 <= kTmemCols, "TMEM columns");
  // A parity wait tells two successive phases of a barrier apart, no more.  A group comes back to a ring kGroups
  // stages later: it must not reach a slot whose phase before the awaited one is still open.  The operand ring empties
  // in order, so kGroups stages suffice; code loads may land out of order, so each slot belongs to one group.
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
  return (size_t)Cfg<TM>::kRingBytes + kEpiWarps * kStageOutBytes + sizeof(Smem<TM>) + 1024;
}
static_assert(smem_bytes<128>() <= 232448 && smem_bytes<64>() <= 232448, "shared memory per CTA");

template <bool kDQ, int kBook, int TM>
__global__ void __launch_bounds__(kThreads, 1)
    gemm_experts_kernel(Scales s, const int* __restrict__ offsets, int experts, int rows, int cols, int m_total,
                        const __grid_constant__ CUtensorMap xmap64, const __grid_constant__ CUtensorMap xmap16,
                        const __grid_constant__ CUtensorMap wmap, __nv_bfloat16* __restrict__ y, unsigned* err) {
  using C = Cfg<TM>;
  constexpr int kStages = C::kStages, kWStages = C::kWStages;
  extern __shared__ uint8_t smem_raw[];
  pdl_launch_dependents();
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw);
  const uint32_t b_smem0 = base, w_smem0 = base + kStages * C::kBBytes;
  const uint8_t* w_gen0 = gbase + kStages * C::kBBytes;
  uint16_t* out_stage = reinterpret_cast<uint16_t*>(gbase + C::kRingBytes);
  auto* sm = reinterpret_cast<Smem<TM>*>(gbase + C::kRingBytes + kEpiWarps * kStageOutBytes);
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
  build_schedule<TM>(&sm->sc, offsets, experts, m_total, rows / kTileN);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm->tmem_base;
  const int units = sm->sc.first[experts], kps = (cols + kTileK - 1) / kTileK;
  const bool odd = cols % kTileK != 0;  // the last stage holds one block

  if (warp >= kProdWarp0 && warp < kTmaWarp) {
    // ------------------------------------------------ producers
    const int group = (warp - kProdWarp0) >> 2;
    const int p = ((warp - kProdWarp0) & 3) * 32 + lane;  // weight row within the tile
    const float mu = kDQ ? __ldg(s.mean) : 0.0f;
    const DecodeMul dm = decode_mul();
    uint32_t it = group;
    int u = blockIdx.x, ks = group;
    const int rb = cols / kBlock;
    int64_t block0 = 0;  // level-1 block of this thread's row at column 0
    auto settle = [&]() {  // move (u, ks) to the unit that holds the stage
      while (ks >= kps && u < units) {
        ks -= kps;
        u += gridDim.x;
      }
      if (u < units) {
        const Unit t = unit_at<TM>(&sm->sc, experts, u);
        block0 = ((int64_t)t.expert * rows + t.n0 + p) * rb;
      }
    };
    settle();
    uint32_t code[2] = {0, 0};  // the stage's scales, loaded one of this group's stages ahead
    float scale[2] = {0.0f, 0.0f};
    auto load_scale = [&]() {
      if (u >= units) return;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (h == 1 && 2 * ks + 1 >= rb) break;
        const int64_t b = block0 + 2 * ks + h;
        if (kDQ) {
          code[h] = __ldg(s.q + b);
          scale[h] = __ldg(s.scale + b / kDqBlock);
        } else {
          scale[h] = __ldg(s.absmax + b);
        }
      }
    };
    load_scale();
    bool ok = true;
    while (u < units && ok) {
      const int ws = it % kWStages, as = it % kStages;
      const uint32_t wph = (it / kWStages) & 1, aph = (it / kStages) & 1;
      float a[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) a[h] = kDQ ? dq_absmax(sm->unit_lut[code[h]], scale[h], mu) : scale[h];
      const int blocks = 2 * ks + 1 < rb ? 2 : 1;
      ks += kGroups;
      if (ks >= kps) settle();
      load_scale();
      ok = wait_or_abort(&sm->wfull[ws], wph, sm, err);
      if (!ok) break;
      const uint4* wsrc = reinterpret_cast<const uint4*>(w_gen0 + ws * kWBytes + p * (kTileK / 2));
      const uint32_t ta = tmem + ((uint32_t)((warp & 3) * 32) << 16) + (uint32_t)(C::kACol0 + as * (kTileK / 2));
#pragma unroll 1
      for (int h = 0; h < blocks; ++h) {
        // 64-byte swizzle: 16-byte piece c of row p lies at piece c ^ ((p / 2) % 4)
        const uint4 w0 = wsrc[(2 * h) ^ ((p >> 1) & 3)], w1 = wsrc[(2 * h + 1) ^ ((p >> 1) & 3)];
        if (h == blocks - 1) {
          fence_proxy_async_smem();  // the slot is refilled by TMA after these reads
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm->wempty[ws]);
        }
        const Table T = make_table<kBook>(h == 0 ? a[0] : a[1]);
        const uint32_t words[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
        uint32_t r[32];  // column j of the row: codes 2j, 2j + 1 as bf16x2
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          uint32_t d[4];
          decode_word(words[c], T, d, dm);
          r[4 * c] = d[0];
          r[4 * c + 1] = d[1];
          r[4 * c + 2] = d[2];
          r[4 * c + 3] = d[3];
        }
        if (h == 0) ok = wait_or_abort(&sm->empty[as], aph ^ 1, sm, err);  // the MMAs left this slot
        if (!ok) break;
        tmem_st32(ta + h * (kHalfK / 2), r);
      }
      if (!ok) break;
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm->full[as]);
      it += kGroups;
    }
  } else if (warp == kTmaWarp) {
    // ------------------------------------------------ TMA: activation tiles
    if (lane == 0) {
      uint32_t it = 0;
      bool ok = true;
      for (int u = blockIdx.x; u < units && ok; u += gridDim.x) {
        const Unit t = unit_at<TM>(&sm->sc, experts, u);
        for (int ks = 0; ks < kps; ++ks, ++it) {
          const int as = it % kStages;
          ok = wait_or_abort(&sm->empty[as], ((it / kStages) & 1) ^ 1, sm, err);
          if (!ok) break;
          const int halves = odd && ks == kps - 1 ? 1 : 2;
          mbar_expect_tx(&sm->full[as], (uint32_t)(t.width * halves) * kHalfK * 2);
          for (int h = 0; h < halves; ++h)
            load_rows(b_smem0 + as * C::kBBytes + h * C::kHalfB, &xmap64, &xmap16, ks * kTileK + h * kHalfK, t.m0,
                      t.width, &sm->full[as]);
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
        const int n = t.expert * rows + t.n0;
        for (int ks = 0; ks < kps; ++ks, ++it) {
          const int ws = it % kWStages;
          ok = wait_or_abort(&sm->wempty[ws], ((it / kWStages) & 1) ^ 1, sm, err);
          if (!ok) break;
          mbar_expect_tx(&sm->wfull[ws], kWBytes);
          tma_load_2d(w_smem0 + ws * kWBytes, &wmap, ks * (kTileK / 2), n, &sm->wfull[ws]);
        }
      }
      for (uint32_t j = (it > kWStages ? it - kWStages : 0); j < it; ++j)
        if (!mbar_wait_bounded(&sm->wfull[j % kWStages], (j / kWStages) & 1, err)) break;
    }
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------ MMA issuer
    const uint32_t tm_u = __shfl_sync(0xffffffffu, tmem, 0);
    const uint64_t bdesc0 = smem_desc_sw128(b_smem0);
    uint32_t as = 0, ph = 0, ucount = 0;
    bool ok = true;
    for (int u = blockIdx.x; u < units && ok; u += gridDim.x, ++ucount) {
      const uint32_t idesc = instr_desc(kTileN, __shfl_sync(0xffffffffu, unit_at<TM>(&sm->sc, experts, u).width, 0));
      const uint32_t acc = ucount % C::kAccs;
      ok = wait_or_abort(&sm->acc_empty[acc], ((ucount / C::kAccs) & 1) ^ 1, sm, err);
      if (!ok) break;
      tc_fence_after();
      const uint32_t d_tm = tm_u + acc * TM;
      for (int ks = 0; ks < kps; ++ks) {
        ok = wait_or_abort(&sm->full[as], ph, sm, err);
        if (!ok) break;
        tc_fence_after();
        const uint32_t a_tm = tm_u + C::kACol0 + as * (kTileK / 2);
        const uint64_t bdesc = bdesc0 + as * (C::kBBytes >> 4);
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < kHalfK / 16; ++kk)
            tc_mma_ts(d_tm, a_tm + kk * 8, bdesc + kk * 2, idesc, (ks | kk) != 0);
          if (!odd || ks < kps - 1) {
#pragma unroll
            for (int kk = 0; kk < kHalfK / 16; ++kk)
              tc_mma_ts(d_tm, a_tm + kHalfK / 2 + kk * 8, bdesc + (C::kHalfB >> 4) + kk * 2, idesc, 1);
          }
          tc_commit(&sm->empty[as]);
        }
        __syncwarp();
        if (++as == kStages) {
          as = 0;
          ph ^= 1;
        }
      }
      if (ok && elect_one()) tc_commit(&sm->acc_full[acc]);
      __syncwarp();
    }
  } else if (warp < kEpiWarps) {
    // ------------------------------------------------ epilogue
    uint32_t ucount = 0;
    for (int u = blockIdx.x; u < units; u += gridDim.x, ++ucount) {
      const Unit t = unit_at<TM>(&sm->sc, experts, u);
      const uint32_t acc = ucount % C::kAccs;
      if (!wait_or_abort(&sm->acc_full[acc], (ucount / C::kAccs) & 1, sm, err)) break;
      tc_fence_after();
      store_unit(t, tmem + ((uint32_t)(warp * 32) << 16) + acc * TM, out_stage, sm, &sm->acc_empty[acc], y, rows);
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
cudaError_t launch(const ExpertsCall& c, const CUtensorMap& x64, const CUtensorMap& x16, const CUtensorMap& wmap,
                   int grid, unsigned* err, cudaStream_t stream) {
  constexpr size_t smem = smem_bytes<TM>();
  static std::atomic<uint64_t> attr_done{0};  // shared-memory opt-in, once per device
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!(attr_done.load() & (1ull << dev))) {
    const cudaError_t e = cudaFuncSetAttribute(gemm_experts_kernel<kDQ, kBook, TM>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    attr_done.fetch_or(1ull << dev);
  }
  const cudaError_t e =
      launch_pdl(gemm_experts_kernel<kDQ, kBook, TM>, dim3(grid), dim3(kThreads), smem, stream, c.scales, c.offsets,
                 c.experts, (int)c.rows, (int)c.cols, (int)c.m, x64, x16, wmap, static_cast<__nv_bfloat16*>(c.out), err);
  count_launches(1);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <int TM>
cudaError_t launch_form(const ExpertsCall& c, const CUtensorMap& x64, const CUtensorMap& x16, const CUtensorMap& wmap,
                        int grid, unsigned* err, cudaStream_t stream) {
  const bool dq = c.scales.absmax == nullptr;
  if (dq)
    return c.scales.book ? launch<true, 1, TM>(c, x64, x16, wmap, grid, err, stream)
                         : launch<true, 0, TM>(c, x64, x16, wmap, grid, err, stream);
  return c.scales.book ? launch<false, 1, TM>(c, x64, x16, wmap, grid, err, stream)
                       : launch<false, 0, TM>(c, x64, x16, wmap, grid, err, stream);
}

}  // namespace

cudaError_t launch_gemm_experts(const ExpertsCall& c, unsigned* err, cudaStream_t stream, int num_sms) {
  CUtensorMap x64, x16, wmap;
  if (!make_map(&x64, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, c.in, c.cols, c.m, kHalfK, 64, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !make_map(&x16, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, c.in, c.cols, c.m, kHalfK, 16, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !make_map(&wmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, c.packed, c.cols / 2, c.rows * c.experts, kTileK / 2, kTileN,
                CU_TENSOR_MAP_SWIZZLE_64B))
    return cudaErrorNotSupported;
  // no more units than the row tiles that m rows can make, each with all column tiles
  const bool wide = c.m > 64 * (int64_t)c.experts;
  const int64_t tm = wide ? 128 : 64;
  const int64_t tiles = (c.m < c.experts ? c.m : c.experts) + c.m / tm;
  const int64_t units = tiles * (c.rows / kTileN);
  const int grid = (int)(units < num_sms ? units : num_sms);
  return wide ? launch_form<128>(c, x64, x16, wmap, grid, err, stream)
              : launch_form<64>(c, x64, x16, wmap, grid, err, stream);
}

}  // namespace nf4
