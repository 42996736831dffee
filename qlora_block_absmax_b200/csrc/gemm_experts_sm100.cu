// gemm_experts_sm100.cu -- the 4-bit matmul grouped by expert, on tcgen05 tensor cores.
//
//   Y[t, n] = bf16_rn( sum_k Wc[e * N + n, k] * X[t, k] )   for offsets[e] <= t < offsets[e + 1]
// with Wc = bf16_rn(RN(code * a)) as in the library's other products ("bitsandbytes", ozercemkelahmet.com/tools, "How
// it works" Step 5), accumulated in fp32: the linear layers of a mixture-of-experts block whose experts are 4-bit
// weights, each row going through the expert that its router chose.
//
// A work unit is a tile of 128 weight rows (UMMA M; 256 for a pair of CTAs) x some activation rows (UMMA N, the tile's own
// width) over the whole reduction, 128 columns (two level-1 blocks per weight row) per stage.  The weight tile is decoded
// by producer warps into TMEM (operand A), the activation tile comes by TMA (operand B), D[n, t] accumulates in TMEM.  Warp
// roles of the one persistent CTA per SM:
//   warps 0-3    epilogue
//   then 16      producers in four groups, two per stage (one for each block), every other stage: thread p decodes row p
//   next         TMA: activation tiles
//   next         TMEM allocator and MMA issuer (the whole warp runs the loop, one lane issues)
//   last         TMA: packed codes
//
// What bounds it.  Few rows: the producers.  8 experts of 14336x4096, 16 rows take 86 us, 2.1 TB/s of codes and scales
// (32 % of the measured copy bandwidth): ~890 cycles per stage, of which the table lookups alone fill the shared-memory
// pipe for 512, the codes, the activation tile and the MMAs' reads of it for most of the rest.  Many rows: 4096 rows take
// 383 us in single launches (1254 TFLOP/s, 77 % of the measured burst rate), 440 to 450 us back to back, when the power
// limit holds the clock near 1.5 GHz; the tensor pipe is busy for 80 % of the cycles, the rest is the one accumulator.
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
constexpr int kGroups = 4;         // two per stage, one for each of its blocks
constexpr int kLanes = kGroups / 2;  // stages being decoded at a time
constexpr int kWBytes = kTileN * kTileK / 2;  // packed codes of a stage
constexpr int kProdWarp0 = kEpiWarps;
constexpr int kTmaWarp = kProdWarp0 + 4 * kGroups;
constexpr int kMmaWarp = kTmaWarp + 1;
constexpr int kTmaWWarp = kTmaWarp + 2;
constexpr int kThreads = (kTmaWWarp + 1) * 32;

// kPair: two CTAs share a tile of 256 weight rows x up to 256 activation rows (cta_group::2).  Each decodes its own 128
// weight rows and loads half of the activation rows, so an SM loads 20 KB instead of 36 KB per 64 columns of a 256-row
// tile; alone, a CTA with tiles of 256 rows was bound by those loads (790 cycles per 64 columns, 620 with a quarter of
// them).  Otherwise tiles of up to 64 rows, for few rows per expert: smaller stages leave room for deeper rings.
template <bool kPair>
struct Cfg {
  static constexpr int kTileM = kPair ? 256 : 64;       // activation rows per tile
  static constexpr int kRowsB = kPair ? 128 : 64;       // of them in one CTA's shared memory
  static constexpr int kTileCols = kPair ? 2 * kTileN : kTileN;
  static constexpr int kStages = kPair ? 3 : 6;         // operand ring: activation tile + 64 TMEM columns of weights
  static constexpr int kWStages = 6;                    // packed codes
  static constexpr int kAccs = kPair ? 1 : 2;           // two accumulators: an epilogue runs beside the next tile
  static constexpr int kHalfB = kRowsB * kHalfK * 2;
  static constexpr int kBBytes = 2 * kHalfB;
  static constexpr int kACol0 = kAccs * kTileM;  // first TMEM column of the decoded tiles
  static constexpr int kTmemCols = 512;
  static_assert(kACol0 + kStages * kTileK / 2 <= kTmemCols, "TMEM columns");
  // A parity wait tells two successive phases of a barrier apart, no more.  A group comes back to a ring kLanes
  // stages later: it must not reach a slot whose phase before the awaited one is still open.  The operand ring empties
  // in order, so kLanes stages suffice; code loads may land out of order, so each slot belongs to one pair of groups.
  static_assert(kStages >= kLanes && kWStages % kLanes == 0, "rings and producer groups");
};

template <bool kPair>
struct Smem {
  uint64_t wfull[Cfg<kPair>::kWStages];
  uint64_t wempty[Cfg<kPair>::kWStages];
  uint64_t full[Cfg<kPair>::kStages];       // activation tile landed, weight tile written
  uint64_t peer_full[Cfg<kPair>::kStages];  // (CTA 0 of a pair) the same in CTA 1, told by its MMA warp
  uint64_t empty[Cfg<kPair>::kStages];
  uint64_t acc_full[2], acc_empty[2];
  uint32_t tmem_base;
  int abort;
  float unit_lut[256];
  Schedule sc;
};

// Shared memory: the packed codes, the epilogue's staging and Smem before the pair table at 64 KB, the activation ring
// after it.  The window of a CTA without static shared memory starts at 1 KB (the kernel checks that all of it fits).
constexpr uint32_t kWindow = 1024;
template <bool kPair>
constexpr size_t smem_bytes() {
  return 2 * (size_t)kPairTable - kWindow + Cfg<kPair>::kStages * Cfg<kPair>::kBBytes;
}
template <bool kPair>
constexpr uint32_t front_bytes() {
  return Cfg<kPair>::kWStages * kWBytes + kEpiWarps * kOutBytes + (uint32_t)sizeof(Smem<kPair>);
}
static_assert(smem_bytes<true>() <= 232448 && smem_bytes<false>() <= 232448, "shared memory per CTA");
static_assert(kWindow + front_bytes<true>() <= kPairTable && kWindow + front_bytes<false>() <= kPairTable, "front part");

template <bool kDQ, int kBook, bool kPair>
__global__ void __launch_bounds__(kThreads, 1)
    gemm_experts_kernel(Scales s, const int* __restrict__ offsets, int experts, int rows, int cols, int m_total,
                        const __grid_constant__ CUtensorMap xmap, const __grid_constant__ CUtensorMap xmap16,
                        const __grid_constant__ CUtensorMap wmap, __nv_bfloat16* __restrict__ y, Split split, unsigned* err) {
  using C = Cfg<kPair>;
  constexpr int kStages = C::kStages, kWStages = C::kWStages;
  extern __shared__ uint8_t smem_raw[];
  pdl_launch_dependents();
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t cta = raw & 0xff000000u;  // in a cluster, a CTA's window lies at its rank's place
  const uint32_t front = (raw + 1023u) & ~1023u, table = cta + kPairTable;
  uint8_t* w_gen0 = smem_raw + (front - raw);
  const uint32_t w_smem0 = front, b_smem0 = table + kPairTable;
  uint8_t* out_stage = w_gen0 + kWStages * kWBytes;
  auto* sm = reinterpret_cast<Smem<kPair>*>(out_stage + kEpiWarps * kOutBytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = kPair ? (int)cluster_rank() : 0;
  // the items of this CTA (or pair): u0, u0 + du, ...
  const int u0 = kPair ? blockIdx.x >> 1 : blockIdx.x, du = kPair ? gridDim.x >> 1 : gridDim.x;
  if (front != cta + kWindow) {  // the window does not start at 1 KB: refuse, touch nothing
    if (threadIdx.x == 0) atomicOr(err, kErrTimeout);
    return;
  }

  if (threadIdx.x == 0) {
    for (int i = 0; i < kWStages; ++i) {
      mbar_init(&sm->wfull[i], 1);
      mbar_init(&sm->wempty[i], 8);
    }
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&sm->full[i], 1 + 8);
      mbar_init(&sm->peer_full[i], 1);
      mbar_init(&sm->empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm->acc_full[i], 1);
      mbar_init(&sm->acc_empty[i], kPair ? 2 * kEpiWarps : kEpiWarps);
    }
    sm->abort = 0;
    fence_mbar_init();
  }
  if (kDQ && threadIdx.x < 256) sm->unit_lut[threadIdx.x] = dq_unit(threadIdx.x, s.dq_code);
  if (warp == kMmaWarp) tmem_alloc<kPair>(&sm->tmem_base, C::kTmemCols);
  if (threadIdx.x == kTmaWarp * 32) {
    prefetch_map(&xmap);
    prefetch_map(&xmap16);
    prefetch_map(&wmap);
  }
  fill_pair_table<kBook>(smem_raw + (table - raw));
  pdl_wait();
  const int kps = (cols + kTileK - 1) / kTileK;
  build_schedule<C::kTileM>(&sm->sc, offsets, experts, m_total, (rows + C::kTileCols - 1) / C::kTileCols, kps,
                            !kPair && split.part != nullptr);
  tc_fence_before();
  __syncthreads();
  if constexpr (kPair) cluster_sync();  // the other CTA's barriers are initialised, its TMEM allocated
  tc_fence_after();
  const uint32_t tmem = sm->tmem_base;
  // Items: the whole units, then `splits` per unit of the rest, split i taking stages [i * kps / splits, ...).  Read from
  // shared memory where they are used, once per item: the producers have no registers to spare for them.
  const bool odd = cols % kTileK != 0;  // the last stage holds one block
  const volatile Schedule* const sv = &sm->sc;
  const int items = sv->items;
  auto first_stage = [&](int w) {
    if (kPair) return 0;
    const int r = w - sv->whole, n = sv->splits;
    return r < 0 || n == 1 ? 0 : r % n * kps / n;
  };
  auto end_stage = [&](int w) {
    if (kPair) return kps;
    const int r = w - sv->whole, n = sv->splits;
    return r < 0 || n == 1 ? kps : (r % n + 1) * kps / n;
  };
  auto unit_of = [&](int w) {
    if (!kPair) {
      const int r = w - sv->whole, n = sv->splits;
      if (r >= 0 && n > 1) w = sv->whole + r / n;
    }
    return unit_at<C::kTileM, C::kTileCols>(&sm->sc, experts, w);
  };

  if (warp >= kProdWarp0 && warp < kTmaWarp) {
    // ------------------------------------------------ producers
    const int group = (warp - kProdWarp0) >> 2, h = group & 1;  // h: this group's block of the stage
    const int p = ((warp - kProdWarp0) & 3) * 32 + lane;        // weight row within the tile
    const float mu = kDQ ? __ldg(s.mean) : 0.0f;
    const uint32_t lane_base = pair_lane(table);
    const uint32_t ta0 = tmem + ((uint32_t)((warp & 3) * 32) << 16) + (uint32_t)(C::kACol0 + h * (kHalfK / 2));
    const int rb = cols / kBlock;
    // Scales of this thread's row, from its block h of the unit's first stage on; the group's blocks are 2 kLanes
    // apart.  A warp's rows lie in 32 different cache lines, so each load instruction costs as many lookups: the scale
    // codes come 16 at a time where rows of codes are 16-byte aligned (`vec`), a second-level scale only when the row
    // enters another block of 256.
    int u = u0, ks = (u0 < items ? first_stage(u0) : 0) + (group >> 1);  // the stage whose scale is loaded next
    const uint8_t* q_row = nullptr;       // (double quant) codes; s_row: second-level scale of the row's first block,
    const float* s_row = nullptr;         // s_off: that block's place among the 256; (plain) the row's scales
    uint32_t s_off = 0, s_at = ~0u;       // s_at: the second-level scale held
    const bool vec = kDQ && rb % 16 == 0 && (reinterpret_cast<uintptr_t>(s.q) & 15) == 0;
    uint4 chunk = make_uint4(0, 0, 0, 0);
    uint32_t code = 0;
    float scale = 0.0f;
    int kend = u0 < items ? end_stage(u0) : 0;  // end of the stages of item u
    auto settle = [&]() {  // move (u, ks) to the unit that holds the stage
      while (u < items && ks >= kend) {
        ks -= kend;
        u += du;
        if (u < items) {
          ks += first_stage(u);
          kend = end_stage(u);
        }
      }
      if (u < items) {
        const Unit t = unit_of(u);
        int n = t.n0 + rank * kTileN + p;
        if (kPair && n >= rows) n = rows - 1;  // an odd last column tile: CTA 1 decodes anything, and stores nothing
        const int64_t b = ((int64_t)t.expert * rows + n) * rb;
        if (kDQ) {
          q_row = s.q + b;
          s_row = s.scale + b / kDqBlock;
          s_off = (uint32_t)(b % kDqBlock);
          s_at = ~0u;
          if (vec) chunk = __ldg(reinterpret_cast<const uint4*>(q_row) + 2 * ks / 16);
        } else {
          s_row = s.absmax + b;
        }
      }
    };
    auto load_scale = [&]() {  // of block 2 ks + h; the second block of an odd reduction's last stage does not exist
      const int b = 2 * ks + h;
      if (u >= items || b >= rb) return;
      if (kDQ) {
        if (vec) {
          if (b % 16 < 2 * kLanes) chunk = __ldg(reinterpret_cast<const uint4*>(q_row + (b & ~15)));
        } else {
          code = __ldg(q_row + b);
        }
        const uint32_t at = (s_off + b) / kDqBlock;
        if (at != s_at) {
          s_at = at;
          scale = __ldg(s_row + at);
        }
      } else {
        scale = __ldg(s_row + b);
      }
    };
    // the block that load_scale went to last: its code's value in [-1, 1] (double quant), and from it its scale
    auto block_unit = [&]() -> float {
      if (!kDQ) return 0.0f;
      if (vec) {
        const uint32_t b = (uint32_t)(2 * ks + h);
        const uint32_t lo = b & 4 ? chunk.y : chunk.x, hi = b & 4 ? chunk.w : chunk.z;
        code = ((b & 8 ? hi : lo) >> (8 * (b & 3))) & 0xffu;
      }
      return sm->unit_lut[code];
    };
    auto block_scale = [&](float unit) -> uint64_t { return both(kDQ ? dq_absmax(unit, scale, mu) : scale); };
    uint32_t ws = group >> 1, wph = 0, as = group >> 1, aph = 1;
    // codes of a stage: 64-byte swizzle, 16-byte piece c of row p lies at piece c ^ ((p / 2) % 4)
    const uint32_t c0 = (uint32_t)(p * (kTileK / 2) + (((2 * h) ^ ((p >> 1) & 3)) << 4));
    uint4 n0, n1;
    auto load_codes = [&]() -> bool {
      if (!wait_or_abort(&sm->wfull[ws], wph, sm, err)) return false;
      n0 = *reinterpret_cast<const uint4*>(w_gen0 + ws * kWBytes + c0);
      n1 = *reinterpret_cast<const uint4*>(w_gen0 + ws * kWBytes + (c0 ^ 16u));
      return true;
    };
    auto release_codes = [&]() {
      fence_proxy_async_smem();  // the slot is refilled by TMA after these reads
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm->wempty[ws]);
      ws += kLanes;
      if (ws >= kWStages) {
        ws -= kWStages;
        wph ^= 1;
      }
    };
    // Software pipeline.  The shared-memory pipe is the busiest, and a load queues behind the table lookups of all
    // sixteen warps; so the codes and the scale of the group's next stage are read while this one is decoded, and only
    // the two halves' lookups wait for their own round.
    settle();
    load_scale();
    bool more = u < items;
    uint64_t aa = 0;
    if (more) {
      aa = block_scale(block_unit());
      more = load_codes();
      if (more) release_codes();
    }
    while (more) {
      const bool some = 2 * ks + h < rb;
      const uint32_t words[8] = {n0.x, n0.y, n0.z, n0.w, n1.x, n1.y, n1.z, n1.w};
      ks += kLanes;
      if (ks >= kend) settle();
      more = u < items;
      load_scale();
      if (more) more = load_codes();
      const uint32_t ta = ta0 + as * (kTileK / 2);  // column j: codes 2j, 2j + 1 of the block as bf16x2
      uint32_t r[16];
#pragma unroll
      for (int c = 0; c < 4; ++c) decode_word_pairs(words[c], lane_base, aa, r + 4 * c);
      const float unit = block_unit();
      if (more) release_codes();
      if (!wait_or_abort(&sm->empty[as], aph, sm, err)) break;  // the MMAs left this slot
      if (some) tmem_st16(ta, r);
#pragma unroll
      for (int c = 0; c < 4; ++c) decode_word_pairs(words[4 + c], lane_base, aa, r + 4 * c);
      if (some) tmem_st16(ta + 16, r);
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm->full[as]);
      as += kLanes;
      if (as >= kStages) {
        as -= kStages;
        aph ^= 1;
      }
      aa = block_scale(unit);
    }
  } else if (warp == kTmaWarp) {
    // ------------------------------------------------ TMA: activation tiles
    if (lane == 0) {
      uint32_t it = 0;
      bool ok = true;
      for (int u = u0; u < items && ok; u += du) {
        const Unit t = unit_of(u);
        for (int ks = first_stage(u), e = end_stage(u); ks < e; ++ks, ++it) {
          const int as = it % kStages;
          ok = wait_or_abort(&sm->empty[as], ((it / kStages) & 1) ^ 1, sm, err);
          if (!ok) break;
          const int halves = odd && ks == kps - 1 ? 1 : 2;
          const uint32_t dst = b_smem0 + as * C::kBBytes;
          if constexpr (kPair) {
            // this CTA's half of the tile's rows; always a box of 128 (what lies behind the tile is loaded, not used:
            // a box per stage and half is quicker than several smaller ones)
            mbar_expect_tx(&sm->full[as], (uint32_t)halves * C::kHalfB);
            for (int h = 0; h < halves; ++h)
              tma_load_2d(dst + h * C::kHalfB, &xmap, ks * kTileK + h * kHalfK, t.m0 + rank * (t.width / 2),
                          &sm->full[as]);
          } else {
            mbar_expect_tx(&sm->full[as], (uint32_t)(t.width * halves) * kHalfK * 2);
            for (int h = 0; h < halves; ++h)
              load_rows(dst + h * C::kHalfB, &xmap, &xmap16, ks * kTileK + h * kHalfK, t.m0, t.width, &sm->full[as]);
          }
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
      for (int u = u0; u < items && ok; u += du) {
        const Unit t = unit_of(u);
        const int n = t.expert * rows + t.n0 + rank * kTileN;
        for (int ks = first_stage(u), e = end_stage(u); ks < e; ++ks, ++it) {
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
    for (int u = u0; u < items && ok; u += du, ++ucount) {
      const uint32_t idesc =
          instr_desc(C::kTileCols,
                     __shfl_sync(0xffffffffu, unit_of(u).width, 0));
      const uint32_t acc = ucount % C::kAccs;
      if (rank == 0) {
        ok = wait_or_abort(&sm->acc_empty[acc], ((ucount / C::kAccs) & 1) ^ 1, sm, err);
        if (!ok) break;
        tc_fence_after();
      }
      const uint32_t d_tm = tm_u + acc * C::kTileM;
      const int k0 = first_stage(u), k1 = end_stage(u);
      for (int ks = k0; ks < k1; ++ks) {
        ok = wait_or_abort(&sm->full[as], ph, sm, err);
        if (!ok) break;
        tc_fence_after();
        if (kPair && rank == 1) {  // tell CTA 0, whose thread issues for both
          tc_fence_before();
          if (elect_one()) mbar_arrive_leader(&sm->peer_full[as]);
        } else {
          if constexpr (kPair) {
            ok = wait_or_abort(&sm->peer_full[as], ph, sm, err);
            if (!ok) break;
            tc_fence_after();
          }
          const uint32_t a_tm = tm_u + C::kACol0 + as * (kTileK / 2);
          const uint64_t bdesc = bdesc0 + as * (C::kBBytes >> 4);
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < kTileK / 16; ++kk) {
              const int h = kk / (kHalfK / 16), j = kk % (kHalfK / 16);
              if (h == 1 && odd && ks == kps - 1) break;
              const uint64_t bd = bdesc + h * (C::kHalfB >> 4) + j * 2;
              if constexpr (kPair)
                tc_mma_ts_pair(d_tm, a_tm + kk * 8, bd, idesc, ks > k0 || kk > 0);
              else
                tc_mma_ts(d_tm, a_tm + kk * 8, bd, idesc, ks > k0 || kk > 0);
            }
            if constexpr (kPair)
              tc_commit_pair(&sm->empty[as]);
            else
              tc_commit(&sm->empty[as]);
          }
        }
        __syncwarp();
        if (++as == kStages) {
          as = 0;
          ph ^= 1;
        }
      }
      if (ok && rank == 0 && elect_one()) {
        if constexpr (kPair)
          tc_commit_pair(&sm->acc_full[acc]);
        else
          tc_commit(&sm->acc_full[acc]);
      }
      __syncwarp();
    }
  } else if (warp < kEpiWarps) {
    // ------------------------------------------------ epilogue
    uint32_t ucount = 0;
    for (int u = u0; u < items; u += du, ++ucount) {
      const Unit t = unit_of(u);
      const uint32_t acc = ucount % C::kAccs;
      if (!wait_or_abort(&sm->acc_full[acc], (ucount / C::kAccs) & 1, sm, err)) break;
      tc_fence_after();
      const int n0 = t.n0 + rank * kTileN;
      const uint32_t taddr = tmem + ((uint32_t)(warp * 32) << 16) + acc * C::kTileM;
      auto release = [&]() {
        if (kPair && rank == 1)
          mbar_arrive_leader(&sm->acc_empty[acc]);
        else
          mbar_arrive(&sm->acc_empty[acc]);
      };
      const int m1 = n0 < rows ? t.m1 : t.m0;  // (CTA 1 of an odd last column tile stores nothing)
      const int r = kPair ? -1 : u - sv->whole, splits = kPair ? 1 : sv->splits;
      if (kPair || r < 0 || splits == 1)
        store_unit(n0, t.m0, m1, t.width, taddr, out_stage, y, rows, release);
      else
        store_split(r, splits, split, n0, t.m0, m1, t.width, taddr, out_stage, y, rows, release);
    }
  }

  tc_fence_before();
  __syncthreads();
  if constexpr (kPair) cluster_sync();  // neither CTA reads the other's shared memory or TMEM any more
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc<kPair>(tmem, C::kTmemCols);
  }
}

template <bool kDQ, int kBook, bool kPair>
cudaError_t launch(const ExpertsCall& c, const CUtensorMap& xbig, const CUtensorMap& x16, const CUtensorMap& wmap,
                   int grid, unsigned* err, cudaStream_t stream) {
  constexpr size_t smem = smem_bytes<kPair>();
  static std::atomic<uint64_t> attr_done{0};  // shared-memory opt-in, once per device
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!(attr_done.load() & (1ull << dev))) {
    const cudaError_t e = cudaFuncSetAttribute(gemm_experts_kernel<kDQ, kBook, kPair>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    attr_done.fetch_or(1ull << dev);
  }
  const cudaError_t e =
      launch_pdl_cluster(gemm_experts_kernel<kDQ, kBook, kPair>, dim3(grid), dim3(kThreads), kPair ? 2 : 1, smem, stream,
                         c.scales, c.offsets, c.experts, (int)c.rows, (int)c.cols, (int)c.m, xbig, x16, wmap, static_cast<__nv_bfloat16*>(c.out), split_at(c), err);
  count_launches(1);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <bool kPair>
cudaError_t launch_form(const ExpertsCall& c, const CUtensorMap& xbig, const CUtensorMap& x16, const CUtensorMap& wmap,
                        int grid, unsigned* err, cudaStream_t stream) {
  const bool dq = c.scales.absmax == nullptr;
  if (dq)
    return c.scales.book ? launch<true, 1, kPair>(c, xbig, x16, wmap, grid, err, stream)
                         : launch<true, 0, kPair>(c, xbig, x16, wmap, grid, err, stream);
  return c.scales.book ? launch<false, 1, kPair>(c, xbig, x16, wmap, grid, err, stream)
                       : launch<false, 0, kPair>(c, xbig, x16, wmap, grid, err, stream);
}

}  // namespace

cudaError_t launch_gemm_experts(const ExpertsCall& c, unsigned* err, cudaStream_t stream, int num_sms) {
  const bool pair = experts_pair(c.m, c.experts, c.rows, c.cols, num_sms);
  CUtensorMap xbig, x16, wmap;
  if (!make_map(&xbig, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, c.in, c.cols, c.m, kHalfK,
                pair ? Cfg<true>::kRowsB : Cfg<false>::kRowsB, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !make_map(&x16, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, c.in, c.cols, c.m, kHalfK, 16, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !make_map(&wmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, c.packed, c.cols / 2, c.rows * c.experts, kTileK / 2, kTileN,
                CU_TENSOR_MAP_SWIZZLE_64B))
    return cudaErrorNotSupported;
  // no more units than the row tiles that m rows can make, each with all column tiles
  const int64_t tm = pair ? Cfg<true>::kTileM : Cfg<false>::kTileM, tn = pair ? 2 * kTileN : kTileN;
  const int64_t tiles = (c.m < c.experts ? c.m : c.experts) + c.m / tm;
  const int64_t units = tiles * ((c.rows + tn - 1) / tn) * (c.workspace != nullptr ? kExpertsMaxSplit : 1);
  const int64_t most = pair ? num_sms / 2 : num_sms;
  const int grid = (int)(units < most ? units : most) * (pair ? 2 : 1);
  return pair ? launch_form<true>(c, xbig, x16, wmap, grid, err, stream)
              : launch_form<false>(c, xbig, x16, wmap, grid, err, stream);
}

}  // namespace nf4
