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
//   A = Wc^T tile [128 k (UMMA M, MN-major)] x [64 n], B = dY tile [rows] x [64 n] (TMA), D in TMEM.
// Two accumulators: one tile's epilogue runs beside the next tile's MMAs.  Warp roles, CTA pairs, decode and pipeline as
// in the forward product; here the shared-memory pipe also carries the decoded tile (128 wavefronts per stage besides the
// table's 256), so half of each block goes through the byte-permute decode instead: 8 experts of 14336x4096, 16 rows 182 -> 167 us, and
// 9 % less time for 4096 rows (in the forward product the same cost 5 to 15 %).
//
// Measured: 8 experts of 14336x4096, 4096 rows 538 us in single launches (894 TFLOP/s), 533 us back to back; 16 rows
// 107 us.  The shared-memory pipe bounds the few rows (68 % of its wavefronts by the counters, TMA and MMA traffic besides),
// the ordering of CTA 1's tile before CTA 0's MMAs the pairs (see the hand-over warps).
#include <cuda.h>

#include <atomic>

#include "experts.cuh"

namespace nf4 {
namespace {

using namespace experts;

constexpr int kTileR = 64;   // weight rows (reduction) per stage
constexpr int kGroups = 4;   // producer groups of four warps, a stage each in turn
constexpr int kWBytes = kTileR * 64;  // packed codes of a stage: two blocks per row
constexpr int kSBytes = kTileR * 16;  // 16-byte scale chunk per row
constexpr int kABytes = kTileR * kTileN * 2;
constexpr int kProdWarp0 = kEpiWarps;
constexpr int kTmaWarp = kProdWarp0 + 4 * kGroups;
constexpr int kMmaWarp = kTmaWarp + 1;
constexpr int kTmaWWarp = kTmaWarp + 2;

// A-tile layout (MN-major, 128-byte swizzle): reduction row r, column e (k) at
//   (r / 8) * kKGroup + (e / 64) * kMnAtom + (r % 8) * 128 + (((e % 64) / 8) ^ (r % 8)) * 16 + (e % 8) * 2
constexpr uint32_t kMnAtom = 1024;
constexpr uint32_t kKGroup = 2048;

// kPair: two CTAs share a tile of 256 output columns x up to 256 rows of dY, each decoding its own 128 columns and loading
// half of the rows; otherwise tiles of 128 columns x up to 64 rows, for few rows per expert.
template <bool kPair>
struct Cfg {
  static constexpr int kTileM = kPair ? 256 : 64;
  static constexpr int kRowsB = kPair ? 128 : 64;  // dY rows in one CTA's shared memory
  static constexpr int kTileCols = kPair ? 2 * kTileN : kTileN;
  static constexpr int kStages = 5;                // operand ring: dY tile + decoded tile
  // CTA 1 of a pair has a hand-over warp per slot of the ring: the MMA issuer's, which has nothing to issue there, and
  // these behind the last one
  static constexpr int kHandWarps = kPair ? kStages - 1 : 0;
  static constexpr int kThreads = (kTmaWWarp + 1 + kHandWarps) * 32;
  static constexpr int kWStages = kPair ? 4 : 8;   // packed codes and scale chunks
  static constexpr int kBBytes = kRowsB * kTileR * 2;
  static constexpr int kTmemCols = 2 * kTileM;     // two accumulators
  // the operand ring empties in order, code loads may land out of order (see the forward product)
  static_assert(kStages >= kGroups && kWStages % kGroups == 0, "rings and producer groups");
};

template <bool kPair>
struct Smem {
  uint64_t wfull[Cfg<kPair>::kWStages];
  uint64_t wempty[Cfg<kPair>::kWStages];
  uint64_t full[Cfg<kPair>::kStages];
  uint64_t peer_full[Cfg<kPair>::kStages];  // (CTA 0 of a pair) the same in CTA 1, told by its hand-over warps
  uint64_t empty[Cfg<kPair>::kStages];
  uint64_t acc_full[2], acc_empty[2];
  uint32_t tmem_base;
  int abort;
  float unit_lut[256];
  Schedule sc;
};

// Shared memory: (pairs) the packed codes, the epilogue's staging and Smem before the pair table at 32 KB; after it the
// operand ring, (alone) the packed codes, and the scale chunks.  The window of a CTA without static shared memory starts
// at 1 KB (the kernel checks that all of it fits).
constexpr uint32_t kWindow = 1024;
template <bool kPair>
constexpr uint32_t front_bytes() {
  return (kPair ? Cfg<kPair>::kWStages * kWBytes : 0) + kEpiWarps * kOutBytes + (uint32_t)sizeof(Smem<kPair>);
}
template <bool kPair>
constexpr size_t smem_bytes() {
  using C = Cfg<kPair>;
  return 2 * (size_t)kPairTableDense - kWindow + C::kStages * (C::kBBytes + kABytes) +
         C::kWStages * (kSBytes + (kPair ? 0 : kWBytes));
}
static_assert(smem_bytes<true>() <= 232448 && smem_bytes<false>() <= 232448, "shared memory per CTA");
static_assert(kWindow + front_bytes<true>() <= kPairTableDense && kWindow + front_bytes<false>() <= kPairTableDense,
              "front part");

// kScaleTma: scale chunks by TMA (rows of scales are whole 16-byte units); otherwise each producer loads its own
template <bool kDQ, bool kScaleTma, int kBook, bool kPair>
__global__ void __launch_bounds__(Cfg<kPair>::kThreads, 1)
    gemm_experts_dx_kernel(Scales s, const int* __restrict__ offsets, int experts, int rows, int cols, int m_total,
                           const __grid_constant__ CUtensorMap ymap, const __grid_constant__ CUtensorMap ymap16,
                           const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap smap,
                           __nv_bfloat16* __restrict__ dx, Split split, unsigned* err) {
  using C = Cfg<kPair>;
  constexpr int kStages = C::kStages, kWStages = C::kWStages;
  extern __shared__ uint8_t smem_raw[];
  pdl_launch_dependents();
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t cta = raw & 0xff000000u;  // in a cluster, a CTA's window lies at its rank's place
  const uint32_t front = (raw + 1023u) & ~1023u, table = cta + kPairTableDense;
  uint8_t* front_gen = smem_raw + (front - raw);
  const uint32_t b_smem0 = table + kPairTableDense, a_smem0 = b_smem0 + kStages * C::kBBytes;
  const uint32_t after = a_smem0 + kStages * kABytes;
  const uint32_t w_smem0 = kPair ? front : after, s_smem0 = kPair ? after : after + kWStages * kWBytes;
  uint8_t* a_gen0 = front_gen + (a_smem0 - front);
  const uint8_t* w_gen0 = front_gen + (w_smem0 - front);
  const uint8_t* s_gen0 = front_gen + (s_smem0 - front);
  uint8_t* out_stage = front_gen + (kPair ? kWStages * kWBytes : 0);
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
      mbar_init(&sm->wempty[i], 4);
    }
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&sm->full[i], 1 + 4);
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
    prefetch_map(&ymap);
    prefetch_map(&ymap16);
    prefetch_map(&wmap);
    if (kScaleTma) prefetch_map(&smap);
  }
  fill_pair_table<kBook, 128>(front_gen + (table - front));
  pdl_wait();
  const int kps = rows / kTileR;
  build_schedule<C::kTileM>(&sm->sc, offsets, experts, m_total, (cols + C::kTileCols - 1) / C::kTileCols, kps,
                            !kPair && split.part != nullptr);
  tc_fence_before();
  __syncthreads();
  if constexpr (kPair) cluster_sync();  // the other CTA's barriers are initialised, its TMEM allocated
  tc_fence_after();
  const uint32_t tmem = sm->tmem_base;
  // Items: the whole units, then `splits` per unit of the rest, split i taking stages [i * kps / splits, ...).  Read from
  // shared memory where they are used, once per item: the producers have no registers to spare for them.
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
    const int group = (warp - kProdWarp0) >> 2;
    const int p = ((warp - kProdWarp0) & 3) * 32 + lane;
    const int r = p & (kTileR - 1), h = p >> 6;  // weight row within the stage, 64-column half of the output tile
    const float mu = kDQ ? __ldg(s.mean) : 0.0f;
    const uint32_t lane_base = pair_lane(table);
    const DecodeMul dm = decode_mul();
    const int rb = cols / kBlock;
    // this thread's 128-byte row of the A tile
    uint8_t* const a_row = a_gen0 + (r >> 3) * kKGroup + h * kMnAtom + (r & 7) * 128;
    const uint32_t swz = (uint32_t)(r & 7) << 4;
    int u = u0, ks = (u0 < items ? first_stage(u0) : 0) + group;  // the stage read next
    int64_t block0 = 0;      // level-1 block of this thread in the unit's first stage
    int kb = 0;              // its column of blocks
    int kend = u0 < items ? end_stage(u0) : 0;  // end of the stages of item u
    auto settle = [&]() {    // move (u, ks) to the unit that holds the stage
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
        kb = (t.n0 + rank * kTileN) / kBlock + h;
        if (kPair && kb >= rb) kb = rb - 1;  // an odd last column tile: CTA 1 decodes anything, and stores nothing
        block0 = ((int64_t)t.expert * rows + r) * rb + kb;
      }
    };
    uint32_t code = 0;
    float scale = 0.0f;
    auto load_scale = [&]() {  // what of the block's scale lies in global memory
      if (u >= items) return;
      const int64_t b = block0 + (int64_t)ks * kTileR * rb;
      if (kDQ) {
        if (!kScaleTma) code = __ldg(s.q + b);
        scale = __ldg(s.scale + b / kDqBlock);
      } else if (!kScaleTma) {
        scale = __ldg(s.absmax + b);
      }
    };
    uint32_t ws = group, wph = 0, as = group, aph = 1;
    // codes of a stage: 64-byte swizzle, 16-byte piece c of row r lies at piece c ^ ((r / 2) % 4)
    const uint32_t c0 = (uint32_t)(r * 64 + (((2 * h) ^ ((r >> 1) & 3)) << 4));
    uint4 n0, n1;
    auto load_codes = [&]() -> bool {
      if (!wait_or_abort(&sm->wfull[ws], wph, sm, err)) return false;
      n0 = *reinterpret_cast<const uint4*>(w_gen0 + ws * kWBytes + c0);
      n1 = *reinterpret_cast<const uint4*>(w_gen0 + ws * kWBytes + (c0 ^ 16u));
      if (kScaleTma) {
        const uint8_t* sc = s_gen0 + ws * kSBytes + r * 16;
        if (kDQ)
          code = sc[kb & 15];
        else
          scale = reinterpret_cast<const float*>(sc)[kb & 3];
      }
      return true;
    };
    auto release_codes = [&]() {
      fence_proxy_async_smem();  // the slot is refilled by TMA after these reads
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm->wempty[ws]);
      ws += kGroups;
      if (ws >= kWStages) {
        ws -= kWStages;
        wph ^= 1;
      }
    };
    auto block_scale = [&](float unit) -> uint64_t { return both(kDQ ? dq_absmax(unit, scale, mu) : scale); };
    // software pipeline as in the forward product
    settle();
    load_scale();
    bool more = u < items;
    uint64_t aa = 0;
    if (more) {
      more = load_codes();
      if (more) release_codes();
      aa = block_scale(kDQ ? sm->unit_lut[code] : 0.0f);
    }
    while (more) {
      const uint32_t words[8] = {n0.x, n0.y, n0.z, n0.w, n1.x, n1.y, n1.z, n1.w};
      ks += kGroups;
      if (ks >= kend) settle();
      more = u < items;
      load_scale();
      if (more) more = load_codes();
      uint8_t* const arow = a_row + as * kABytes;
      uint32_t q[16];
#pragma unroll
      for (int c = 0; c < 4; ++c) decode_word_pairs_dense(words[c], lane_base, aa, q + 4 * c);
      const float unit = kDQ ? sm->unit_lut[code] : 0.0f;
      if (more) release_codes();
      if (!wait_or_abort(&sm->empty[as], aph, sm, err)) break;  // the MMAs left this slot
#pragma unroll
      for (int c = 0; c < 4; ++c)
        *reinterpret_cast<uint4*>(arow + ((c << 4) ^ swz)) = make_uint4(q[4 * c], q[4 * c + 1], q[4 * c + 2], q[4 * c + 3]);
      {  // the second half by byte permutes: the ALU pipe has room, the shared-memory pipe has not
        const Table T = make_table<kBook>(__uint_as_float((uint32_t)aa));
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t d[4];
          decode_word(words[4 + c], T, d, dm);
          q[4 * c] = d[0];
          q[4 * c + 1] = d[1];
          q[4 * c + 2] = d[2];
          q[4 * c + 3] = d[3];
        }
      }
#pragma unroll
      for (int c = 0; c < 4; ++c)
        *reinterpret_cast<uint4*>(arow + (((c + 4) << 4) ^ swz)) =
            make_uint4(q[4 * c], q[4 * c + 1], q[4 * c + 2], q[4 * c + 3]);
      fence_proxy_async_smem();  // generic-proxy writes, read by the tensor cores (async proxy)
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm->full[as]);
      as += kGroups;
      if (as >= kStages) {
        as -= kStages;
        aph ^= 1;
      }
      aa = block_scale(unit);
    }
  } else if (warp == kTmaWarp) {
    // ------------------------------------------------ TMA: dY tiles
    if (lane == 0) {
      uint32_t it = 0;
      bool ok = true;
      for (int u = u0; u < items && ok; u += du) {
        const Unit t = unit_of(u);
        for (int ks = first_stage(u), e = end_stage(u); ks < e; ++ks, ++it) {
          const int as = it % kStages;
          ok = wait_or_abort(&sm->empty[as], ((it / kStages) & 1) ^ 1, sm, err);
          if (!ok) break;
          const uint32_t dst = b_smem0 + as * C::kBBytes;
          if constexpr (kPair) {  // always a box of 128 rows, as in the forward product
            mbar_expect_tx(&sm->full[as], C::kBBytes);
            tma_load_2d(dst, &ymap, ks * kTileR, t.m0 + rank * (t.width / 2), &sm->full[as]);
          } else {
            mbar_expect_tx(&sm->full[as], (uint32_t)t.width * kTileR * 2);
            load_rows(dst, &ymap, &ymap16, ks * kTileR, t.m0, t.width, &sm->full[as]);
          }
        }
      }
      for (uint32_t j = (it > kStages ? it - kStages : 0); j < it; ++j)  // drain the copies still in flight
        if (!mbar_wait_bounded(&sm->full[j % kStages], (j / kStages) & 1, err)) break;
    }
  } else if (warp == kTmaWWarp) {
    // ------------------------------------------------ TMA: packed codes and scale chunks
    if (lane == 0) {
      uint32_t it = 0;
      bool ok = true;
      for (int u = u0; u < items && ok; u += du) {
        const Unit t = unit_of(u);
        const int n = t.expert * rows, k0 = t.n0 + rank * kTileN;
        for (int ks = first_stage(u), e = end_stage(u); ks < e; ++ks, ++it) {
          const int ws = it % kWStages;
          ok = wait_or_abort(&sm->wempty[ws], ((it / kWStages) & 1) ^ 1, sm, err);
          if (!ok) break;
          mbar_expect_tx(&sm->wfull[ws], kWBytes + (kScaleTma ? kSBytes : 0));
          tma_load_2d(w_smem0 + ws * kWBytes, &wmap, k0 / 2, n + ks * kTileR, &sm->wfull[ws]);
          // the 16-byte chunk holding block columns k0 / 64 and k0 / 64 + 1 (the first is even)
          if (kScaleTma)
            tma_load_2d(s_smem0 + ws * kSBytes, &smap, (k0 / kBlock) & (kDQ ? ~15 : ~3), n + ks * kTileR,
                        &sm->wfull[ws]);
        }
      }
      for (uint32_t j = (it > kWStages ? it - kWStages : 0); j < it; ++j)
        if (!mbar_wait_bounded(&sm->wfull[j % kWStages], (j / kWStages) & 1, err)) break;
    }
  } else if (kPair && rank == 1 && warp >= kMmaWarp) {
    // ------------------------------------------------ CTA 1: tell CTA 0, whose thread issues for both
    // The decoded tile consists of ordinary stores by this CTA's producers, and an MMA that CTA 0 issues reads it: what
    // they handed over at `full` goes on to CTA 0 with a release at cluster scope, and is acquired there.  Such a release
    // takes some 1100 to 1900 cycles, longer than a stage; so each slot of the ring has a warp that waits for it.  8 experts
    // of 14336x4096, 4096 rows, single launches: 538 us; with one warp for all slots 1180, two 730, three 580, with the
    // release in the producers 610.  (Without the scope, which leaves the order to chance, it was 455.)
    const uint32_t as = warp == kMmaWarp ? 0 : warp - kTmaWWarp;
    const uint32_t stages = u0 < items ? (uint32_t)((items - u0 + du - 1) / du) * (uint32_t)kps : 0;
    uint32_t ph = 0;
    for (uint32_t it = as; it < stages; it += kStages, ph ^= 1) {
      if (!wait_or_abort(&sm->full[as], ph, sm, err)) break;
      if (elect_one()) mbar_arrive_leader_release(&sm->peer_full[as]);
      __syncwarp();
    }
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------ MMA issuer (of a pair in CTA 0)
    const uint32_t tm_u = __shfl_sync(0xffffffffu, tmem, 0);
    const uint64_t adesc0 = smem_desc_mn_sw128(a_smem0, kMnAtom, kKGroup), bdesc0 = smem_desc_sw128(b_smem0);
    uint32_t as = 0, ph = 0, ucount = 0;
    bool ok = true;
    for (int u = u0; u < items && ok; u += du, ++ucount) {
      const uint32_t idesc = instr_desc(
          C::kTileCols, __shfl_sync(0xffffffffu, unit_of(u).width, 0),
          /*a_mn=*/true);
      const uint32_t acc = ucount & 1;
      ok = wait_or_abort(&sm->acc_empty[acc], ((ucount >> 1) & 1) ^ 1, sm, err);
      if (!ok) break;
      tc_fence_after();
      const uint32_t d_tm = tm_u + acc * C::kTileM;
      const int k0 = first_stage(u), k1 = end_stage(u);
      for (int ks = k0; ks < k1; ++ks) {
        ok = wait_or_abort(&sm->full[as], ph, sm, err);
        if (!ok) break;
        tc_fence_after();
        if constexpr (kPair) {
          ok = wait_or_abort_leader(&sm->peer_full[as], ph, sm, err);
          if (!ok) break;
          tc_fence_after();
        }
        const uint64_t adesc = adesc0 + as * (kABytes >> 4), bdesc = bdesc0 + as * (C::kBBytes >> 4);
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < kTileR / 16; ++kk) {  // 16 weight rows per MMA: two 8-row groups, 32 bytes of dY
            const uint64_t ad = adesc + kk * (2 * kKGroup >> 4), bd = bdesc + kk * 2;
            if constexpr (kPair)
              tc_mma_ss_pair(d_tm, ad, bd, idesc, ks > k0 || kk > 0);
            else
              tc_mma_ss(d_tm, ad, bd, idesc, ks > k0 || kk > 0);
          }
          if constexpr (kPair)
            tc_commit_pair(&sm->empty[as]);
          else
            tc_commit(&sm->empty[as]);
        }
        __syncwarp();
        if (++as == kStages) {
          as = 0;
          ph ^= 1;
        }
      }
      if (ok && elect_one()) {
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
      const uint32_t acc = ucount & 1;
      if (!wait_or_abort(&sm->acc_full[acc], (ucount >> 1) & 1, sm, err)) break;
      tc_fence_after();
      const int n0 = t.n0 + rank * kTileN;  // first output column
      const uint32_t taddr = tmem + ((uint32_t)(warp * 32) << 16) + acc * C::kTileM;
      auto release = [&]() {
        if (kPair && rank == 1)
          mbar_arrive_leader(&sm->acc_empty[acc]);
        else
          mbar_arrive(&sm->acc_empty[acc]);
      };
      const int m1 = n0 < cols ? t.m1 : t.m0;  // (CTA 1 of an odd last column tile stores nothing)
      const int r = kPair ? -1 : u - sv->whole, splits = kPair ? 1 : sv->splits;
      if (kPair || r < 0 || splits == 1)
        store_unit(n0, t.m0, m1, t.width, taddr, out_stage, dx, cols, release);
      else
        store_split(r, splits, split, n0, t.m0, m1, t.width, taddr, out_stage, dx, cols, release);
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

struct Maps {
  CUtensorMap y, y16, w, s;
};

template <bool kDQ, bool kScaleTma, int kBook, bool kPair>
cudaError_t launch(const ExpertsCall& c, const Maps& m, int grid, unsigned* err, cudaStream_t stream) {
  constexpr size_t smem = smem_bytes<kPair>();
  static std::atomic<uint64_t> attr_done{0};  // shared-memory opt-in, once per device
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!(attr_done.load() & (1ull << dev))) {
    const cudaError_t e = cudaFuncSetAttribute(gemm_experts_dx_kernel<kDQ, kScaleTma, kBook, kPair>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    attr_done.fetch_or(1ull << dev);
  }
  const cudaError_t e = launch_pdl_cluster(gemm_experts_dx_kernel<kDQ, kScaleTma, kBook, kPair>, dim3(grid),
                                           dim3(Cfg<kPair>::kThreads), kPair ? 2 : 1, smem, stream, c.scales, c.offsets, c.experts,
                                           (int)c.rows, (int)c.cols, (int)c.m, m.y, m.y16, m.w, m.s,
                                           static_cast<__nv_bfloat16*>(c.out), split_at(c), err);
  count_launches(1);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <bool kDQ, bool kScaleTma, int kBook>
cudaError_t launch_width(const ExpertsCall& c, const Maps& m, bool pair, int grid, unsigned* err, cudaStream_t stream) {
  return pair ? launch<kDQ, kScaleTma, kBook, true>(c, m, grid, err, stream)
              : launch<kDQ, kScaleTma, kBook, false>(c, m, grid, err, stream);
}

template <bool kDQ, bool kScaleTma>
cudaError_t launch_book(const ExpertsCall& c, const Maps& m, bool pair, int grid, unsigned* err, cudaStream_t stream) {
  return c.scales.book ? launch_width<kDQ, kScaleTma, 1>(c, m, pair, grid, err, stream)
                       : launch_width<kDQ, kScaleTma, 0>(c, m, pair, grid, err, stream);
}

}  // namespace

cudaError_t launch_gemm_experts_dx(const ExpertsCall& c, unsigned* err, cudaStream_t stream, int num_sms) {
  const bool pair = experts_pair(c.m, c.experts, c.cols, c.rows, num_sms);
  const bool dq = c.scales.absmax == nullptr;
  const int64_t rb = c.cols / kBlock, stack = c.rows * c.experts;
  Maps m;
  if (!make_map(&m.y, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, c.in, c.rows, c.m, kTileR,
                pair ? Cfg<true>::kRowsB : Cfg<false>::kRowsB, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !make_map(&m.y16, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, c.in, c.rows, c.m, kTileR, 16, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !make_map(&m.w, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, c.packed, c.cols / 2, stack, 64, kTileR,
                CU_TENSOR_MAP_SWIZZLE_64B))
    return cudaErrorNotSupported;
  const void* sbase = dq ? (const void*)c.scales.q : (const void*)c.scales.absmax;
  bool scale_tma = (dq ? rb : 4 * rb) % 16 == 0 && reinterpret_cast<uintptr_t>(sbase) % 16 == 0;
  if (scale_tma)
    scale_tma = dq ? make_map(&m.s, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, sbase, rb, stack, 16, kTileR,
                              CU_TENSOR_MAP_SWIZZLE_NONE)
                   : make_map(&m.s, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, sbase, rb, stack, 4, kTileR,
                              CU_TENSOR_MAP_SWIZZLE_NONE);
  if (!scale_tma) m.s = m.w;  // unused by the kernel variant
  // no more units than the row tiles that m rows can make, each with all column tiles
  const int64_t tm = pair ? Cfg<true>::kTileM : Cfg<false>::kTileM, tn = pair ? 2 * kTileN : kTileN;
  const int64_t tiles = (c.m < c.experts ? c.m : c.experts) + c.m / tm;
  const int64_t units = tiles * ((c.cols + tn - 1) / tn) * (c.workspace != nullptr ? kExpertsMaxSplit : 1);
  const int64_t most = pair ? num_sms / 2 : num_sms;
  const int grid = (int)(units < most ? units : most) * (pair ? 2 : 1);
  if (dq)
    return scale_tma ? launch_book<true, true>(c, m, pair, grid, err, stream)
                     : launch_book<true, false>(c, m, pair, grid, err, stream);
  return scale_tma ? launch_book<false, true>(c, m, pair, grid, err, stream)
                   : launch_book<false, false>(c, m, pair, grid, err, stream);
}

}  // namespace nf4
