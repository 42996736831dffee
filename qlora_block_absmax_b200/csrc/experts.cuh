// experts.cuh -- what the expert products (gemm_experts_sm100.cu, gemm_experts_dx_sm100.cu) share: the schedule of
// ragged tiles, the activation-tile loads and the epilogue.
//
// Rows [offsets[e], offsets[e + 1]) of the activations belong to expert e, whose weight is rows [e * N, (e + 1) * N)
// of one stacked 4-bit weight.  The offsets are read on the GPU, so a launch does not know its tiles: every CTA reads
// them, counts each expert's tiles and walks the units u = blockIdx.x, + gridDim.x, ... of the same list.  An expert of
// m rows has ceil(m / TM) row tiles of equal width (a multiple of 16, the UMMA N); rows of a tile past the expert's
// last one belong to another expert, are multiplied along and never stored.
#pragma once
#include "nf4_common.cuh"
#include "nf4_decode.cuh"
#include "internal.h"
#include "umma.cuh"

namespace nf4 {
namespace experts {

using namespace umma;

// In shared memory, filled once per launch.
struct Schedule {
  int first[kMaxExperts + 1];  // first unit of expert e; first[experts] = all units
  int row[kMaxExperts + 1];    // first row of expert e (offsets, held within the activations)
  int end[kMaxExperts];        // one past its last row
  int whole;                   // units that are one item each; the others are `splits` items each
  int splits;
  int items;
};

// Split reductions (tiles of 64 rows).  The units are dealt out in rounds over the CTAs, and the last round is seldom full:
// one token through two experts makes 64 units of a 4096-row weight for 148 SMs, 192 units make 1.3 rounds.  So the
// reduction of each unit of the last round is cut into `splits` items of at least kMinSplitStages stages.  An item's fp32
// accumulator goes to the workspace; each epilogue warp (32 columns) that finds itself the last of its unit adds all of
// them in order and stores the rows.  Nobody waits for another CTA, so launches that share the GPU cannot block one
// another.  (One row through each of two experts of 4096x14336: 58.9 -> 36 us; gradient of 16 rows, 8 experts of
// 14336x4096: 161 -> 107 us.  Pairs are not split: in the forward product a 256-row tile's exchange cost what the fuller
// round saved; the gradient's pairs, whose units are longer, were not tried.)
constexpr int kMinSplitStages = 4;

struct Split {
  uint4* part;      // [items][pitch]: [chunk of 32 rows][column half][4][128 threads]
  unsigned* count;  // arrivals per unit and epilogue warp
  int pitch;        // 16-byte pieces per item
};

inline Split split_at(const ExpertsCall& c) {
  auto* w = static_cast<uint8_t*>(c.workspace);
  if (w == nullptr) return Split{nullptr, nullptr, 0};
  return Split{reinterpret_cast<uint4*>(w + kExpertsCountBytes), reinterpret_cast<unsigned*>(w),
               (int)(experts_partial_bytes(c.m) / 16)};
}

// The number of splits of `rest` units whose rounds over the grid take the fewest stages; an item's exchange counts as
// three of them.  Lane s of a warp looks at s + 1 splits.
__device__ __forceinline__ int split_of(int rest, int grid, int kps) {
  const unsigned s = (threadIdx.x & (kExpertsMaxSplit - 1)) + 1, items = (unsigned)rest * s;
  unsigned cost = 0xffffffffu;
  if (s == 1 || (items <= (unsigned)(kExpertsItems * grid) && kps >= (int)s * kMinSplitStages))
    cost = ((items + grid - 1) / grid * ((kps + s - 1) / s + (s > 1 ? 3 : 0)) << 4) + (s - 1);
  return (int)(__reduce_min_sync(0xffffffffu, cost) & 15u) + 1;
}

struct Unit {
  int expert, n0;     // expert; first output column (of N, or of K for the gradient)
  int m0, m1, width;  // activation rows [m0, m1) of a tile `width` wide
};

// All threads of the CTA; `ntn`: column tiles per expert, `kps`: stages per unit, `split`: split reductions are open.  The
// caller synchronises the CTA afterwards.  Offsets outside 0..m or decreasing (a caller's error) are held to the range,
// so no tile reaches outside the activations.
template <int TM>
__device__ __forceinline__ void build_schedule(Schedule* sc, const int* __restrict__ offsets, int experts, int m,
                                               int ntn, int kps, bool split) {
  const int tid = threadIdx.x, lane = tid & 31;
  for (int e = tid; e < experts; e += blockDim.x) {
    int a = __ldg(offsets + e), b = __ldg(offsets + e + 1);
    a = a < 0 ? 0 : a > m ? m : a;
    b = b < a ? a : b > m ? m : b;
    sc->row[e] = a;
    sc->end[e] = b;
  }
  __syncthreads();
  if (tid < 32) {  // prefix sum of the experts' units, 32 experts at a time
    int base = 0;
    for (int e0 = 0; e0 < experts; e0 += 32) {
      const int e = e0 + lane;
      int own = e < experts ? (sc->end[e] - sc->row[e] + TM - 1) / TM * ntn : 0;
      int sum = own;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, sum, d);
        if (lane >= d) sum += v;
      }
      if (e < experts) sc->first[e] = base + sum - own;
      base += __shfl_sync(0xffffffffu, sum, 31);
    }
    const int rest = split ? base % (int)gridDim.x : 0;
    const int splits = split_of(rest, gridDim.x, kps);
    if (lane == 0) {
      sc->first[experts] = base;
      sc->whole = base - rest;
      sc->splits = splits;
      sc->items = base - rest + rest * splits;
    }
  }
}

__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}

// Decode through a shared table of fp32 code pairs: entry v (a byte of two codes) at 256 v, sixteen copies of 8 bytes,
// lane l reading copy l % 16, so each half-warp phase of a 64-bit load meets every bank once.  The table is 64 KB-aligned:
// one byte permute of the packed word with the lane's offset and the table's upper address bytes is the address.  A pair
// costs that permute, one load, one packed multiply and one convert -- 16 instructions per word of 8 codes, 8 of them on
// the ALU pipe, where the byte-permute decode (nf4_decode.cuh) takes 21 and 19 and a table of 16 products per block; the
// price is 8 shared-memory wavefronts per word and warp.  The values are the same: bf16_rn(RN(code * a)).
constexpr uint32_t kPairTable = 65536;  // bytes and alignment (the second half of every 256 bytes stays unused)

__constant__ float c_code_experts[2][16] = {NF4_CODE_INIT, FP4_CODE_INIT};  // by code book

// The gradient keeps its decoded tiles in shared memory and has no 64 KB to spare: there the rows are 128 bytes, the
// table 32 KB, and the address takes a shift and a LOP3 instead of the permute.
constexpr uint32_t kPairTableDense = 32768;

template <int kBook, int kRow = 256>
__device__ __forceinline__ void fill_pair_table(uint8_t* table) {
  for (int i = threadIdx.x; i < 256 * 8; i += blockDim.x) {  // two copies of an entry
    const int v = i >> 3;
    const float hi = c_code_experts[kBook][v >> 4], lo = c_code_experts[kBook][v & 15];
    *reinterpret_cast<float4*>(table + v * kRow + (i & 7) * 16) = make_float4(hi, lo, hi, lo);
  }
}

// byte 0: 8 * (lane % 16), byte 1: 0, bytes 2-3: the upper half of the table's shared address
__device__ __forceinline__ uint32_t pair_lane(uint32_t table) { return table | (uint32_t)((threadIdx.x & 15) * 8); }

__device__ __forceinline__ uint32_t scaled_pair(uint32_t addr, uint64_t aa) {
  uint32_t d;
  asm("{\n .reg .b64 c;\n .reg .f32 x, y;\n ld.shared.b64 c, [%1];\n mul.rn.f32x2 c, c, %2;\n"
      " mov.b64 {x, y}, c;\n cvt.rn.bf16x2.f32 %0, y, x;\n}"
      : "=r"(d)
      : "r"(addr), "l"(aa));
  return d;
}

// 8 codes of a packed word -> out[b] = (code 2b, code 2b + 1) * a
__device__ __forceinline__ void decode_word_pairs(uint32_t w, uint32_t lane_base, uint64_t aa, uint32_t* out) {
  out[0] = scaled_pair(prmt(w, lane_base, 0x7604u), aa);
  out[1] = scaled_pair(prmt(w, lane_base, 0x7614u), aa);
  out[2] = scaled_pair(prmt(w, lane_base, 0x7624u), aa);
  out[3] = scaled_pair(prmt(w, lane_base, 0x7634u), aa);
}

__device__ __forceinline__ void decode_word_pairs_dense(uint32_t w, uint32_t lane_base, uint64_t aa, uint32_t* out) {
  out[0] = scaled_pair(((w << 7) & 0x7f80u) | lane_base, aa);
  out[1] = scaled_pair(((w >> 1) & 0x7f80u) | lane_base, aa);
  out[2] = scaled_pair(((w >> 9) & 0x7f80u) | lane_base, aa);
  out[3] = scaled_pair(((w >> 17) & 0x7f80u) | lane_base, aa);
}

__device__ __forceinline__ uint64_t both(float a) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %1};" : "=l"(d) : "f"(a));
  return d;
}

// 32 lanes x 16 consecutive 32-bit columns from registers; st_wait before they are read
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// One lane of a converged warp.  The MMA warp runs its loop with all lanes and lets one of them issue: the loop's
// addresses and descriptors then stay in uniform registers, where a loop inside `if (lane == 0)` moves each of them
// over for every instruction.
__device__ __forceinline__ bool elect_one() {
  uint32_t e;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(e));
  return e != 0;
}

// Unit u of the list: experts in order, their column tiles (kCols wide) next, row tiles innermost (the row tiles of a
// column tile run at the same time and share its codes in L2).
template <int TM, int kCols = kTileN>
__device__ __forceinline__ Unit unit_at(const Schedule* sc, int experts, int u) {
  int lo = 0, hi = experts;  // first[lo] <= u < first[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (sc->first[mid] <= u)
      lo = mid;
    else
      hi = mid;
  }
  Unit t;
  t.expert = lo;
  const int r0 = sc->row[lo], rows = sc->end[lo] - r0;
  const int ntm = (rows + TM - 1) / TM;
  const int v = u - sc->first[lo];
  const int tm = v % ntm;
  t.n0 = v / ntm * kCols;
  constexpr int kAlign = kCols / kTileN * 16;  // each CTA of a pair loads half the tile, in boxes of 16 rows
  t.width = ((rows + ntm - 1) / ntm + kAlign - 1) & ~(kAlign - 1);
  t.m0 = r0 + tm * t.width;
  const int m1 = t.m0 + t.width;
  t.m1 = m1 < sc->end[lo] ? m1 : sc->end[lo];
  return t;
}

// ------------------------------------------------------------------ CTA pairs (cta_group::2)

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %cluster_ctarank;" : "=r"(r));
  return r;
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Arrive at CTA 0's barrier of the same name, to say that TMEM was written or read (ordered by the tcgen05 fences around the
// arrival) or that a TMA load has landed (its completion seen on a local barrier).  It orders no ordinary store: with a
// release at cluster scope it would, at 1100 cycles per stage of the forward product's issue loop (499 -> 544 us at 8 experts
// of 14336x4096, 4096 rows).
__device__ __forceinline__ void mbar_arrive_leader(uint64_t* bar) {
  asm volatile(
      "{\n .reg .b32 a;\n mapa.shared::cluster.u32 a, %0, 0;\n mbarrier.arrive.shared::cluster.b64 _, [a];\n}" ::"r"(
          smem_u32(bar))
      : "memory");
}

// The same with a release at cluster scope, which wait_or_abort_leader acquires: what this thread has written, or seen
// written, to its own shared memory is written for CTA 0's thread too.
__device__ __forceinline__ void mbar_arrive_leader_release(uint64_t* bar) {
  asm volatile(
      "{\n .reg .b32 a;\n mapa.shared::cluster.u32 a, %0, 0;\n"
      " mbarrier.arrive.release.cluster.shared::cluster.b64 _, [a];\n}" ::"r"(smem_u32(bar))
      : "memory");
}

__device__ __forceinline__ bool mbar_try_wait_cluster(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n"
      " selp.u32 %0, 1, 0, p;\n}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// wait_or_abort with the acquire that mbar_arrive_leader_release asks for
template <class Sm>
__device__ __forceinline__ bool wait_or_abort_leader(uint64_t* bar, uint32_t parity, Sm* sm, unsigned* err) {
  if (mbar_try_wait_cluster(bar, parity)) return true;
  if (aborted(sm)) return false;
  const unsigned long long t0 = global_ns();
  do {
    for (int i = 0; i < 64; ++i)
      if (mbar_try_wait_cluster(bar, parity)) return true;
  } while (global_ns() - t0 <= kWaitLimitNs);
  atomicOr(err, kErrTimeout);
  *(volatile int*)&sm->abort = 1;
  return false;
}

// D (TMEM of both CTAs, 128 rows each) (+)= A (TMEM of both) . B (half of its rows in each CTA's shared memory)
__device__ __forceinline__ void tc_mma_ts_pair(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                               uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(acc)
      : "memory");
}

// the same with A (128 rows in each CTA) in shared memory
__device__ __forceinline__ void tc_mma_ss_pair(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                               uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(acc)
      : "memory");
}

// arrive at the barrier of both CTAs once the MMAs issued so far have finished
__device__ __forceinline__ void tc_commit_pair(uint64_t* bar) {
  asm volatile(
      "{\n .reg .b16 m;\n mov.b16 m, 3;\n"
      " tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], m;\n}" ::"r"(
          smem_u32(bar))
      : "memory");
}

template <bool kPair>
__device__ __forceinline__ void tmem_alloc(uint32_t* dst, uint32_t cols) {
  if constexpr (kPair) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;\n"
                 "tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::"r"(smem_u32(dst)),
                 "r"(cols)
                 : "memory");
  } else {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n"
                 "tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::"r"(smem_u32(dst)),
                 "r"(cols)
                 : "memory");
  }
}

template <bool kPair>
__device__ __forceinline__ void tmem_dealloc(uint32_t base, uint32_t cols) {
  if constexpr (kPair)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(base), "r"(cols) : "memory");
  else
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(base), "r"(cols) : "memory");
}

// `width` activation rows from row m0, 64 columns from x, as boxes of 64 and 16 rows (both whole swizzle atoms)
__device__ __forceinline__ void load_rows(uint32_t dst, const CUtensorMap* map64, const CUtensorMap* map16, int x,
                                          int m0, int width, uint64_t* bar) {
  int r = 0;
  for (; r + 64 <= width; r += 64) tma_load_2d(dst + r * 128, map64, x, m0 + r, bar);
  for (; r < width; r += 16) tma_load_2d(dst + r * 128, map16, x, m0 + r, bar);
}

// 16 lanes x 32 consecutive fp32 columns in the layout of an mma accumulator: registers 4i, 4i + 1 are lane L / 4,
// columns 8i + 2 (L % 4) + {0, 1} of thread L, registers 4i + 2, 4i + 3 lane L / 4 + 8
__device__ __forceinline__ void tmem_ld_16x256(uint32_t taddr, uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
        "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
      : "r"(taddr)
      : "memory");
}
// The registers pass through the wait, so that no use of them is scheduled before it.
__device__ __forceinline__ void tmem_ld_wait(uint32_t (&v)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]),
                 "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15])::"memory");
}

// four 8x8 matrices of 16-bit elements, stored transposed: lane L gives the address of row L % 8 of matrix L / 8
__device__ __forceinline__ void stmatrix_x4_trans(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(a), "r"(b),
               "r"(c), "r"(d)
               : "memory");
}

constexpr int kOutPitch = 80;                 // bytes per row of 32 bf16: 16 to spare, against bank conflicts
constexpr int kOutBytes = 32 * kOutPitch;     // an epilogue warp's staging

// The epilogue of warps 0..3: accumulator (TMEM lanes = output columns, columns = activation rows) -> bf16 rows.  The
// shared-memory pipe is the producers' busiest and this waits in the same queue, so the turn from columns to rows takes
// few instructions: per 32x32 block four transposing matrix stores, four 16-byte loads and four 16-byte stores to y (with
// a 2-byte shared store per value a 256-row tile took 4000 cycles, with 2-byte stores to y 5300, like this 3600).
struct RowWriter {
  uint8_t* stage;
  uint32_t st;
  int r0, q0;
  __device__ __forceinline__ explicit RowWriter(uint8_t* stage_all) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    stage = stage_all + warp * kOutBytes;
    // matrix q = lane / 8 of a store: rows (activation rows) 8 (q / 2) .., columns 8 (q % 2) ..
    st = smem_u32(stage) + (uint32_t)((8 * (lane >> 4) + (lane & 7)) * kOutPitch + ((lane >> 3) & 1) * 16);
    r0 = lane >> 2;  // this lane's pieces of the block: rows r0, r0 + 8, .., 16 bytes q0
    q0 = lane & 3;
  }
  // 32 rows x output columns 16 half .. of the warp (as tmem_ld_16x256 gives them) into the staging
  __device__ __forceinline__ void put(const uint32_t (&a)[16], int half) const {
#pragma unroll
    for (int h = 0; h < 2; ++h) {  // 16 activation rows
      uint32_t p[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        p[i] = pack_bf16x2(__uint_as_float(a[8 * h + 2 * i]), __uint_as_float(a[8 * h + 2 * i + 1]));
      stmatrix_x4_trans(st + h * 16 * kOutPitch + half * 32, p[0], p[1], p[2], p[3]);
    }
  }
  // the block to its place `p` in y, the first `left` rows of it
  __device__ __forceinline__ void flush(__nv_bfloat16* p, int ldy, int left) const {
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint4 o = *reinterpret_cast<const uint4*>(stage + (r0 + 8 * i) * kOutPitch + q0 * 16);
      if (r0 + 8 * i < left) *reinterpret_cast<uint4*>(p + (int64_t)(r0 + 8 * i) * ldy + q0 * 8) = o;
    }
    __syncwarp();
  }
};

// Tile of output columns n0 .., rows m0 .. m1 - 1, `width` wide.  `release` is called by each warp once it has read its
// part of the accumulator: the tile's successor waits for that.
template <class Release>
__device__ __forceinline__ void store_unit(int n0, int m0, int m1, int width, uint32_t taddr, uint8_t* stage_all,
                                           __nv_bfloat16* __restrict__ y, int ldy, Release release) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const RowWriter out(stage_all);
  __nv_bfloat16* p = y + (int64_t)m0 * ldy + n0 + warp * 32;
  const int chunks = (width + 31) / 32;
#pragma unroll 1
  for (int c = 0; c < chunks; ++c) {
    uint32_t a[16], b[16];
    tmem_ld_16x256(taddr + c * 32, a);
    tmem_ld_16x256(taddr + (16u << 16) + c * 32, b);
    tmem_ld_wait(a);
    tmem_ld_wait(b);
    if (c == chunks - 1) {  // read in full: the accumulator may be overwritten
      tc_fence_before();
      __syncwarp();
      if (lane == 0) release();
    }
    out.put(a, 0);
    out.put(b, 1);
    out.flush(p, ldy, m1 - m0 - c * 32);
    p += (int64_t)32 * ldy;
  }
}

// The same for item r (of `splits` per unit) of the split units.
template <class Release>
__device__ __forceinline__ void store_split(int r, int splits, const Split& sp, int n0, int m0, int m1, int width,
                                            uint32_t taddr, uint8_t* stage_all, __nv_bfloat16* __restrict__ y, int ldy,
                                            Release release) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, tid = threadIdx.x;
  const int chunks = (width + 31) / 32, unit = r / splits;
  auto slot = [&](int item, int c, int h, int i) {
    return sp.part + (size_t)item * sp.pitch + ((c * 2 + h) * 4 + i) * 128 + tid;
  };
#pragma unroll 1
  for (int c = 0; c < chunks; ++c) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t a[16];
      tmem_ld_16x256(taddr + ((uint32_t)(16 * h) << 16) + c * 32, a);
      tmem_ld_wait(a);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        __stcg(slot(r, c, h, i), make_uint4(a[4 * i], a[4 * i + 1], a[4 * i + 2], a[4 * i + 3]));
    }
  }
  tc_fence_before();
  __syncwarp();
  if (lane == 0) release();
  __threadfence();
  __syncwarp();
  unsigned before = 0;
  unsigned* const count = sp.count + unit * kEpiWarps + warp;
  if (lane == 0) before = atomicAdd(count, 1u);
  if (__shfl_sync(0xffffffffu, before, 0) != (unsigned)splits - 1) return;
  if (lane == 0) *count = 0;  // ready for the next call
  __threadfence();
  const RowWriter out(stage_all);
#pragma unroll 1
  for (int c = 0; c < chunks; ++c) {
#pragma unroll 1
    for (int h = 0; h < 2; ++h) {
      float sum[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) sum[i] = 0.0f;
#pragma unroll 1
      for (int k = 0; k < splits; ++k) {  // in order: the result does not depend on who came last
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint4 o = __ldcg(slot(unit * splits + k, c, h, i));
          sum[4 * i] += __uint_as_float(o.x);
          sum[4 * i + 1] += __uint_as_float(o.y);
          sum[4 * i + 2] += __uint_as_float(o.z);
          sum[4 * i + 3] += __uint_as_float(o.w);
        }
      }
      uint32_t v[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = __float_as_uint(sum[i]);
      out.put(v, h);
    }
    out.flush(y + (int64_t)(m0 + c * 32) * ldy + n0 + warp * 32, ldy, m1 - m0 - c * 32);
  }
}

}  // namespace experts
}  // namespace nf4
