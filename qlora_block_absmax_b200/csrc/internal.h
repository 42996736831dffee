// internal.h -- launchers behind the C ABI (see include/nf4.h for semantics).
// Arguments are validated by the callers in api.cu; launchers only size grids.
#pragma once
#include <cuda_runtime.h>
#include <cstdint>

namespace nf4 {

// Launch with programmatic stream serialization: the kernel may start while the
// previous kernel in the stream finishes; it waits for it (griddepcontrol.wait)
// before touching global memory.
template <typename... KArgs, typename... Args>
cudaError_t launch_pdl(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream,
                       Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...);
}

// The same for clusters of `cluster` CTAs.
template <typename... KArgs, typename... Args>
cudaError_t launch_pdl_cluster(void (*kernel)(KArgs...), dim3 grid, dim3 block, unsigned cluster, size_t smem,
                               cudaStream_t stream, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...);
}

constexpr int kBlock = 64;      // level-1 block (elements per absmax)
constexpr int kDqBlock = 256;   // level-2 block (absmax values per second-level scale)

// Level-1 scales as the kernels see them: plain fp32 absmax, or the
// double-quantized record (8-bit codes + second-level block absmax + mean).
// count of kernels launched (read by nf4_kernel_launches)
void count_launches(int n);

struct Scales {
  const float* absmax;   // non-null: plain scales
  const uint8_t* q;      // double-quantized codes
  const float* scale;    // second-level block absmax
  const float* mean;     // device pointer to the removed mean
  int dq_code;           // 0 = E4M3, 1 = int8
  int book;              // 4-bit code book: 0 = NF4, 1 = FP4 (E2M1 / 6)
};

// blocksize 32, 64, 128 or 256
cudaError_t launch_quantize(const void* src, bool bf16, int64_t n, int blocksize, uint8_t* packed, float* absmax,
                            int book, cudaStream_t stream, int num_sms);

// several tensors of one dtype, block size and code book in one launch (w0 and iters are filled by the launcher)
constexpr int kQuantManyMax = 256;
struct QuantItem {
  const void* src;  // n elements, 16-byte aligned
  uint8_t* packed;  // ceil(n / 2)
  float* absmax;    // ceil(n / blocksize)
  int64_t n;        // >= 1
  int64_t w0;       // first warp iteration of this tensor in the launch's sequence
};
struct QuantManyParams {
  QuantItem item[kQuantManyMax];
  int32_t count;  // >= 1
  int64_t iters;  // warp iterations of all tensors
};
cudaError_t launch_quantize_many(QuantManyParams& p, bool bf16, int blocksize, int book, cudaStream_t stream,
                                 int num_sms);

// workspace: zero before its first use, left ready by every completed call; `clear` zeroes it first
cudaError_t launch_double_quant(const float* absmax, int64_t nb, int dq_code, uint8_t* q, float* scale,
                                float* mean, void* workspace, bool clear, unsigned* err, cudaStream_t stream,
                                int num_sms);
constexpr size_t kDoubleQuantWorkspace = 256;

// double quantization of several absmax arrays in two launches (one exact-sum record per tensor in the workspace)
constexpr int kDqManyMax = 256;
constexpr size_t kDqManyRecord = 128;  // workspace bytes per tensor
struct DqItem {
  const float* a;  // absmax [nb], 16-byte aligned
  uint8_t* q;      // codes [nb]
  float* scale;    // [ceil(nb / 256)]
  float* mean;     // [1]
  int64_t nb;      // >= 1
  int64_t e0;      // first element of this array in the concatenation of all of them
  int64_t g0;      // first 256-block likewise
};
struct DqManyParams {
  DqItem item[kDqManyMax];
  int32_t count;   // >= 1
  int64_t total;   // sum of nb
  int64_t groups;  // sum of ceil(nb / 256)
};
cudaError_t launch_double_quant_many(const DqManyParams& p, int dq_code, void* workspace, cudaStream_t stream,
                                     int num_sms);

// blocksize 32, 64, 128 or 256
cudaError_t launch_dequantize(const uint8_t* packed, const Scales& s, int64_t n, int blocksize, void* out,
                              bool out_bf16, cudaStream_t stream, int num_sms);

// one CTA per 16-row tile (gemv.cu); batch up to 64
cudaError_t launch_gemv(const uint8_t* packed, const Scales& s, int64_t rows, int64_t cols, const void* x,
                        int batch, void* y, unsigned* err, cudaStream_t stream, int num_sms);

// several weights (same cols and scale kind) on one input in one launch, count <= kMaxGroup
constexpr int kMaxGroup = 4;
cudaError_t launch_gemv_group(const uint8_t* const* packed, const Scales* s, const int64_t* rows, int count,
                              int64_t cols, const void* x, int batch, void* const* y, unsigned* err,
                              cudaStream_t stream, int num_sms);

// one GEMV of the persistent stream: weight [rows, cols] (rows % 16 == 0, cols % 64 == 0), its input x [batch, cols]
// and output y [batch, rows]; up to kMaxStreamItems of them in one launch, batch 1..8
struct GemvItem {
  const uint8_t* packed;
  Scales s;
  const void* x;
  void* y;
  int64_t rows, cols;
};
constexpr int kMaxStreamItems = 256;
cudaError_t launch_gemv_items(const GemvItem* items, int count, int batch, unsigned* err, cudaStream_t stream,
                              int num_sms);

size_t gemm_workspace_bytes(int64_t rows, int64_t cols, int64_t m);
cudaError_t launch_gemm(const uint8_t* packed, const Scales& s, int64_t rows, int64_t cols, const void* x,
                        int64_t m, void* y, void* workspace, unsigned* err, cudaStream_t stream, int num_sms);

// 4-bit matmul plus a low-rank adapter: T = scale * X . A^T as a bf16 pair [hi | lo] into the first bytes of
// the workspace ([m, 64] bf16), then the GEMM with one adapter stage per output tile (r in {16, 32})
cudaError_t launch_lora_down(const void* x, const void* a, int64_t m, int64_t cols, int r, float scale, void* t,
                             cudaStream_t stream);
size_t gemm_lora_workspace_bytes(int64_t rows, int64_t cols, int64_t m);
cudaError_t launch_gemm_lora(const uint8_t* packed, const Scales& s, int64_t rows, int64_t cols, const void* x,
                             int64_t m, const void* lora_down, const void* lora_up, int lora_r, float lora_scale,
                             void* y, void* workspace, unsigned* err, cudaStream_t stream, int num_sms);

// input gradient dX = dY . Wc (rows % 64 == 0, cols % 128 == 0)
size_t gemm_dx_workspace_bytes(int64_t rows, int64_t cols, int64_t m);
cudaError_t launch_gemm_dx(const uint8_t* packed, const Scales& s, int64_t rows, int64_t cols, const void* dy,
                           int64_t m, void* dx, void* workspace, unsigned* err, cudaStream_t stream, int num_sms);

// products grouped by expert: rows [offsets[e], offsets[e + 1]) of `in` with expert e's weight, rows
// [e * rows, (e + 1) * rows) of the stacked weight (rows % 128 == 0, cols % 64 == 0; for the gradient rows % 64 == 0,
// cols % 128 == 0; experts * rows, cols and m within int32)
constexpr int kMaxExperts = 256;
struct ExpertsCall {
  const uint8_t* packed;
  Scales scales;
  int experts;
  int64_t rows, cols;  // of one expert
  const int* offsets;  // device, experts + 1
  const void* in;      // [m, cols], or [m, rows] for the gradient
  int64_t m;           // >= 1
  void* out;           // [m, rows], or [m, cols]
  void* workspace;     // experts_workspace_bytes, or null when that is 0
};
// CTA pairs with tiles of 256 rows, or CTAs alone with tiles of 64?  A stage costs about the same in either (it is the
// decode of 128 weight rows per CTA), so the rounds over the SMs decide, for rows spread evenly over the experts; alone,
// the last round can be split (where the reduction is long enough) and counts by its share.  2 experts of 256x4096, 1000
// rows: 4 pair units are one round, 32 units alone, split, a quarter of one (25.0 against 16.8 us).  Where pairs are taken with
// little to spare: 10 experts of 2048x4096, 128 rows each, 2 rounds of pairs against 320 units alone, 38 against 55 us (the
// gradient of 4096x2048, whose pairs pay for their hand-over, 54 against 67).
inline bool experts_pair(int64_t m, int experts, int64_t out_cols, int64_t reduction, int num_sms) {
  const int64_t each = (m + experts - 1) / experts;
  if (each <= 64) return false;
  const int64_t alone = experts * ((each + 63) / 64) * (out_cols / 128);
  const int64_t pairs = experts * ((each + 255) / 256) * ((out_cols + 255) / 256), workers = num_sms > 1 ? num_sms / 2 : 1;
  const int64_t rounds = (pairs + workers - 1) / workers;
  return reduction < 1024 ? rounds <= (alone + num_sms - 1) / num_sms : rounds * num_sms <= alone;
}
// Split reductions (tiles of 64 rows only): arrival counters, then one fp32 accumulator per item, at most kExpertsItems
// items per SM.
constexpr int kExpertsMaxSplit = 8;
constexpr int kExpertsItems = 4;
constexpr size_t kExpertsCountBytes = 4096;  // fewer split units than SMs, 4 counters each
// of one accumulator: up to 32 rows lie closer together
inline size_t experts_partial_bytes(int64_t m) { return m > 32 ? 64 * 128 * 4 : 32 * 128 * 4; }
// 0 where m rows are not split, else a size that does not depend on m (one buffer serves every m, and m = 1 is split where
// any m is)
inline size_t experts_workspace_bytes(int64_t m, int experts, int64_t out_cols, int64_t reduction, int num_sms) {
  // no split is worth its exchange where a unit is short, and little where even the fewest possible units make many rounds
  if (reduction < 1024 || num_sms > 255 || experts_pair(m, experts, out_cols, reduction, num_sms)) return 0;
  if ((m + 63) / 64 * (out_cols / 128) > 8 * (int64_t)num_sms) return 0;
  return kExpertsCountBytes + (size_t)kExpertsItems * num_sms * experts_partial_bytes(64);
}
cudaError_t launch_gemm_experts(const ExpertsCall& c, unsigned* err, cudaStream_t stream, int num_sms);
cudaError_t launch_gemm_experts_dx(const ExpertsCall& c, unsigned* err, cudaStream_t stream, int num_sms);

// a weight of uniform 4-bit codes with group scales (see group.cuh); the quantizer writes through these pointers
struct GroupWeight {
  const uint8_t* packed;  // [rows, cols / 2]
  const void* scale;      // [rows, cols / group] bf16 or fp16
  const uint8_t* zero;    // [rows, cols / group], or null: 8 everywhere
  int64_t rows, cols;     // cols a multiple of group
  int group;              // 32, 64 or 128
  bool half;              // fp16 scales (else bf16)
};
// src_dtype / out_dtype: 0 fp32, 1 bf16, 2 fp16
cudaError_t launch_quantize_groups(const void* src, int src_dtype, const GroupWeight& g, cudaStream_t stream,
                                   int num_sms);
cudaError_t launch_dequantize_groups(const GroupWeight& g, void* out, int out_dtype, cudaStream_t stream,
                                     int num_sms);
// x and y of the scales' type, batch 1..8
cudaError_t launch_gemv_groups(const GroupWeight& w, const void* x, int batch, void* y, cudaStream_t stream,
                               int num_sms);

// failure-path self-test: a bounded wait that runs out (see selftest.cu)
cudaError_t launch_wait_timeout(unsigned* err, cudaStream_t stream);

}  // namespace nf4
