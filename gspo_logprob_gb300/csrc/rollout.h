// Host-side declarations of the rollout operators (logit shaping, adapters beside
// the head), as internal.h has those of the head and its loss.
#pragma once
#include "internal.h"

namespace gh {

// kernel kinds after those of KernelKind
constexpr int K_SHAPE = 18;
constexpr int K_SHAPED_LOGP = 19;
constexpr int K_SHAPED_MERGE = 20;
constexpr int K_SHAPED_GRAD = 21;
constexpr int K_ADAPTER_LOW = 22;
constexpr int K_ADAPTER_TC = 23;
static_assert(K_ADAPTER_TC + 1 == GH_NUM_KERNEL_KINDS, "a name for every kind");

// bf16 [depth, rows, inner] tensor map read in boxes of 16 elements by box_rows
// rows, 32-byte swizzle, zero fill out of bounds (strides in bytes).
bool make_tmap_bf16_k16(CUtensorMap* map, const void* base, uint64_t inner, uint64_t rows, uint64_t depth,
                        uint64_t row_stride, uint64_t depth_stride, uint32_t box_rows);

// --- logit shaping (shape_kernels.cu) -----------------------------------------
constexpr int SHAPE_MAX_HIST = (1 << 20) - 1;  // history tokens a row may have
constexpr int SHAPE_MAX_BIAS = 2047;           // entries of a bias list
constexpr int SHAPE_MIN_SEG = 512;             // columns of the shortest partial of the log-prob
struct ShapeArgs {
  gh_shaping s;
  int R, V;
  int dtype, out_dtype;  // gh_dtype of the logits and of `out`
  const void* logits;
  int64_t ld;
  void* out;  // shaped logits or dlogits
  int64_t out_ld;
  const int32_t* targets;
  const uint8_t* mask;
  const float* lse;
  const float* coef;
  const float* grad_out;
  float2* part;  // [R, segments] (max, sum of exp(z' - max))
  float* zy;     // [R]
  float* logp;
  float* lse_out;
  int* status;
  // set by the launchers
  int cols, ntiles, rows_per_cta, nseg, room;
  bool vec_in, vec_out;
};
int64_t shape_segments(int64_t V);
cudaError_t launch_shape(ShapeArgs a, cudaStream_t st);
// segment partials and target logits, and logp and LSE too where a.ntiles (which it sets) is 1
cudaError_t launch_shaped_logp(ShapeArgs& a, cudaStream_t st);
cudaError_t launch_shaped_merge(const ShapeArgs& a, cudaStream_t st);  // logp and LSE from them, after launch_shaped_logp
cudaError_t launch_shaped_grad(ShapeArgs a, cudaStream_t st);

// --- head with adapters (adapter_kernels.cu) -----------------------------------
struct AdapterPlan {
  int tile_rows;    // rows that share a list of adapters (and a tensor-core tile)
  int rank_chunks;  // 16-wide chunks of a rank
  int max_chunks;   // chunks a row tile may have
  int list_ld;
  int terms;        // bf16 terms that add up to u
  int64_t u_rows;   // rows of 16 elements
  size_t u_bytes, list_bytes;
};
AdapterPlan adapter_plan(int64_t N, int64_t rank, int64_t num_adapters, int out_dtype);
struct AdapterArgs {
  int N, D, V, rank, num_adapters;
  int dtype, out_dtype;
  const void* H;
  const void* W;
  const void* A;
  const void* B;
  const float* scale;
  const int32_t* ids;
  void* out;
  int64_t ld;
  bool vec_out;  // output rows start on 16-byte boundaries
  void* U;       // bf16 [u_rows, 16], or fp32 [N, rank]
  int32_t* list;
  int* counter;  // bf16, one row tile: the warps of the launch that have written their part of U
  int tile_rows, rank_chunks, max_chunks, list_ld, terms;
  int* status;
};
// u, unless the product computes it itself (bf16, one row tile)
bool adapter_low_apart(const AdapterArgs& a);
cudaError_t launch_adapter_low(const AdapterArgs& a, cudaStream_t st);
cudaError_t launch_adapter_logits(const AdapterArgs& a, cudaStream_t st);

}  // namespace gh
