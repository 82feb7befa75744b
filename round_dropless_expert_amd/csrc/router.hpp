// Internal interface of the operators around the experts' products. All
// launchers enqueue on the given stream and return the launch's error.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ragged.hpp"

namespace moe {

// Experts a token chooses at most, and groups of experts: a wavefront's lanes.
constexpr int kRouterMaxTopK = 64;
constexpr int kRouterMaxGroups = 64;

struct RouterParams {
  const void* logits;  // [T][E], ld apart
  const float* bias;   // [E] or NULL
  int32_t* idx;        // [T][k]
  float* weight;       // [T][k]
  int64_t T, ld;
  ElemType type;       // of logits
  int E, k;
  int groups, per_group, top_groups, group_top;
  float scale;
  bool sigmoid, renormalize;
  bool vec;            // rows are 16-byte aligned and hold whole vectors
  bool bias_vec;       // and so is bias
  int lanes_per_group, group_factor; // set by the launch
};
hipError_t launch_router(RouterParams p, hipStream_t st);

struct RouterGradParams {
  const void* logits;
  const int32_t* idx;
  const float* dweight;
  void* dlogits;
  int64_t T, ld;
  int E, k;
  float scale;
  bool sigmoid, renormalize;
  bool vec;
};
hipError_t launch_router_backward(ElemType t, const RouterGradParams& p, int num_cus,
                                  hipStream_t st);

// Workspace of the sort: int32 counts of its chunks.
size_t sort_bytes(int64_t n, int E);
hipError_t launch_sort(int64_t n, int E, const int32_t* idx, int32_t* perm, int32_t* pos,
                       int32_t* offsets, int32_t* counts, hipStream_t st);

struct CollectParams {
  const void* z;        // [rows], ld_z apart
  const void* dy;       // [T], ld_y apart
  const int32_t* pos;   // [T][k]
  const float* weight;  // [T][k] or NULL
  void* y;              // [T], ld_y apart
  void* dz;             // [rows], ld_dz apart, or NULL
  float* dweight;       // [T][k] or NULL
  int64_t T, rows, d, ld_z, ld_y, ld_dz;
  int k;
};
hipError_t launch_collect(ElemType t, const CollectParams& p, int num_cus, hipStream_t st);
hipError_t launch_collect_backward(ElemType t, const CollectParams& p, int num_cus,
                                   hipStream_t st);

// Codes of an 8-bit row at most: a product of two is at most 127^2 (2^14 with a
// program's own -128), so 2^17 - 1 of them sum below 2^31.
constexpr int kInt8MaxWidth = (1 << 17) - 1;
inline int64_t int8_stride(int64_t K) { return (K + 15) / 16 * 16; }
hipError_t launch_int8_quantize(ElemType t, int64_t rows, int64_t K, const void* x, int64_t ld_x,
                                int64_t src_rows, const int32_t* index, int index_div,
                                const int32_t* n_rows, int8_t* codes, float* scales, int num_cus,
                                hipStream_t st);
hipError_t launch_int8_dequantize(ElemType t, int64_t rows, int64_t K, const int8_t* codes,
                                  const float* scales, void* y, int64_t ld_y,
                                  const int32_t* n_rows, int num_cus, hipStream_t st);
hipError_t launch_int8_gemm(const RaggedShape& s, const int32_t* offsets, const int8_t* xq,
                            const float* xs, const int8_t* wq, const float* ws, void* y,
                            int num_cus, hipStream_t st);

constexpr int kOrthoMaxSide = 16384;
constexpr int kOrthoMaxSteps = 32;
// Orthogonalised updates of E matrices [N][K].
size_t orthogonalize_bytes(int E, int N, int K);
hipError_t launch_orthogonalize(ElemType t, int E, int N, int K, const void* g, void* y, int steps,
                                const float* coefficients, float scale, char* ws, int num_cus,
                                hipStream_t st);

}  // namespace moe
