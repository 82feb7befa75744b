// Launch of the LDS-ring product kernels (ragged_ring.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace moe {

enum class RingKind {
  kForwardBF16,
  kForwardF16,
  kInputGradBF16,
  kInputGradF16,
  kMxBF16,  // MXFP4 operands, by the output's type
  kMxF16,
  kMxF32
};

// Rows of every operand start at 16-byte boundaries and hold whole 16-byte
// chunks of c; strides are in bytes, below 2^22.
struct RingParams {
  const char* act;  // [rows], cbytes of c each, lda apart
  const char* w;    // [E] matrices of wbytes: [B] rows of cbytes (forward), or
                    // [C] rows of B 16-bit features (input gradient), ldw apart
  char* out;        // [rows][B], ldo apart
  const char* act_scales;  // MXFP4: [rows], lds apart
  const char* w_scales;    // [E][B], lds apart
  const int32_t* offsets;
  int64_t lda, ldw, ldo, lds, wbytes;
  int rows, E, B;
  int C;       // input gradient: rows of a weight matrix
  int cbytes;  // bytes of c in a row of act
  int out_vec; // rows of out are 16-byte aligned and hold whole chunks
};

// Weight gradient: strides in bytes (16-byte multiples), chunk * stride below
// 2^31.
struct WgradRingParams {
  const char* dy;  // [rows][N], ldy apart
  const char* x;   // [rows][K], ldx apart
  float* dw;       // [E][N][K]
  float* slots;    // [n_slots][N][K]
  const int32_t* offsets;
  int64_t ldy, ldx;
  int rows, E, N, K;
  int chunk, n_slots;
  int accumulate;
  int group;       // set by the launch: workgroups that take a chunk's tiles together
};

hipError_t launch_wgrad_ring(bool is_bf16, const WgradRingParams& params, int num_cus,
                             hipStream_t st);

// The same products for experts of few rows (ragged_skinny.hip; forward
// kinds).
hipError_t launch_skinny(RingKind kind, const RingParams& p, int num_cus, hipStream_t st);

hipError_t launch_ring(RingKind kind, const RingParams& p, int num_cus, hipStream_t st);

}  // namespace moe
