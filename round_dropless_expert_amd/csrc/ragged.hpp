// Internal interface of the ragged expert operators: products over rows
// sorted by expert and their gradients, SwiGLU, and the 4-bit format. All
// launchers enqueue on the given stream and return the launch's error.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace moe {

enum class ElemType { kF32 = 0, kBF16 = 1, kF16 = 2 };

inline int elem_bytes(ElemType t) { return t == ElemType::kF32 ? 4 : 2; }

// Experts a ragged call takes at most, and the widest row (elements): a
// tile of 256 rows then stays below 2^31 bytes, so offsets inside a tile
// are 32-bit while the tile's origin is a 64-bit address.
constexpr int kRaggedMaxExperts = 1024;
constexpr int64_t kRaggedMaxWidth = int64_t(1) << 20;

// y[i][n] = sum_k x[i][k] w[e][n][k] for the rows i of expert e,
// offsets[e] <= i < offsets[e + 1] (clamped to [0, rows]).
struct RaggedShape {
  int64_t rows;
  int E, N, K;
  ElemType type;
  int64_t ld_x, ld_y;  // elements
};

// Weight gradient: the rows of an expert are summed in chunks of at most
// `chunk` rows. Chunk 0 goes straight to dw, the others to fp32 slots
// [N][K] of the workspace, which a second launch adds in chunk order: the
// order of the sum is fixed by the shape, so results repeat bit for bit.
// There are at most rows / chunk slots.
struct DwSplit {
  int64_t chunk;
  int64_t slots;
};
DwSplit dw_split(const RaggedShape& s);

hipError_t launch_ragged_gemm(const RaggedShape& s, const int32_t* offsets, const void* x,
                              const void* w, void* y, int num_cus, hipStream_t st);
hipError_t launch_ragged_dx(const RaggedShape& s, const int32_t* offsets, const void* dy,
                            const void* w, void* dx, int num_cus, hipStream_t st);
hipError_t launch_ragged_dw(const RaggedShape& s, const int32_t* offsets, const void* x,
                            const void* dy, float* dw, float* slots, bool accumulate,
                            int num_cus, hipStream_t st);

// h = silu(g) u for rows [g, u] of gu, and its gradient. n_rows: rows to
// process, on the device (clamped to [0, rows]), or NULL for all.
hipError_t launch_swiglu(ElemType t, int64_t rows, int64_t f, const void* gu, int64_t ld_gu,
                         void* h, int64_t ld_h, const int32_t* n_rows, int num_cus,
                         hipStream_t st);
hipError_t launch_swiglu_backward(ElemType t, int64_t rows, int64_t f, const void* gu,
                                  int64_t ld_gu, const void* dh, int64_t ld_dh, void* dgu,
                                  int64_t ld_dgu, const int32_t* n_rows, int num_cus,
                                  hipStream_t st);

// Values of a block that share one scale, and the bytes of a scale row.
constexpr int kMxBlock = 32;
inline int64_t mx_scale_stride(int64_t K) { return (K / kMxBlock + 3) / 4 * 4; }

hipError_t launch_mx_quantize(ElemType t, int64_t rows, int64_t K, const void* x, int64_t ld_x,
                              int64_t src_rows, const int32_t* index, int index_div,
                              const int32_t* n_rows, uint8_t* codes, uint8_t* scales,
                              int num_cus, hipStream_t st);
hipError_t launch_mx_dequantize(ElemType t, int64_t rows, int64_t K, const uint8_t* codes,
                                const uint8_t* scales, void* y, int64_t ld_y,
                                const int32_t* n_rows, int num_cus, hipStream_t st);
hipError_t launch_mx_gemm(const RaggedShape& s, const int32_t* offsets, const uint8_t* xq,
                          const uint8_t* xs, const uint8_t* wq, const uint8_t* ws, void* y,
                          int num_cus, hipStream_t st);

}  // namespace moe
