// Global loads of the general ragged product kernel: which 16 bytes each thread
// takes of an operand's stage, and which stages are loaded unchecked. Free of
// device builtins, so that the same code runs on the host against buffers that
// end where their memory ends.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace moe {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// 16 bytes of a row of which `n` elements exist (n may be <= 0), the rest
// zero. `room`: if there are fewer than 16 bytes, so many more lie before
// `at` in the row, and one load ending at the last element serves. The address
// need only be aligned to an element: gfx950 loads 16 bytes from any address.
template <typename T>
__host__ __device__ __forceinline__ u32x4 load16(const T* at, int n, bool room) {
  constexpr int kV = 16 / sizeof(T);
  union {
    T e[kV];
    u32x4 v;
  } r;
  r.v = u32x4{0, 0, 0, 0};
  if (n >= kV) {
    __builtin_memcpy(&r.v, at, 16);
    return r.v;
  }
  if (n <= 0) return r.v;
  if (room) {
    unsigned __int128 w;
    __builtin_memcpy(&w, at - (kV - n), 16);
    w >>= (kV - n) * 8 * (int)sizeof(T);
    __builtin_memcpy(&r.v, &w, 16);
    return r.v;
  }
#pragma unroll
  for (int i = 0; i < kV; ++i)
    if (i < n) r.e[i] = at[i];
  return r.v;
}

// Stages of kCk values of c in which `count` of them are summed: `whole` ones
// that are loaded unchecked, from the first c on, and at most two checked ones
// behind them, which hold at least `keep` values of c (where there are so many).
struct StageSplit {
  int whole, checked;
};
__host__ __device__ __forceinline__ StageSplit split_stages(int count, int kCk, int keep) {
  const int whole = count > keep ? (count - keep) / kCk : 0;
  return StageSplit{whole, (count - whole * kCk + kCk - 1) / kCk};
}

// One operand's share of a stage: `kExt` rows of its output index by kStage
// bytes of c, as 16-byte pieces. kAlong: c lies along the operand's rows,
// otherwise down its columns.
template <typename T, bool kAlong, int kExt, int kStage>
struct OperandLoads {
  static constexpr int kEs = sizeof(T);
  static constexpr int kV = 16 / kEs;
  static constexpr int kCk = kStage / kEs;
  static constexpr int kChunks = kStage / 16;  // of a row along c
  static constexpr int kPieces = kExt * kChunks / 256;  // 16-byte pieces per thread
  typedef u32x4 regs_t[kPieces];

  const T* base;  // c = 0 of the tile's first row
  int64_t ld;
  int ext;  // rows of the output index that exist
  // Where this thread's pieces of a whole stage lie, from the stage's first
  // c: rows past ext read the last one instead (they feed outputs that are
  // never stored).
  int64_t at[kPieces];
  // Values of c that have to follow an unchecked stage. None if no such load
  // leaves its row. Otherwise (down, a last, partial chunk of columns) a load
  // reads up to kV - 1 elements past its row's end: they lie in the next row
  // where rows are so far apart, and in the next kV - 1 rows at any distance.
  int keep;
  bool room;  // down: a row has 16 bytes up to the tile's last column

  // `before`: rows of the output index before the tile's
  __host__ __device__ __forceinline__ void set(const T* b, int64_t l, int e, int before, int tid) {
    base = b;
    ld = l;
    ext = e;
    room = before + e >= kV;
    keep = kAlong || ext >= kExt || ext % kV == 0 ? 0 : ld >= kV - ext % kV ? 1 : kV - 1;
#pragma unroll
    for (int u = 0; u < kPieces; ++u) {
      const int id = tid + 256 * u;
      if constexpr (kAlong) {
        const int row = id / kChunks;
        at[u] = (row < ext ? row : ext - 1) * ld + (id % kChunks) * kV;
      } else {
        constexpr int kPer = kExt * kEs / 16;
        const int row = (id % kPer) * kV;
        at[u] = (id / kPer) * ld + (row < ext ? row : 0);
      }
    }
  }
  // pieces of a whole stage at c0
  __host__ __device__ __forceinline__ void load(regs_t& reg, int c0) const {
    const T* from = base + (kAlong ? c0 : c0 * ld);
#pragma unroll
    for (int u = 0; u < kPieces; ++u) __builtin_memcpy(&reg[u], from + at[u], 16);
  }
  // pieces of the stage at c0, where c exists below c_end
  __host__ __device__ __forceinline__ void load_some(regs_t& reg, int c0, int c_end,
                                                     int tid) const {
#pragma unroll
    for (int u = 0; u < kPieces; ++u) {
      const int id = tid + 256 * u;
      if constexpr (kAlong) {
        const int row = id / kChunks, c = c0 + (id % kChunks) * kV;
        reg[u] = load16(base + row * ld + c, row < ext ? c_end - c : 0, c_end >= kV);
      } else {
        constexpr int kPer = kExt * kEs / 16;
        const int c = c0 + id / kPer, row = (id % kPer) * kV;
        reg[u] = load16(base + c * ld + row, c < c_end ? ext - row : 0, room);
      }
    }
  }
};

}  // namespace moe
