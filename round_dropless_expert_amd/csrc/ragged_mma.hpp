// What the LDS-ring kernels of the ragged operators share: LDS-direct loads,
// their waits, accumulator reads and the tile store.
#pragma once

#include "ragged_device.hpp"

namespace moe {

typedef __attribute__((address_space(3))) char lds_char;
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr int kRsrcWord3 = 0x00020000;  // raw buffer
constexpr int kNonTemporal = 2;         // cache policy of a buffer operation
// Past every buffer range (all below 2^31): loads return zeros, stores drop.
constexpr uint32_t kOutOfRange = 0x80000000u;

// LDS-direct loads of 16 or 4 bytes a lane: lane i's voff + soff of the
// buffer to LDS at lds + size * i. In asm, so that the compiler neither
// moves them nor waits on them: every wait is the kernel's own vmcnt count.
// They have no register results.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void lds_load16(__amdgpu_buffer_rsrc_t rsrc, uint32_t voff,
                                           uint32_t soff, uint32_t lds) {
  asm volatile(
      "s_mov_b32 m0, %0\n\t"
      "s_nop 0\n\t"
      "buffer_load_dwordx4 %1, %2, %3 offen lds"
      :
      : "s"(lds), "v"(voff), "s"(rsrc), "s"(soff)
      : "m0");
}
__device__ __forceinline__ void lds_load4(__amdgpu_buffer_rsrc_t rsrc, uint32_t voff,
                                          uint32_t soff, uint32_t lds) {
  asm volatile(
      "s_mov_b32 m0, %0\n\t"
      "s_nop 0\n\t"
      "buffer_load_dword %1, %2, %3 offen lds"
      :
      : "s"(lds), "v"(voff), "s"(rsrc), "s"(soff)
      : "m0");
}
#pragma clang diagnostic pop

// At most N of this wavefront's vector-memory operations outstanding, its
// LDS reads done, then the workgroup barrier.
template <int N>
__device__ __forceinline__ void wait_vmem_barrier() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(N) : "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// An accumulator element, read from its AGPR at this point of the program.
__device__ __forceinline__ float acc_read(float a) {
  float v;
  asm volatile("v_accvgpr_read_b32 %0, %1" : "=v"(v) : "a"(a));
  return v;
}

__device__ __forceinline__ int acc_read(int a) {
  int v;
  asm volatile("v_accvgpr_read_b32 %0, %1" : "=v"(v) : "a"(a));
  return v;
}

// What a sum is multiplied by before it is stored: nothing, or a scale of its
// row and one of its column (floats, from the tile's first on; reads past the
// last return zeros).
struct NoScale {
  static constexpr bool kOn = false;
};
struct RowColScale {
  static constexpr bool kOn = true;
  __amdgpu_buffer_rsrc_t rows, cols;
  __device__ __forceinline__ float row(int r) const {
    return __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(rows, r * 4, 0, 0));
  }
  __device__ __forceinline__ f32x4 col4(int c) const {
    return __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(cols, c * 4, 0, 0));
  }
};

// A wavefront's part of a tile's output: rows of `out` (ldo bytes apart, mr of
// them in the tile), columns n0 .. of B. Lane (l32, half) holds, for row l32
// of a 32-row block, columns 8 q + 4 half + 0..3 of each 32-column block. The
// wavefront turns 32 rows x 128 bytes around in 4 KiB of LDS and stores whole
// 128-byte row pieces (kVec: rows are 16-byte aligned and hold whole
// chunks). 16-byte chunk q of row r sits at q ^ (r % 8), against bank
// conflicts. kAdd: added to what is there. (The accumulators are read by
// asm: the caller gives the last MFMAs the wait states that the compiler
// cannot see.)
template <typename Out, int WI, int WJ, bool kVec, bool kAdd, int kPolicy, typename Acc,
          typename Scale = NoScale>
__device__ __forceinline__ void store_tile(const Acc (&acc)[WI][WJ], char* stg, char* out,
                                           uint32_t ldo, int mr, int B, int n0, int wn, int wm,
                                           int lane, const Scale& scale = Scale()) {
  constexpr int BN = 64 * WI, BM = 64 * WJ;
  constexpr int kOs = sizeof(Out), kPerBlk = kOs == 2 ? 2 : 1;  // 32-column blocks
  constexpr int kChunk = 16 / kOs;
  static_assert(!kAdd || kOs == 4, "added in fp32");
  typedef Out vec_t __attribute__((ext_vector_type(kChunk)));
  const int half = lane >> 5, l32 = lane & 31;
  const __amdgpu_buffer_rsrc_t ro = __builtin_amdgcn_make_buffer_rsrc(
      (void*)out, 0, (int)((uint32_t)(mr - 1) * ldo + (uint32_t)B * kOs), kRsrcWord3);
  const int rrow = lane >> 3, rchunk = lane & 7;
  f32x4 col_scale[Scale::kOn ? WI * 4 : 1];
  if constexpr (Scale::kOn)
#pragma unroll
    for (int i = 0; i < WI * 4; ++i)
      col_scale[i] = scale.col4(wn * (BN / 2) + i * 8 + 4 * half);
#pragma unroll
  for (int jb = 0; jb < WJ; ++jb) {
    const int row0 = wm * (BM / 2) + jb * 32;
    float row_scale = 1.f;
    if constexpr (Scale::kOn) row_scale = scale.row(row0 + l32);
#pragma unroll
    for (int ip = 0; ip < WI / kPerBlk; ++ip) {
#pragma unroll
      for (int u = 0; u < kPerBlk; ++u) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          typedef Out vec4_t __attribute__((ext_vector_type(4)));
          vec4_t o;
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            const auto sum = acc_read(acc[kPerBlk * ip + u][jb][4 * q + v]);
            if constexpr (Scale::kOn)
              o[v] = from_f32<Out>((float)sum * row_scale *
                                   col_scale[(kPerBlk * ip + u) * 4 + q][v]);
            else
              o[v] = from_f32<Out>(sum);
          }
          if constexpr (kOs == 2) {
            const int chunk = (u * 4 + q) ^ (l32 & 7);
            *reinterpret_cast<u32x2*>(stg + l32 * 128 + chunk * 16 + half * 8) =
                __builtin_bit_cast(u32x2, o);
          } else {
            const int chunk = (2 * q + half) ^ (l32 & 7);
            *reinterpret_cast<u32x4*>(stg + l32 * 128 + chunk * 16) =
                __builtin_bit_cast(u32x4, o);
          }
        }
      }
      const int col = n0 + wn * (BN / 2) + ip * 32 * kPerBlk + rchunk * kChunk;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = i * 8 + rrow;
        vec_t v = __builtin_bit_cast(vec_t, *reinterpret_cast<const u32x4*>(
                                                stg + r * 128 + ((rchunk ^ (r & 7)) * 16)));
        const uint32_t at = (uint32_t)(row0 + r) * ldo + (uint32_t)col * kOs;
        if constexpr (kVec) {
          // rows past mr fall past the range
          const uint32_t off = col < B ? at : kOutOfRange;
          if constexpr (kAdd)
            v += __builtin_bit_cast(
                vec_t, __builtin_amdgcn_raw_buffer_load_b128(ro, (int)off, 0, 0));
          __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, v), ro, (int)off, 0,
                                                 kPolicy);
        } else if (row0 + r < mr) {
          Out* o = reinterpret_cast<Out*>(out + at);
          if (col + kChunk <= B) {
            // gfx950 stores 16 bytes to any address
            if constexpr (kAdd) {
              vec_t was;
              __builtin_memcpy(&was, o, 16);
              v += was;
            }
            __builtin_memcpy(o, &v, 16);
          } else {
#pragma unroll
            for (int k = 0; k < kChunk; ++k)
              if (col + k < B) o[k] = kAdd ? o[k] + v[k] : v[k];
          }
        }
      }
    }
  }
}

}  // namespace moe
