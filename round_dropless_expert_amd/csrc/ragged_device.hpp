// Device helpers of the ragged expert operators.
#pragma once

#include "device_common.hpp"
#include "ragged.hpp"

namespace moe {

typedef _Float16 f16;
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ float to_f32(f16 v) { return static_cast<float>(v); }
// float -> fp16 rounds to nearest even (v_cvt_f16_f32); past 65504 + half a
// step it is infinite.
template <>
__device__ __forceinline__ f16 from_f32<f16>(float v) { return static_cast<f16>(v); }

// Rows of expert e: [start, start + rows), with offsets clamped to [0, n],
// so that no offsets, however wrong, lead a kernel out of its buffers.
__device__ __forceinline__ void expert_rows(const int32_t* offsets, int e, int n, int* start,
                                            int* rows) {
  int a = offsets[e], b = offsets[e + 1];
  a = a < 0 ? 0 : (a > n ? n : a);
  b = b < 0 ? 0 : (b > n ? n : b);
  *start = a;
  *rows = b > a ? b - a : 0;
}

// Units (tiles, jobs) of one launch at most. Offsets in order stay far below
// (the ABI refuses larger shapes); overlapping ones can pass it, and are then
// not worked on: every sum of 64 experts' units fits 32 bits, so a check
// behind each keeps all of them exact.
constexpr uint32_t kMaxUnits = 1u << 26;

// The expert whose units hold unit t, when expert e owns units(rows_e)
// consecutive units: every wavefront scans 64 experts at a time. All lanes
// return the same values; false past the last unit.
struct ExpertUnit {
  int e, start, rows;  // the expert and its rows
  int first;           // its first unit
};
template <typename Units>
__device__ __forceinline__ bool find_unit(const int32_t* offsets, int E, int n, int t,
                                          Units units, ExpertUnit* out) {
  const int lane = threadIdx.x & (kWave - 1);
  int carry = 0;
  for (int base = 0; base < E; base += kWave) {
    const int e = base + lane;
    int start = 0, rows = 0, own = 0;
    if (e < E) {
      expert_rows(offsets, e, n, &start, &rows);
      own = units(rows);
    }
    const int incl = wave_inclusive_scan(own) + carry;
    carry = __builtin_amdgcn_readlane(incl, kWave - 1);
    if ((uint32_t)carry > kMaxUnits) return false;
    const int before = __builtin_popcountll(__builtin_amdgcn_ballot_w64(incl <= t));
    if (before < kWave && base + before < E) {
      out->e = base + before;
      out->start = __builtin_amdgcn_readlane(start, before);
      out->rows = __builtin_amdgcn_readlane(rows, before);
      out->first = __builtin_amdgcn_readlane(incl - own, before);
      return true;
    }
  }
  return false;
}

// The unit of this workgroup when the units are dealt to the XCDs in
// contiguous eighths (workgroup b runs on XCD b % 8): false where it has none.
template <typename Units>
__device__ __forceinline__ bool find_xcd_unit(const int32_t* offsets, int E, int n, Units units,
                                              int* t, ExpertUnit* out) {
  const int lane = threadIdx.x & (kWave - 1);
  const int xcd = (int)(blockIdx.x % 8), place = (int)(blockIdx.x / 8);
  int total = 0;
  for (int base = 0; base < E; base += kWave) {
    int start = 0, rows = 0, own = 0;
    if (base + lane < E) {
      expert_rows(offsets, base + lane, n, &start, &rows);
      own = units(rows);
    }
    const int incl = wave_inclusive_scan(own);
    total += __builtin_amdgcn_readlane(incl, kWave - 1);
    if ((uint32_t)total > kMaxUnits) return false;
    if (E <= kWave) {  // one pass finds it
      const int share = (total + 7) / 8;
      *t = xcd * share + place;
      if (place >= share || *t >= total) return false;
      const int l = __builtin_popcountll(__builtin_amdgcn_ballot_w64(incl <= *t));
      out->e = l;
      out->start = __builtin_amdgcn_readlane(start, l);
      out->rows = __builtin_amdgcn_readlane(rows, l);
      out->first = __builtin_amdgcn_readlane(incl - own, l);
      return true;
    }
  }
  const int share = (total + 7) / 8;
  *t = xcd * share + place;
  return place < share && find_unit(offsets, E, n, *t, units, out);
}

// Slots of the experts below e: an expert's chunks past its first.
__device__ __forceinline__ int slots_before(const int32_t* offsets, int e, int n, int chunk) {
  const int lane = threadIdx.x & 63;
  int sum = 0;
  for (int base = 0; base < e; base += kWave) {
    int start, rows, own = 0;
    if (base + lane < e) {
      expert_rows(offsets, base + lane, n, &start, &rows);
      own = rows > 0 ? (int)(((int64_t)rows + chunk - 1) / chunk) - 1 : 0;
    }
    sum += __builtin_amdgcn_readlane(wave_inclusive_scan(own), kWave - 1);
  }
  return sum;
}

// Rows that an elementwise call processes.
__device__ __forceinline__ int64_t live_rows(int64_t rows, const int32_t* n_rows) {
  if (!n_rows) return rows;
  const int64_t n = *n_rows;
  return n < 0 ? 0 : (n < rows ? n : rows);
}

}  // namespace moe
