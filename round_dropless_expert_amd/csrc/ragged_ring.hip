// Products over rows sorted by expert through an LDS ring (gfx950 matrix
// cores): the forward and the input gradient for 16-bit types, and the
// forward for MXFP4 operands, where rows are 16-byte aligned.
//
//   out[i][b] = sum_c act[i][c] W(e, b, c)
//
// Forward: W(e, b, c) = w[e][b][c], both operands hold c along their rows.
// Input gradient: W(e, b, c) = w[e][c][b], c runs down the weights' columns.
//
// Persistent: one workgroup per CU walks output tiles, numbered expert by
// expert (row tile fastest), each XCD a contiguous run of them, so that the
// workgroups of an XCD share operand panels in its L2. A tile is 64 WI
// features x 64 WJ rows, 2 x 2 wavefronts of 32 WI x 32 WJ. The MFMA's row
// operand is a block of weight rows, its column operand a block of token
// rows, so a lane ends with runs of consecutive features of one token.
//
// c advances 64 bytes a row per stage: 32 values of 16 bits, 64 of 8 or 128 of
// 4, two MFMA steps either way (32x32x16, 32x32x32 or 32x32x64, all 32 cycles). SPB stages
// form a slot of a four-slot ring filled by LDS-direct loads, up to three
// slots in flight, one barrier per slot; the ring runs on into the next
// tile, whose first slots land while this one is stored. Fragment reads run
// one step ahead of the MFMAs, loads are spread between them.
//
// Every output is one fixed sequence of MFMA steps over ascending c, so a
// row's result does not depend on the tile, the tile's shape or the rows
// around it.
//
// Three tiles share this file. 256 x 256 (wide_ring_kernel, below) for experts
// of many rows; 256 x 128 and 128 x 64 (ring_kernel) where experts have few
// rows and a larger tile would multiply rows that do not exist. The small
// tiles are bound by reading the weights once: 512 rows over 64 experts, N =
// 4096, K = 1536, bf16 (805 MB of weights) 152-157 us, 5.2 TB/s; in MXFP4 (214
// MB) 54 us, 4.0 TB/s, and 42 where the last-level cache holds them. 64-byte
// stages and four slots there, since three stages in flight cover the memory's
// latency; the L2's request rate does not matter yet.
#include "ragged_ring.hpp"
#include "ring_body.hpp"

namespace moe {
namespace {

// Tiles of a ragged product, expert by expert. kRows: the experts' rows are kept
// in LDS too.
template <typename Op, typename Out, int BN, int BM, bool kOutVec, bool kRows>
struct RaggedJob {
  struct Tile {
    int e, start, m, n0, m0;
  };
  struct Table {
    int32_t tiles_to[kRaggedMaxExperts];  // tiles of the experts up to e
    int32_t n_tiles;
    int32_t first_row[kRows ? kRaggedMaxExperts : 1];
    int32_t n_rows[kRows ? kRaggedMaxExperts : 1];
  };
  static constexpr int kStaging = 4096;
  const RingParams& p;
  Table& table;

  // The tile table, by wavefront 0.
  __device__ __forceinline__ int setup(int wave, int lane) {
    const int nt = (p.B + BN - 1) / BN;
    if (wave == 0) {
      int carry = 0;
      for (int base = 0; base < p.E; base += kWave) {
        int start = 0, rows = 0;
        if (base + lane < p.E) expert_rows(p.offsets, base + lane, p.rows, &start, &rows);
        const int incl = wave_inclusive_scan((rows + BM - 1) / BM * nt) + carry;
        if (base + lane < p.E) {
          table.tiles_to[base + lane] = incl;
          if constexpr (kRows) {
            table.first_row[base + lane] = start;
            table.n_rows[base + lane] = rows;
          }
        }
        carry = __builtin_amdgcn_readlane(incl, kWave - 1);
        if ((uint32_t)carry > kMaxUnits) break;  // overlapping offsets: no tiles
      }
      if (lane == 0) table.n_tiles = (uint32_t)carry > kMaxUnits ? 0 : carry;
    }
    __syncthreads();
    return __builtin_amdgcn_readfirstlane(table.n_tiles);
  }

  __device__ __forceinline__ Tile locate(int t) const {
    const int lane = threadIdx.x & (kWave - 1);
    const int nt = (p.B + BN - 1) / BN;
    Tile T;
    int e = 0;
    for (int base = 0; base < p.E; base += kWave) {
      const bool before = base + lane < p.E && table.tiles_to[base + lane] <= t;
      e += __builtin_popcountll(__builtin_amdgcn_ballot_w64(before));
    }
    T.e = e;
    if constexpr (kRows) {
      T.start = table.first_row[e];
      T.m = table.n_rows[e];
    } else {
      expert_rows(p.offsets, e, p.rows, &T.start, &T.m);
    }
    T.start = __builtin_amdgcn_readfirstlane(T.start);
    T.m = __builtin_amdgcn_readfirstlane(T.m);
    const int mt = (T.m + BM - 1) / BM;
    const int local =
        t - (e > 0 ? __builtin_amdgcn_readfirstlane(table.tiles_to[e - 1]) : 0);
    place_tile(local, mt, nt, &T.m0, &T.n0);
    T.m0 *= BM;
    T.n0 *= BN;
    return T;
  }

  __device__ __forceinline__ int features(const Tile& T) const {
    return p.B - T.n0 < BN ? p.B - T.n0 : BN;
  }
  __device__ __forceinline__ int rows(const Tile& T) const {
    return T.m - T.m0 < BM ? T.m - T.m0 : BM;
  }

  template <bool kTransW>
  __device__ __forceinline__ void operands(const Tile& T, bool exists, __amdgpu_buffer_rsrc_t* rw,
                                           __amdgpu_buffer_rsrc_t* ra) const {
    const uint32_t lda = (uint32_t)p.lda, ldw = (uint32_t)p.ldw;
    const char* wb = p.w + (int64_t)T.e * p.wbytes;
    if constexpr (kTransW)  // features past B read the next row's: never stored
      *rw = __builtin_amdgcn_make_buffer_rsrc(
          (void*)(wb + (int64_t)T.n0 * 2), 0,
          exists ? (int)((uint32_t)(p.C - 1) * ldw + (uint32_t)(p.B - T.n0) * 2u) : 0, kRsrcWord3);
    else
      *rw = __builtin_amdgcn_make_buffer_rsrc(
          (void*)(wb + (int64_t)T.n0 * p.ldw), 0,
          exists ? (int)((uint32_t)(features(T) - 1) * ldw + (uint32_t)p.cbytes) : 0, kRsrcWord3);
    *ra = __builtin_amdgcn_make_buffer_rsrc(
        (void*)(p.act + ((int64_t)T.start + T.m0) * p.lda), 0,
        exists ? (int)((uint32_t)(rows(T) - 1) * lda + (uint32_t)p.cbytes) : 0, kRsrcWord3);
  }

  // MXFP4 scales of a tile's weight rows (w) or tokens
  __device__ __forceinline__ __amdgpu_buffer_rsrc_t scale_rows(const Tile& T, bool w,
                                                               bool exists) const {
    const int64_t row = w ? (int64_t)T.e * p.B + T.n0 : (int64_t)T.start + T.m0;
    return __builtin_amdgcn_make_buffer_rsrc(
        (void*)((w ? p.w_scales : p.act_scales) + row * p.lds), 0,
        exists ? (int)((uint32_t)(w ? features(T) : rows(T)) * (uint32_t)p.lds) : 0, kRsrcWord3);
  }
  // The same for reads of 16 bytes: a row's last may reach past it, into the
  // next row, or past the array, which the range ends (dword by dword).
  __device__ __forceinline__ __amdgpu_buffer_rsrc_t scale_lines(const Tile& T, bool w,
                                                                bool exists) const {
    const int64_t w_row = (int64_t)T.e * p.B + T.n0, row = (int64_t)T.start + T.m0;
    const int64_t left = ((w ? (int64_t)p.E * p.B - w_row : p.rows - row)) * p.lds;
    const int64_t most = (int64_t)(w ? features(T) : rows(T)) * p.lds + 12;
    return __builtin_amdgcn_make_buffer_rsrc(
        (void*)(w ? p.w_scales + w_row * p.lds : p.act_scales + row * p.lds), 0,
        exists ? (int)(left < most ? left : most) : 0, kRsrcWord3);
  }

  template <int WI, int WJ>
  __device__ __forceinline__ void store(const Tile& T, const typename Op::acc_t (&acc)[WI][WJ],
                                        char* stg, int wn, int wm, int lane) const {
    static_assert(BN == 64 * WI && BM == 64 * WJ, "the job's tile");
    const int64_t row = (int64_t)T.start + T.m0;
    char* out = p.out + row * p.ldo;
    if constexpr (Op::kInt) {
      RowColScale s;
      s.rows = __builtin_amdgcn_make_buffer_rsrc((void*)(p.act_scales + row * 4), 0, rows(T) * 4,
                                                 kRsrcWord3);
      s.cols = __builtin_amdgcn_make_buffer_rsrc(
          (void*)(p.w_scales + ((int64_t)T.e * p.B + T.n0) * 4), 0, (p.B - T.n0) * 4, kRsrcWord3);
      store_tile<Out, WI, WJ, kOutVec, false, kNonTemporal>(acc, stg, out, (uint32_t)p.ldo,
                                                            rows(T), p.B, T.n0, wn, wm, lane, s);
    } else {
      store_tile<Out, WI, WJ, kOutVec, false, kNonTemporal>(acc, stg, out, (uint32_t)p.ldo,
                                                            rows(T), p.B, T.n0, wn, wm, lane);
    }
  }
};

template <typename Op, typename Out, int WI, int WJ, int SPB, bool kTransW, bool kOutVec>
__global__ __launch_bounds__(256, 1) void ring_kernel(RingParams p) {
  typedef RaggedJob<Op, Out, 64 * WI, 64 * WJ, kOutVec, true> job_t;
  __shared__ typename job_t::Table table;
  job_t job{p, table};
  ring<Op, WI, WJ, SPB, kTransW>(job);
}

// The 256 x 256 tile on wide slots.
//
// 98304 rows over 64 experts, N = 4096, K = 7168: bf16 4.6-4.8 ms, 1.20-1.25
// PFLOP/s, MFMA pipes busy 76% of the cycles at 1.7 GHz (of 2.4: the chip's
// power limit); MXFP4 1.44-1.55 ms, 3.7-4.0 PFLOP/s, busy 60% at 1.7 GHz, the
// rest waits for a slot's loads (1.4e8 requests to the L2: one a CU every 4.6
// cycles). The same on 64-byte stages in four slots: 5.01 and 2.02 ms. Input
// gradient, 32768 rows over 32 experts, N = K = 2048, bf16: 264-291 us, 0.94-1.04
// PFLOP/s.
// In 8-bit integers the same product takes 2.45-2.5 ms, 2.3-2.35 POP/s (a large library
// product reaches 2.1-2.2): MFMA pipes busy 78% of the cycles at 1.4 GHz, the chip's
// power limit for them. 512 rows over 64 experts, N = 4096, K = 1536 (409 MB): 81 us, 5.0
// TB/s, in the 128 x 64 tile.
template <typename Op, typename Out, bool kTransW, bool kOutVec>
__global__ __launch_bounds__(256, 1) void wide_ring_kernel(RingParams p) {
  typedef RaggedJob<Op, Out, 256, 256, kOutVec, false> job_t;
  __shared__ typename job_t::Table table;
  job_t job{p, table};
  wide_ring<Op, kTransW>(job);
}

// Products that go to the skinny kernel: fewer tiles of the ring's smallest
// shape than CUs, and at most 32 rows a (mean) expert or two of the skinny
// kernel's 32 x 16 blocks a CU. Skinny against ring, bf16, one expert: 4096 x
// 4096, a row 8.6 and 30 us, 32 rows 15 and 30, 64 rows (512 blocks) 20 and
// 31, 128 rows (1024 blocks) 38 and 27; 1024 x 4096, 256 rows (512 blocks) 17
// and 26. With a tile for every CU the ring is the faster for single rows too
// (eight experts of 4096 x 1536, a row each: 17 against 24 us).
bool skinny_takes(const RingParams& p, int num_cus) {
  const int64_t active = p.rows < p.E ? p.rows : p.E;
  const int64_t mean = (p.rows + active - 1) / active;
  return active * ((mean + 63) / 64) * ((p.B + 127) / 128) < num_cus &&
         (mean <= 32 ||
          active * ((mean + 31) / 32) * ((p.B + 15) / 16) <= 2 * (int64_t)num_cus);
}

template <typename Op, typename Out, int WI, int WJ, int SPB, bool kTransW>
hipError_t launch(const RingParams& p, int grid, hipStream_t st) {
  if (p.out_vec)
    hipLaunchKernelGGL((ring_kernel<Op, Out, WI, WJ, SPB, kTransW, true>), dim3((unsigned)grid),
                       dim3(256), 0, st, p);
  else
    hipLaunchKernelGGL((ring_kernel<Op, Out, WI, WJ, SPB, kTransW, false>), dim3((unsigned)grid),
                       dim3(256), 0, st, p);
  return hipGetLastError();
}

// Output tile: features x rows of an expert. The offsets are on the device,
// so the choice goes by the experts' mean number of rows: waves of tiles over
// the CUs times a tile's area over its relative speed.
template <typename Op, typename Out, bool kTransW>
hipError_t choose(const RingParams& p, int num_cus, hipStream_t st) {
  const int64_t active = p.rows < p.E ? p.rows : p.E;
  const int64_t mean = (p.rows + active - 1) / active;
  auto cost = [&](int bn, int bm, float speed) {
    const int64_t tiles = active * ((mean + bm - 1) / bm) * ((p.B + bn - 1) / bn);
    return (float)((tiles + num_cus - 1) / num_cus) * (float)bn * (float)bm / speed;
  };
  const float big = cost(256, 256, 1.0f), medium = cost(256, 128, 0.85f),
              small = cost(128, 64, 0.45f);
  const int grid = num_cus < 8 ? 8 : num_cus / 8 * 8;
  if (big <= medium && big <= small) {
    if (p.out_vec)
      hipLaunchKernelGGL((wide_ring_kernel<Op, Out, kTransW, true>), dim3((unsigned)grid),
                         dim3(256), 0, st, p);
    else
      hipLaunchKernelGGL((wide_ring_kernel<Op, Out, kTransW, false>), dim3((unsigned)grid),
                         dim3(256), 0, st, p);
    return hipGetLastError();
  }
  if (medium <= small) return launch<Op, Out, 4, 2, 1, kTransW>(p, grid, st);
  return launch<Op, Out, 2, 1, 2, kTransW>(p, grid, st);
}

}  // namespace

hipError_t launch_ring(RingKind kind, const RingParams& p, int num_cus, hipStream_t st) {
  if (kind != RingKind::kInputGradBF16 && kind != RingKind::kInputGradF16 &&
      skinny_takes(p, num_cus))
    return launch_skinny(kind, p, num_cus, st);
  switch (kind) {
    case RingKind::kForwardBF16: return choose<OpBf16, bf16, false>(p, num_cus, st);
    case RingKind::kForwardF16: return choose<OpF16, f16, false>(p, num_cus, st);
    case RingKind::kInputGradBF16: return choose<OpBf16, bf16, true>(p, num_cus, st);
    case RingKind::kInputGradF16: return choose<OpF16, f16, true>(p, num_cus, st);
    case RingKind::kMxBF16: return choose<OpMx, bf16, false>(p, num_cus, st);
    case RingKind::kMxF16: return choose<OpMx, f16, false>(p, num_cus, st);
    case RingKind::kMxF32: return choose<OpMx, float, false>(p, num_cus, st);
    case RingKind::kI8BF16: return choose<OpI8, bf16, false>(p, num_cus, st);
    case RingKind::kI8F16: return choose<OpI8, f16, false>(p, num_cus, st);
    default: return choose<OpI8, float, false>(p, num_cus, st);
  }
}

}  // namespace moe
