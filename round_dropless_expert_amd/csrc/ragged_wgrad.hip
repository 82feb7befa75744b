// Weight gradient of the product over rows sorted by expert, 16-bit types,
// through an LDS ring (gfx950 matrix cores):
//
//   dw[e][n][k] = sum over e's rows i of dy[i][n] x[i][k]      (fp32)
//
// The contraction runs down the rows of both operands, while the matrix
// cores want each lane to hold consecutive rows of one column: stages of 32
// rows are copied into LDS as they lie, by LDS-direct loads that read 256
// bytes of a row at a time, and the fragments come back through gfx950's
// transposing LDS read. A workgroup computes a 256 (n) x 256 (k) tile of one
// expert's chunk of rows with 2 x 2 wavefronts of 128 x 128. Four LDS slots
// form a ring with three stages in flight. Persistent: the ring runs on
// across a workgroup's tiles, so that the next tile's first stages land
// while the current one is stored.
//
// Experts have very different numbers of rows, and a tile takes as long as
// its chunk has rows. The tiles of a chunk are dealt out in blocks of `group`
// (32 where a chunk has that many: the workgroups of one XCD, which then
// share the chunk's rows in its L2), largest chunk first, each block to the
// group of workgroups with the least work so far; past kDealt blocks they go
// round the groups in turn. Every workgroup works the whole deal out for
// itself, so it needs no memory and no order of arrival.
//
// An expert with more rows than a chunk is summed in several tiles; those
// past the first go to slots of the workspace and a second launch adds them
// in chunk order.
//
// 32768 rows over 32 experts, N = K = 2048, bf16: 316-349 us, 790-870 TFLOP/s;
// the slots' addition 13 us more. The MFMA pipes are busy 45% of the cycles. By
// variants that left work out: the loads cost 85 us (each stage is 32 rows of
// 512 bytes from two operands, and a tile has only some 32 stages), the
// store of the fp32 tile 64 us (537 MB of dw in all), the fragment reads 16.
//
// Every workgroup orders the experts by E^2 comparisons in LDS, which counts at
// the most experts: 16384 rows, N = K = 256, 512 experts (134 MB of dw) 64 us,
// 1024 (268 MB, 56 us at a copy's rate) 177; the general kernel takes 73 and 211.
#include "ragged_mma.hpp"
#include "ragged_ring.hpp"

namespace moe {
namespace {

constexpr int kTile = 256;
constexpr int kStageRows = 32;
constexpr int kOpBytes = kStageRows * kTile * 2;  // one operand's stage
constexpr int kSlotBytes = 2 * kOpBytes;          // dy, then x
constexpr int kSlots = 4;
constexpr int kLoads = kSlotBytes / (256 * 16);  // 16-byte loads per thread and stage
template <typename T>
__device__ __forceinline__ f32x16 mma(u32x4 a, u32x4 b, f32x16 c) {
  if constexpr (__is_same(T, bf16))
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a),
                                                  __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

// Smallest value of the 64 lanes.
__device__ __forceinline__ uint32_t wave_min(uint32_t v) {
#define MOE_MIN_STEP(ctrl, rows)                                                             \
  {                                                                                          \
    const uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp((int)0xffffffff, (int)v, ctrl,  \
                                                             rows, 0xf, false);              \
    v = v < o ? v : o;                                                                       \
  }
  MOE_MIN_STEP(0x111, 0xf)  // row_shr:1, 2, 4, 8: lane 15 of each row of 16
  MOE_MIN_STEP(0x112, 0xf)
  MOE_MIN_STEP(0x114, 0xf)
  MOE_MIN_STEP(0x118, 0xf)
  MOE_MIN_STEP(0x142, 0xa)  // row_bcast:15 into rows 1 and 3
  MOE_MIN_STEP(0x143, 0xc)  // row_bcast:31 into rows 2 and 3
#undef MOE_MIN_STEP
  return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

constexpr int kDealt = 64;

// kVec: rows of dw are 16-byte aligned and hold whole 16-byte chunks.
template <typename T, bool kVec>
__global__ __launch_bounds__(256, 1) void ragged_wgrad_kernel(WgradRingParams p) {
  __shared__ __attribute__((aligned(1024))) char lds[kSlots][kSlotBytes];
  // 4 KiB a wavefront for its tile's store; while the deal is worked out,
  // the experts' rows
  __shared__ __attribute__((aligned(1024))) char staging[4][4096];
  int32_t* const n_rows = reinterpret_cast<int32_t*>(&staging[0][0]);
  __shared__ int32_t order[kRaggedMaxExperts];      // experts by falling rows
  __shared__ int32_t blocks_to[kRaggedMaxExperts];  // blocks up to that place of the order
  __shared__ int32_t dealt[kDealt];                 // this group's among the first blocks
  __shared__ int32_t n_dealt, n_blocks;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wa = wave & 1, wb = wave >> 1;  // this wavefront's 128 x 128 quarter

  const int ta = (p.N + kTile - 1) / kTile, tb = (p.K + kTile - 1) / kTile;
  const int per = ta * tb;
  for (int e = tid; e < p.E; e += 256) {
    int start, rows;
    expert_rows(p.offsets, e, p.rows, &start, &rows);
    n_rows[e] = rows;
  }
  __syncthreads();
  for (int e = tid; e < p.E; e += 256) {
    const int r = n_rows[e];
    int before = 0;
    for (int j = 0; j < p.E; ++j) before += n_rows[j] > r || (n_rows[j] == r && j < e);
    order[before] = e;
  }
  __syncthreads();

  // this workgroup's group and its place in it; an XCD's workgroups (b % 8)
  // are consecutive
  const int place = (int)(blockIdx.x % 8) * ((int)gridDim.x / 8) + (int)(blockIdx.x / 8);
  const int groups = (int)gridDim.x / p.group;
  const int my_group = place / p.group, member = place % p.group;
  const int per_blocks = (per + p.group - 1) / p.group;  // blocks of a chunk
  auto parts_of = [&](int rows) {
    const int n = (int)(((int64_t)rows + p.chunk - 1) / p.chunk);
    return n == 0 && !p.accumulate ? 1 : n;  // without rows: its zeros are stored
  };
  if (wave == 0) {
    int blocks = 0;
    for (int base = 0; base < p.E; base += kWave) {
      const int i = base + lane;
      const int jobs = i < p.E ? parts_of(n_rows[order[i]]) : 0;
      const int incl = wave_inclusive_scan(jobs * per_blocks) + blocks;
      if (i < p.E) blocks_to[i] = incl;
      blocks = __builtin_amdgcn_readlane(incl, kWave - 1);
      if ((uint32_t)blocks > kMaxUnits) break;
    }
    if ((uint32_t)blocks > kMaxUnits) blocks = 0;  // overlapping offsets: no jobs
    // the deal: lane g holds group g's work so far, in stages (a block's
    // store counts as eight)
    int mine = 0;
    if (groups < kDealt) {
      const int n = blocks < kDealt ? blocks : kDealt;
      uint32_t load = lane < groups ? 0u : 0x7fffffffu;
      int place_e = 0, part = 0, blk = 0;
      int rows = __builtin_amdgcn_readfirstlane(n_rows[order[0]]);
      int parts = parts_of(rows);
      for (int s = 0; s < n; ++s) {
        while (part == parts) {  // the next expert with blocks
          part = 0;
          ++place_e;
          rows = __builtin_amdgcn_readfirstlane(n_rows[order[place_e]]);
          parts = parts_of(rows);
        }
        const int left = rows - part * p.chunk;
        const uint32_t cost = (uint32_t)((left < p.chunk ? left : p.chunk) / kStageRows + 8);
        const uint32_t least = wave_min(load);
        const int g = __builtin_ctzll(__builtin_amdgcn_ballot_w64(load == least));
        if (lane == g) load += cost;
        if (g == my_group) {
          if (lane == 0) dealt[mine] = s;
          ++mine;
        }
        if (++blk == per_blocks) {
          blk = 0;
          ++part;
        }
      }
    }
    if (lane == 0) {
      n_dealt = mine;
      n_blocks = blocks;
    }
  }
  __syncthreads();
  const int total = __builtin_amdgcn_readfirstlane(n_blocks);
  const int mine = __builtin_amdgcn_readfirstlane(n_dealt);
  const int in_turn = groups < kDealt ? kDealt : 0;  // blocks from here on go in turn

  struct Tile {
    int e, part, a0, b0, cnt;  // cnt: rows of the chunk (-1: no tile)
    int64_t row;               // first row
  };
  // The k-th job of this workgroup: false past its last. A block may have no
  // tile for this member: cnt = -1.
  auto job = [&](int k, Tile* J) -> bool {
    int t;
    if (k < mine) {
      t = __builtin_amdgcn_readfirstlane(dealt[k]);
    } else {
      // every second turn backwards: the blocks fall in size
      const int turn = k - mine;
      t = in_turn + turn * groups + (turn & 1 ? groups - 1 - my_group : my_group);
      if (t >= total) return false;
    }
    int i = 0;
    for (int base = 0; base < p.E; base += kWave) {
      const bool before = base + lane < p.E && blocks_to[base + lane] <= t;
      i += __builtin_popcountll(__builtin_amdgcn_ballot_w64(before));
    }
    const int local = t - (i > 0 ? __builtin_amdgcn_readfirstlane(blocks_to[i - 1]) : 0);
    const int e = __builtin_amdgcn_readfirstlane(order[i]);
    int start, rows;
    expert_rows(p.offsets, e, p.rows, &start, &rows);
    start = __builtin_amdgcn_readfirstlane(start);
    rows = __builtin_amdgcn_readfirstlane(rows);
    const int tile = local % per_blocks * p.group + member;
    J->e = e;
    J->part = local / per_blocks;
    J->a0 = tile / tb * kTile;
    J->b0 = tile % tb * kTile;
    const int left = rows - J->part * p.chunk;
    J->cnt = tile < per ? (left < p.chunk ? left : p.chunk) : -1;
    J->row = (int64_t)start + (int64_t)J->part * p.chunk;
    return true;
  };

  // Loads of a stage: wavefronts 0-1 fetch dy, 2-3 x; each 128 columns, as
  // eight pieces of 1 KiB: four rows by 256 bytes, lane i row i / 16 of the
  // piece. Chunk c of row r sits at c ^ 4 (r % 4): the transposing reads
  // then cover all banks. Columns past the matrix read the next row's (or
  // zeros past the last): they feed sums that are never stored. Rows past
  // the chunk lie past the range and read as zeros. The range is checked by
  // whole dwords, so an odd width is rounded up to one.
  const int op = wave >> 1;
  const uint32_t ld = (uint32_t)(op == 0 ? p.ldy : p.ldx);  // bytes
  const char* src = op == 0 ? p.dy : p.x;
  const int width = op == 0 ? p.N : p.K;
  const uint32_t vo =
      (uint32_t)(lane >> 4) * ld + (uint32_t)((lane & 15) ^ (4 * (lane >> 4))) * 16;
  const uint32_t dst0 = (uint32_t)(uintptr_t)(lds_char*)&lds[0][0] +
                        (uint32_t)(op * kOpBytes + (wave & 1) * (kOpBytes / 2));
  struct FetchTile {
    __amdgpu_buffer_rsrc_t rs;
    int stages;
  };
  auto fetch_tile = [&](const Tile& J) {
    FetchTile F;
    const int col = (op == 0 ? J.a0 : J.b0) + 128 * (wave & 1);
    F.stages = J.cnt > 0 ? (J.cnt + kStageRows - 1) / kStageRows : 0;
    F.rs = __builtin_amdgcn_make_buffer_rsrc(
        (void*)(src + J.row * ld + (int64_t)col * 2), 0,
        J.cnt > 0 && col < width
            ? (int)((uint32_t)(J.cnt - 1) * ld + (((uint32_t)(width - col) * 2u + 3u) & ~3u))
            : 0,
        kRsrcWord3);
    return F;
  };
  // The fetch cursor: job fj, its stage fs; past the last job, stages that
  // load nothing, so that every stage issues the same loads.
  int fj = 0, fs = 0;
  Tile FT;
  bool more = job(0, &FT);
  if (!more) return;
  FetchTile F = fetch_tile(FT);
  auto next_stage = [&]() -> uint32_t {
    while (more && fs >= F.stages) {
      fs = 0;
      more = job(++fj, &FT);
      if (more) F = fetch_tile(FT);
    }
    const uint32_t off = more ? (uint32_t)(fs * kStageRows) * ld : kOutOfRange;
    ++fs;
    return off;
  };
  auto fetch = [&](uint32_t off, int slot, int x) {
    lds_load16(F.rs, vo, off + (uint32_t)(4 * x) * ld, dst0 + (uint32_t)(slot * kSlotBytes + x * 1024));
  };

  // Transposed read: in each group of 16 lanes, lane i receives 16-bit
  // element i % 4 of the 8 bytes addressed by lanes 4 j + i / 4, j = 0..3.
  // Lanes 4 j + q of group g address row 8 (g / 2) + j (+ 4) of the step's
  // 16 and columns 16 (g % 2) + 4 q of a 32-column block.
  const int grp = lane >> 4, gj = (lane >> 2) & 3, gq = lane & 3;
  const int tr = (2 * (grp >> 1)) * 1024 + gj * 256 + (gq & 1) * 8;
  const lds_char* ldsb = (const lds_char*)&lds[0][0];
  auto frag = [&](int o, int slot, int blk, int ks) -> u32x4 {
    const int chunk = (blk * 4 + 2 * (grp & 1) + (gq >> 1)) ^ (4 * gj);
    const lds_char* at = ldsb + slot * kSlotBytes + o * kOpBytes +
                         (o == 0 ? wa : wb) * (kOpBytes / 2) + ks * 4096 + tr + chunk * 16;
    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)at);
    const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(at + 1024));
    return __builtin_bit_cast(u32x4, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
  };

  f32x16 acc[4][4];  // [k block][n block]: lanes are rows n
  u32x4 fb0[4], fa0[4], fb1[4], fa1[4];
  // in the order the MFMAs first use them
  auto read_one = [&](u32x4 (&fb)[4], u32x4 (&fa)[4], int slot, int ks, int x) {
    if (x == 0)
      fb[0] = frag(1, slot, 0, ks);
    else if (x <= 4)
      fa[x - 1] = frag(0, slot, x - 1, ks);
    else
      fb[x - 4] = frag(1, slot, x - 4, ks);
  };
  constexpr int kOps = 12;  // 8 fragment reads, a load after every second
  auto mma_step = [&](const u32x4 (&fb)[4], const u32x4 (&fa)[4], auto op_) {
#pragma unroll
    for (int n = 0; n < 16; ++n) {
      const int i = n / 4, j = n % 4;
      acc[i][j] = mma<T>(fb[i], fa[j], acc[i][j]);
#pragma unroll
      for (int x = n * kOps / 16; x < (n + 1) * kOps / 16; ++x) op_(x);
      __builtin_amdgcn_sched_barrier(0);
    }
  };

  // dw is next read when the backward has ended: non-temporal, so that its
  // lines do not displace operands in L2 (balanced gate/up, both gradients:
  // 599 -> 584 us). Slots are read again by the next launch. (The
  // accumulators are read by asm: the nops are the wait states the compiler
  // cannot see.)
  auto epilogue = [&](const Tile& J) {
    asm volatile("s_nop 7\n\ts_nop 7\n\ts_nop 7\n\ts_nop 7" ::: "memory");
    const int mr = p.N - J.a0 < kTile ? p.N - J.a0 : kTile;
    const uint32_t ldo = (uint32_t)p.K * 4u;
    char* stg = &staging[wave][0];
    float* dw = p.dw + ((int64_t)J.e * p.N + J.a0) * p.K;
    if (J.part > 0) {
      const int slot = slots_before(p.offsets, J.e, p.rows, p.chunk) + J.part - 1;
      if ((uint32_t)slot >= (uint32_t)p.n_slots) return;  // overlapping offsets
      float* out = p.slots + ((int64_t)slot * p.N + J.a0) * p.K;
      store_tile<float, 4, 4, kVec, false, 0>(acc, stg, (char*)out, ldo, mr, p.K, J.b0, wb, wa,
                                              lane);
    } else if (p.accumulate) {
      store_tile<float, 4, 4, kVec, true, kNonTemporal>(acc, stg, (char*)dw, ldo, mr, p.K, J.b0,
                                                        wb, wa, lane);
    } else {
      store_tile<float, 4, 4, kVec, false, kNonTemporal>(acc, stg, (char*)dw, ldo, mr, p.K, J.b0,
                                                         wb, wa, lane);
    }
  };

  // prologue: three stages in flight, the first waited for
#pragma unroll
  for (int st = 0; st < 3; ++st) {
    const uint32_t off = next_stage();
#pragma unroll
    for (int x = 0; x < 8; ++x) fetch(off, st, x);
  }
  wait_vmem_barrier<2 * kLoads>();
#pragma unroll
  for (int x = 0; x < 8; ++x) read_one(fb0, fa0, 0, 0, x);

  // Stage g (slot g % 4): the first step's MFMAs run while the second's
  // fragments are read and half of stage g + 3 is fetched into the slot of
  // g - 1; the barrier waits for g + 1; the second step's MFMAs run while
  // g + 1's first fragments are read and the rest of g + 3 is fetched.
  int g = 0;
  Tile CT;
  for (int cj = 0; job(cj, &CT); ++cj) {
    if (CT.cnt < 0) continue;
    const int stages = (CT.cnt + kStageRows - 1) / kStageRows;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.f;
    for (int cs = 0; cs < stages; ++cs, ++g) {
      const int u = g & 3;
      const uint32_t off = next_stage();
      mma_step(fb0, fa0, [&](int x) {
        if (x % 3 < 2)
          read_one(fb1, fa1, u, 1, x - x / 3);
        else
          fetch(off, (u + 3) & 3, x / 3);
      });
      wait_vmem_barrier<kLoads + kLoads / 2>();
      mma_step(fb1, fa1, [&](int x) {
        if (x % 3 < 2)
          read_one(fb0, fa0, (u + 1) & 3, 0, x - x / 3);
        else
          fetch(off, (u + 3) & 3, 4 + x / 3);
      });
    }
    epilogue(CT);
  }
  // the loads that ran past the last stage read nothing but still write LDS
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
}

}  // namespace

hipError_t launch_wgrad_ring(bool is_bf16, const WgradRingParams& params, int num_cus,
                             hipStream_t st) {
  const int grid = num_cus < 8 ? 8 : num_cus / 8 * 8;
  WgradRingParams p = params;
  // the largest group that wastes at most an eighth of a chunk's blocks
  const int tiles = ((p.N + kTile - 1) / kTile) * ((p.K + kTile - 1) / kTile);
  for (p.group = 32; p.group > 1; p.group /= 2)
    if ((tiles + p.group - 1) / p.group * p.group * 8 <= tiles * 9 && grid / 8 % p.group == 0) break;
  const bool vec = p.K % 4 == 0 && (reinterpret_cast<uintptr_t>(p.dw) & 15) == 0;
  if (is_bf16 && vec)
    hipLaunchKernelGGL((ragged_wgrad_kernel<bf16, true>), dim3(grid), dim3(256), 0, st, p);
  else if (is_bf16)
    hipLaunchKernelGGL((ragged_wgrad_kernel<bf16, false>), dim3(grid), dim3(256), 0, st, p);
  else if (vec)
    hipLaunchKernelGGL((ragged_wgrad_kernel<f16, true>), dim3(grid), dim3(256), 0, st, p);
  else
    hipLaunchKernelGGL((ragged_wgrad_kernel<f16, false>), dim3(grid), dim3(256), 0, st, p);
  return hipGetLastError();
}

}  // namespace moe
