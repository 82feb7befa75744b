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
// c advances 64 bytes a row per stage: 32 values of 16 bits or 128 of 4, two
// MFMA steps either way (32x32x16 or 32x32x64, both 32 cycles). SPB stages
// form a slot of a four-slot ring filled by LDS-direct loads, up to three
// slots in flight, one barrier per slot; the ring runs on into the next
// tile, whose first slots land while this one is stored. Fragment reads run
// one step ahead of the MFMAs, loads are spread between them.
//
// Every output is one fixed sequence of MFMA steps over ascending c, so a
// row's result does not depend on the tile, the tile's shape or the rows
// around it.
#include "ragged_device.hpp"
#include "ragged_ring.hpp"

namespace moe {
namespace {

typedef __attribute__((address_space(3))) char lds_char;
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr int kRsrcWord3 = 0x00020000;  // raw buffer
constexpr int kNonTemporal = 2;
constexpr int kSlots = 4;
constexpr int kRowBytes = 64;  // bytes of c per row and stage
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

// Operand kinds.
struct OpBf16 {
  static constexpr bool kScaled = false;
  __device__ static __forceinline__ f32x16 mma(u32x4 a, u32x4 b, int, int, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  }
};
struct OpF16 {
  static constexpr bool kScaled = false;
  __device__ static __forceinline__ f32x16 mma(u32x4 a, u32x4 b, int, int, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a),
                                                  __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  }
};
// 4-bit values: lane l supplies row l % 32, values 32 (l / 32) .. + 31 of
// the step's 64 (one block) and the block's scale byte.
struct OpMx {
  static constexpr bool kScaled = true;
  __device__ static __forceinline__ f32x16 mma(u32x4 a, u32x4 b, int sa, int sb, f32x16 c) {
    const i32x8 av = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
    const i32x8 bv = {(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(av, bv, c, 4, 4, 0, sa, 0, sb);
  }
};

template <int WI, int WJ>
struct Frags {
  u32x4 a[WI], b[WJ];
  int sa[WI], sb[WJ];  // scale bytes (MXFP4)
};

// One MFMA step with kOps other operations spread over it in a fixed order
// (op(x) after MFMA i for x in [i kOps / M, (i + 1) kOps / M)), each group
// fenced so that the compiler keeps the order.
template <typename Op, int WI, int WJ, int kOps, typename F>
__device__ __forceinline__ void mma_step(f32x16 (&acc)[WI][WJ], const Frags<WI, WJ>& f, F op) {
  constexpr int M = WI * WJ;
#pragma unroll
  for (int i = 0; i < M; ++i) {
    acc[i / WJ][i % WJ] = Op::mma(f.a[i / WJ], f.b[i % WJ], f.sa[i / WJ], f.sb[i % WJ],
                                  acc[i / WJ][i % WJ]);
#pragma unroll
    for (int x = i * kOps / M; x < (i + 1) * kOps / M; ++x) op(x);
    __builtin_amdgcn_sched_barrier(0);
  }
}

// Where a tile's operands live; uniform.
template <int kScaleLoads>
struct TileSrc {
  __amdgpu_buffer_rsrc_t rw, ra;
  __amdgpu_buffer_rsrc_t rs[kScaleLoads > 0 ? kScaleLoads : 1];
};

template <typename Op, typename Out, int WI, int WJ, int SPB, bool kTransW>
__global__ __launch_bounds__(256, 1) void ring_kernel(RingParams p) {
  constexpr bool kScaled = Op::kScaled;
  static_assert(!kScaled || !kTransW, "MXFP4: forward only");
  constexpr int BN = 64 * WI, BM = 64 * WJ;
  constexpr int kWPasses = WI, kTPasses = WJ, kPasses = WI + WJ;
  // scale dwords of a stage: one per row, 64 rows a load, the four
  // wavefronts in turn (a load past the last piece reads nothing)
  constexpr int kScaleLoads = kScaled ? (kPasses + 3) / 4 : 0;
  constexpr int kScaleBytes = kScaleLoads * 4 * 256;
  constexpr int kStageBytes = (BN + BM) * kRowBytes + kScaleBytes;
  constexpr int kSlotBytes = SPB * kStageBytes;
  constexpr int kPer = kPasses + kScaleLoads;  // loads per stage and thread
  constexpr int kLoads = SPB * kPer;
  constexpr int kReads = WI + WJ;
  // A slot's loads are spread over its MFMA steps; a barrier waits for the
  // next slot's: behind those in issue order are the slot after it and the
  // part of the third issued before the barrier.
  constexpr int kSteps = 2, kStepsPerSlot = SPB * kSteps;
  constexpr int kLoadsPerStep = (kLoads + kStepsPerSlot - 1) / kStepsPerSlot;
  constexpr int kLoadsLast = kLoads - (kStepsPerSlot - 1) * kLoadsPerStep > 0
                                 ? kLoads - (kStepsPerSlot - 1) * kLoadsPerStep
                                 : 0;
  constexpr int kWait = kLoads + (kLoads - kLoadsLast);
  static_assert(kWait <= 63, "vmcnt range");
  static_assert(kSlotBytes >= 4 * 4096, "the epilogue stages 4 KiB a wavefront in slot 3");

  __shared__ __attribute__((aligned(1024))) char slot0[kSlotBytes];
  __shared__ __attribute__((aligned(1024))) char slot1[kSlotBytes];
  __shared__ __attribute__((aligned(1024))) char slot2[kSlotBytes];
  __shared__ __attribute__((aligned(1024))) char slot3[kSlotBytes];
  __shared__ int32_t tiles_to[kRaggedMaxExperts];  // tiles of the experts up to e
  __shared__ int32_t first_row[kRaggedMaxExperts];
  __shared__ int32_t n_rows[kRaggedMaxExperts];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wn = wave & 1, wm = wave >> 1;
  const int half = lane >> 5, l32 = lane & 31;

  // The tile table, by wavefront 0.
  const int nt = (p.B + BN - 1) / BN;
  if (wave == 0) {
    int carry = 0;
    for (int base = 0; base < p.E; base += kWave) {
      int start = 0, rows = 0;
      if (base + lane < p.E) expert_rows(p.offsets, base + lane, p.rows, &start, &rows);
      const int incl = wave_inclusive_scan((rows + BM - 1) / BM * nt) + carry;
      if (base + lane < p.E) {
        tiles_to[base + lane] = incl;
        first_row[base + lane] = start;
        n_rows[base + lane] = rows;
      }
      carry = __builtin_amdgcn_readlane(incl, kWave - 1);
    }
  }
  __syncthreads();
  const int total = __builtin_amdgcn_readfirstlane(tiles_to[p.E - 1]);

  // XCD-contiguous walk: workgroup b runs on XCD b % 8.
  const int G = gridDim.x;
  int tile = (int)(blockIdx.x % 8) * (G / 8) + (int)(blockIdx.x / 8);
  if (tile >= total) return;

  struct Tile {
    int e, start, m, n0, m0;
  };
  auto locate = [&](int t) {
    Tile T;
    int e = 0;
    for (int base = 0; base < p.E; base += kWave) {
      const bool before = base + lane < p.E && tiles_to[base + lane] <= t;
      e += __builtin_popcountll(__builtin_amdgcn_ballot_w64(before));
    }
    T.e = e;
    T.start = __builtin_amdgcn_readfirstlane(first_row[e]);
    T.m = __builtin_amdgcn_readfirstlane(n_rows[e]);
    const int mt = (T.m + BM - 1) / BM;
    const int local =
        t - (e > 0 ? __builtin_amdgcn_readfirstlane(tiles_to[e - 1]) : 0);
    T.n0 = local / mt * BN;
    T.m0 = local % mt * BM;
    return T;
  };

  const uint32_t lda = (uint32_t)p.lda, ldw = (uint32_t)p.ldw;  // bytes of a row
  // Load lanes. Operand with c along its rows: pass i holds rows 64 i .. +
  // 63, lane tid moves 16 bytes of row tid / 4, to chunk tid % 4 of its 64
  // bytes; logical chunk q sits at q ^ ((row / 4) % 4), so that the 16 rows a
  // fragment read touches in a cycle cover all banks.
  const int lr = tid >> 2, lc = (tid & 3) ^ ((lr >> 2) & 3);
  const uint32_t vo_t = (uint32_t)lr * lda + (uint32_t)lc * 16;
  // Weights with c down their columns: a stage is 32 rows c; 128 features of
  // it are eight pieces of 1 KiB, four rows by 256 bytes, so that a load
  // reads whole 128-byte lines. Chunk q of row r sits at q ^ 4 (r % 4): the
  // transposing read below then covers all banks.
  const uint32_t vo_w =
      kTransW ? (uint32_t)(lane >> 4) * ldw + (uint32_t)((lane & 15) ^ (4 * (lane >> 4))) * 16
              : (uint32_t)lr * ldw + (uint32_t)lc * 16;
  // the last stage may hold fewer than 64 bytes of c (always whole 16-byte
  // chunks): the lanes past them read nothing
  const int KT = (p.cbytes + kRowBytes - 1) / kRowBytes;
  const int tail = p.cbytes - (KT - 1) * kRowBytes;
  const bool dead = lc * 16 >= tail;
  const uint32_t vo_t_last = dead ? kOutOfRange : vo_t;
  const uint32_t vo_w_last = !kTransW && dead ? kOutOfRange : vo_w;
  const int KS = (KT + SPB - 1) / SPB;
  const int KS4 = (KS + kSlots - 1) / kSlots * kSlots;
  const uint32_t wstage = kTransW ? 32u * ldw : (uint32_t)kRowBytes;
  uint32_t wpass[kWPasses], tpass[kTPasses];
#pragma unroll
  for (int i = 0; i < kWPasses; ++i) {
    const int piece = wave * kWPasses + i;  // kTransW
    wpass[i] = kTransW ? (uint32_t)(4 * (piece & 7)) * ldw + (uint32_t)(piece >> 3) * 256u
                       : (uint32_t)(64 * i) * ldw;
  }
#pragma unroll
  for (int j = 0; j < kTPasses; ++j) tpass[j] = (uint32_t)(64 * j) * lda;

  typedef TileSrc<kScaleLoads> src_t;
  auto sources = [&](const Tile& T, bool exists) {
    src_t S;
    const int fw = p.B - T.n0 < BN ? p.B - T.n0 : BN;
    const int mr = T.m - T.m0 < BM ? T.m - T.m0 : BM;
    const char* wb = p.w + (int64_t)T.e * p.wbytes;
    if constexpr (kTransW)  // features past B read the next row's: never stored
      S.rw = __builtin_amdgcn_make_buffer_rsrc(
          (void*)(wb + (int64_t)T.n0 * 2), 0,
          exists ? (int)((uint32_t)(p.C - 1) * ldw + (uint32_t)(p.B - T.n0) * 2u) : 0, kRsrcWord3);
    else
      S.rw = __builtin_amdgcn_make_buffer_rsrc(
          (void*)(wb + (int64_t)T.n0 * p.ldw), 0,
          exists ? (int)((uint32_t)(fw - 1) * ldw + (uint32_t)p.cbytes) : 0, kRsrcWord3);
    const int64_t row = (int64_t)T.start + T.m0;
    S.ra = __builtin_amdgcn_make_buffer_rsrc(
        (void*)(p.act + row * p.lda), 0,
        exists ? (int)((uint32_t)(mr - 1) * lda + (uint32_t)p.cbytes) : 0, kRsrcWord3);
#pragma unroll
    for (int j = 0; j < kScaleLoads; ++j) {
      // piece j 4 + wave: 64 weight rows, then 64 token rows
      const int piece = j * 4 + wave;
      const bool w = piece < kWPasses;
      const int r0 = (w ? piece : piece - kWPasses) * 64;
      const int live = (w ? fw : mr) - r0;
      const char* base = w ? p.w_scales + ((int64_t)T.e * p.B + T.n0 + r0) * p.lds
                           : p.act_scales + (row + r0) * p.lds;
      S.rs[j] = __builtin_amdgcn_make_buffer_rsrc(
          (void*)base, 0,
          exists && piece < kPasses && live > 0 ? (int)((uint32_t)(live < 64 ? live : 64) *
                                                        (uint32_t)p.lds)
                                                : 0,
          kRsrcWord3);
    }
    return S;
  };

  const uint32_t lds_wave = (uint32_t)wave * 1024u;
  const uint32_t vo_s = (uint32_t)lane * (uint32_t)p.lds;
  struct StageOff {
    uint32_t w[SPB], t[SPB], vw[SPB], vt[SPB];
  };
  auto stage_off = [&](int ks) {
    StageOff o;
#pragma unroll
    for (int sub = 0; sub < SPB; ++sub) {
      const int g = ks * SPB + sub;
      const bool in = g < KT, last = g == KT - 1;
      o.w[sub] = in ? (uint32_t)g * wstage : kOutOfRange;
      o.t[sub] = in ? (uint32_t)g * (uint32_t)kRowBytes : kOutOfRange;
      o.vw[sub] = last ? vo_w_last : vo_w;
      o.vt[sub] = last ? vo_t_last : vo_t;
    }
    return o;
  };
  auto fetch_one = [&](char* slot, const StageOff& o, const src_t& S, int x) {
    const int sub = x / kPer, i = x % kPer;
    const uint32_t at = (uint32_t)(uintptr_t)(lds_char*)slot + sub * kStageBytes;
    if (i < kWPasses) {
      const uint32_t dst = kTransW ? at + (uint32_t)(wave * kWPasses + i) * 1024u
                                   : at + i * 4096 + lds_wave;
      lds_load16(S.rw, o.vw[sub], wpass[i] + o.w[sub], dst);
    } else if (i < kPasses) {
      lds_load16(S.ra, o.vt[sub], tpass[i - kWPasses] + o.t[sub], at + i * 4096 + lds_wave);
    } else if constexpr (kScaled) {
      const int j = i - kPasses;
      // a stage's four scale bytes of a row: 1/16 of its bytes of codes
      lds_load4(S.rs[j], vo_s, o.t[sub] == kOutOfRange ? kOutOfRange : o.t[sub] / 16,
                at + (BN + BM) * kRowBytes + (uint32_t)(j * 4 + wave) * 256u);
    }
  };

  // Fragments. Transposed weights come from gfx950's transposing LDS read:
  // in each group of 16 lanes, lane i receives 16-bit element i % 4 of the 8
  // bytes addressed by lanes 4 j + i / 4, j = 0..3. Lanes 4 j + q of group g
  // address row c = 8 (g / 2) + j (+ 4 for the second read) of the step and
  // features 16 (g % 2) + 4 q, so lane l receives feature l % 32 at eight
  // consecutive c: the MFMA operand of that feature.
  const int grp = lane >> 4, gj = (lane >> 2) & 3, gq = lane & 3;
  const int tr_row = (2 * (grp >> 1)) * 1024 + gj * 256 + (gq & 1) * 8;
  auto wfrag = [&](const char* stage, int ib, int s) -> u32x4 {
    if constexpr (kTransW) {
      const int blk = wn * WI + ib;  // 32-feature block of the tile
      const int chunk = ((blk & 3) * 4 + 2 * (grp & 1) + (gq >> 1)) ^ (4 * gj);
      const char* at = stage + (blk >> 2) * 8192 + s * 4096 + tr_row + chunk * 16;
      const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(lds_char*)at);
      const s16x4 hi =
          __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(lds_char*)(at + 1024));
      return __builtin_bit_cast(u32x4, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    } else {
      const int row = wn * (BN / 2) + ib * 32 + l32;
      return *reinterpret_cast<const u32x4*>(stage + row * kRowBytes +
                                             (((2 * s + half) ^ ((row >> 2) & 3)) << 4));
    }
  };
  auto tfrag = [&](const char* stage, int jb, int s) -> u32x4 {
    const int row = BN + wm * (BM / 2) + jb * 32 + l32;
    return *reinterpret_cast<const u32x4*>(stage + row * kRowBytes +
                                           (((2 * s + half) ^ ((row >> 2) & 3)) << 4));
  };
  // scale byte of a row's block 2 s + half. A block past K holds no codes,
  // but its scale byte may be anything: in the stage that ends K, 0 (keep:
  // this lane's mask of step s)
  auto sfrag = [&](const char* stage, int row, int s, int keep) -> int {
    return keep & *reinterpret_cast<const uint8_t*>(stage + (BN + BM) * kRowBytes + row * 4 +
                                                    2 * s + half);
  };
  Frags<WI, WJ> f0, f1;
  // `g`: the stage's number
  auto keep_of = [&](int g, int s) {
    return !kScaled || g != KT - 1 || (2 * s + half) * 16 < tail ? 255 : 0;
  };
  auto read_one = [&](Frags<WI, WJ>& f, const char* stage, int s, int keep, int r) {
    if (r < WI) {
      f.a[r] = wfrag(stage, r, s);
      if constexpr (kScaled) f.sa[r] = sfrag(stage, wn * (BN / 2) + r * 32 + l32, s, keep);
    } else {
      f.b[r - WI] = tfrag(stage, r - WI, s);
      if constexpr (kScaled)
        f.sb[r - WI] = sfrag(stage, BN + wm * (BM / 2) + (r - WI) * 32 + l32, s, keep);
    }
  };

  Tile T = locate(tile);
  src_t cur = sources(T, true);
  {
    const StageOff o0 = stage_off(0), o1 = stage_off(1), o2 = stage_off(2);
#pragma unroll
    for (int x = 0; x < kLoads; ++x) fetch_one(slot0, o0, cur, x);
#pragma unroll
    for (int x = 0; x < kLoads; ++x) fetch_one(slot1, o1, cur, x);
#pragma unroll
    for (int x = 0; x < kLoads; ++x) fetch_one(slot2, o2, cur, x);
  }
  wait_vmem_barrier<kWait>();
#pragma unroll
  for (int r = 0; r < kReads; ++r) read_one(f0, slot0, 0, keep_of(0, 0), r);

  f32x16 acc[WI][WJ];
  while (true) {
    const int tile_n = tile + G;
    const bool has_next = tile_n < total;
    Tile Tn = T;
    if (has_next) Tn = locate(tile_n);
    const src_t nxt = sources(Tn, has_next);

#pragma unroll
    for (int i = 0; i < WI; ++i)
#pragma unroll
      for (int j = 0; j < WJ; ++j)
#pragma unroll
        for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.f;

    // Slot position ks in CUR (NXT holds ks + 1); its steps also fetch ring
    // position ks + 3 into FSLOT: this tile's, or past its end KS4 the next
    // tile's. The barrier before the last step waits for ks + 1.
#define MOE_SLOT(CUR, NXT, FSLOT, KS_)                                                  \
  {                                                                                     \
    const StageOff SO = stage_off((KS_) + kSlots - 1 - fofs);                           \
    _Pragma("unroll") for (int sub = 0; sub < SPB; ++sub) {                             \
      const char* cs = CUR + sub * kStageBytes;                                         \
      const char* ns = sub + 1 < SPB ? CUR + (sub + 1) * kStageBytes : NXT;             \
      const int g = (KS_) * SPB + sub;                                                  \
      const int k1 = keep_of(g, 1);                                                     \
      mma_step<Op, WI, WJ, kReads + kLoadsPerStep>(acc, f0, [&](int x) {                \
        if (x < kReads) {                                                               \
          read_one(f1, cs, 1, k1, x);                                                   \
        } else {                                                                        \
          const int li = 2 * sub * kLoadsPerStep + x - kReads;                          \
          if (li < kLoads) fetch_one(FSLOT, SO, F, li);                                 \
        }                                                                               \
      });                                                                               \
      if (sub + 1 == SPB) wait_vmem_barrier<kWait>();                                   \
      const int k0 = keep_of(g + 1 == KS4 * SPB ? 0 : g + 1, 0);                        \
      mma_step<Op, WI, WJ, kReads + kLoadsPerStep>(acc, f1, [&](int x) {                \
        if (x < kReads) {                                                               \
          read_one(f0, ns, 0, k0, x);                                                   \
        } else {                                                                        \
          const int li = (2 * sub + 1) * kLoadsPerStep + x - kReads;                    \
          if (li < kLoads) fetch_one(FSLOT, SO, F, li);                                 \
        }                                                                               \
      });                                                                               \
    }                                                                                   \
  }
    src_t F = cur;
    int fofs = 0;
    for (int ks = 0; ks < KS4; ks += kSlots) {
      MOE_SLOT(slot0, slot1, slot3, ks)
      if (ks + kSlots == KS4) {
        F = nxt;
        fofs = KS4;
      }
      MOE_SLOT(slot1, slot2, slot0, ks + 1)
      MOE_SLOT(slot2, slot3, slot1, ks + 2)
      MOE_SLOT(slot3, slot0, slot2, ks + 3)
    }
#undef MOE_SLOT

    // Epilogue. Lane (l32, half) holds, for token l32 of a 32-token block,
    // features 8 q + 4 half + 0..3 of each 32-feature block. Each wavefront
    // turns 32 tokens x 128 bytes of features around in its 4 KiB of slot 3
    // (consumed by the last step; next filled after the barrier below) and
    // stores whole 128-byte row pieces. 16-byte chunk q of row r sits at q ^
    // (r % 8), against bank conflicts. Non-temporal: the output is next read
    // when this launch has ended and should not displace operands in L2.
    // (The accumulators are read by asm: give the last MFMAs the wait states
    // that the compiler cannot see.)
    asm volatile("s_nop 7\n\ts_nop 7\n\ts_nop 7\n\ts_nop 7" ::: "memory");
    {
      constexpr int kOs = sizeof(Out), kPerBlk = kOs == 2 ? 2 : 1;  // 32-feature blocks
      const int mr = T.m - T.m0 < BM ? T.m - T.m0 : BM;
      const uint32_t ldo = (uint32_t)p.ldo;
      const __amdgpu_buffer_rsrc_t ro = __builtin_amdgcn_make_buffer_rsrc(
          (void*)(p.out + ((int64_t)T.start + T.m0) * p.ldo), 0,
          (int)((uint32_t)(mr - 1) * ldo + (uint32_t)p.B * kOs), kRsrcWord3);
      char* stg = slot3 + wave * 4096;
      const int rrow = lane >> 3, rchunk = lane & 7;
#pragma unroll
      for (int jb = 0; jb < WJ; ++jb) {
        const int row0 = wm * (BM / 2) + jb * 32;
#pragma unroll
        for (int ip = 0; ip < WI / kPerBlk; ++ip) {
#pragma unroll
          for (int u = 0; u < kPerBlk; ++u) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              typedef Out vec4_t __attribute__((ext_vector_type(4)));
              vec4_t o;
#pragma unroll
              for (int v = 0; v < 4; ++v)
                o[v] = from_f32<Out>(acc_read(acc[kPerBlk * ip + u][jb][4 * q + v]));
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
          const int feat = T.n0 + wn * (BN / 2) + ip * 32 * kPerBlk + rchunk * (16 / kOs);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int r = i * 8 + rrow;
            const u32x4 v = *reinterpret_cast<const u32x4*>(
                stg + r * 128 + ((rchunk ^ (r & 7)) * 16));
            // rows past the expert's fall past the range
            const uint32_t at = (uint32_t)(row0 + r) * ldo + (uint32_t)feat * kOs;
            if (p.out_vec) {
              __builtin_amdgcn_raw_buffer_store_b128(v, ro, feat < p.B ? at : kOutOfRange, 0,
                                                     kNonTemporal);
            } else if (row0 + r < mr) {
              Out* o = reinterpret_cast<Out*>(p.out + ((int64_t)T.start + T.m0) * p.ldo + at);
              typedef Out vec_t __attribute__((ext_vector_type(16 / kOs)));
              const vec_t e = __builtin_bit_cast(vec_t, v);
#pragma unroll
              for (int k = 0; k < 16 / kOs; ++k)
                if (feat + k < p.B) o[k] = e[k];
            }
          }
        }
      }
    }
    // every wavefront's staging reads are done before the next tile's ring
    // writes slot 3
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    if (!has_next) break;
    // slot 0 holds the next tile's first stage
#pragma unroll
    for (int r = 0; r < kReads; ++r) read_one(f0, slot0, 0, keep_of(0, 0), r);
    tile = tile_n;
    T = Tn;
    cur = nxt;
  }
  // the loads that ran past the last tile read nothing but still write LDS
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
}

template <typename Op, typename Out, int WI, int WJ, int SPB, bool kTransW>
hipError_t launch(const RingParams& p, int grid, hipStream_t st) {
  hipLaunchKernelGGL((ring_kernel<Op, Out, WI, WJ, SPB, kTransW>), dim3((unsigned)grid), dim3(256),
                     0, st, p);
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
  if (big <= medium && big <= small) return launch<Op, Out, 4, 4, 1, kTransW>(p, grid, st);
  if (medium <= small) return launch<Op, Out, 4, 2, 1, kTransW>(p, grid, st);
  return launch<Op, Out, 2, 1, 2, kTransW>(p, grid, st);
}

}  // namespace

hipError_t launch_ring(RingKind kind, const RingParams& p, int num_cus, hipStream_t st) {
  switch (kind) {
    case RingKind::kForwardBF16: return choose<OpBf16, bf16, false>(p, num_cus, st);
    case RingKind::kForwardF16: return choose<OpF16, f16, false>(p, num_cus, st);
    case RingKind::kInputGradBF16: return choose<OpBf16, bf16, true>(p, num_cus, st);
    case RingKind::kInputGradF16: return choose<OpF16, f16, true>(p, num_cus, st);
    case RingKind::kMxBF16: return choose<OpMx, bf16, false>(p, num_cus, st);
    case RingKind::kMxF16: return choose<OpMx, f16, false>(p, num_cus, st);
    default: return choose<OpMx, float, false>(p, num_cus, st);
  }
}

}  // namespace moe
