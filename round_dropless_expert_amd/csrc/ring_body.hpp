// The LDS-ring product kernels (gfx950 matrix cores): the loops that the ragged
// products and the orthogonalised updates share. A job says which tiles there
// are, where their operands lie and what becomes of their sums:
//
//   setup(wave, lane)       prepares the job, returns its number of tiles
//   locate(t)               tile t, uniform over the workgroup
//   operands(T, exists, ..) the buffers of a tile's operands; empty ones where
//                           the tile does not exist
//   store(T, acc, ..)       the tile's sums, with kStaging bytes of LDS a wavefront
//   p                       row strides lda, ldw, bytes of c in a row cbytes
#pragma once

#include "ragged_mma.hpp"

namespace moe {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef int i32x16 __attribute__((ext_vector_type(16)));

constexpr int kSlots = 4;
constexpr int kRowBytes = 64;  // bytes of c per row and stage

// Operand kinds.
struct OpBf16 {
  typedef f32x16 acc_t;
  static constexpr bool kScaled = false, kInt = false;
  template <int kStep>
  __device__ static __forceinline__ f32x16 mma(u32x4 a, u32x4 b, int, int, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  }
};
struct OpF16 {
  typedef f32x16 acc_t;
  static constexpr bool kScaled = false, kInt = false;
  template <int kStep>
  __device__ static __forceinline__ f32x16 mma(u32x4 a, u32x4 b, int, int, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a),
                                                  __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  }
};
// 4-bit values: lane l supplies row l % 32, values 32 (l / 32) .. + 31 of
// the step's 64 (one block) and the block's scale, byte 2 kStep of its
// scale register (the instruction's byte select).
struct OpMx {
  typedef f32x16 acc_t;
  static constexpr bool kScaled = true, kInt = false;
  template <int kStep>
  __device__ static __forceinline__ f32x16 mma(u32x4 a, u32x4 b, int sa, int sb, f32x16 c) {
    const i32x8 av = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
    const i32x8 bv = {(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(av, bv, c, 4, 4, 2 * kStep, sa,
                                                           2 * kStep, sb);
  }
};

// 8-bit integers, summed exactly; the tile store applies the scales.
struct OpI8 {
  typedef i32x16 acc_t;
  static constexpr bool kScaled = false, kInt = true;
  template <int kStep>
  __device__ static __forceinline__ i32x16 mma(u32x4 a, u32x4 b, int, int, i32x16 c) {
    return __builtin_amdgcn_mfma_i32_32x32x32_i8(__builtin_bit_cast(i32x4, a),
                                                 __builtin_bit_cast(i32x4, b), c, 0, 0, 0);
  }
};

template <int WI, int WJ>
struct Frags {
  u32x4 a[WI], b[WJ];
};
// Scales of a stage (MXFP4): byte 0 is the lane's block of step 0, byte 2 of
// step 1.
template <int WI, int WJ>
struct Scales {
  int a[WI], b[WJ];
};

// Operation x of a step that mixes kReads fragment reads evenly with n loads:
// the loads among the first x operations.
__host__ __device__ constexpr int loads_before(int x, int reads, int n) {
  return x * n / (reads + n);
}

// One MFMA step with kOps other operations spread over it in a fixed order
// (op(x) after MFMA i for x in [i kOps / M, (i + 1) kOps / M)), each group
// fenced so that the compiler keeps the order.
template <typename Op, int kStep, int WI, int WJ, int kOps, typename F>
__device__ __forceinline__ void mma_step(typename Op::acc_t (&acc)[WI][WJ], const Frags<WI, WJ>& f,
                                         const Scales<WI, WJ>& s, F op) {
  constexpr int M = WI * WJ;
#pragma unroll
  for (int i = 0; i < M; ++i) {
    acc[i / WJ][i % WJ] = Op::template mma<kStep>(f.a[i / WJ], f.b[i % WJ], s.a[i / WJ],
                                                  s.b[i % WJ], acc[i / WJ][i % WJ]);
#pragma unroll
    for (int x = i * kOps / M; x < (i + 1) * kOps / M; ++x) op(x);
    __builtin_amdgcn_sched_barrier(0);
  }
}

// Row tile and feature tile of an expert's local tile, of mt x nt. An XCD
// works on 32 consecutive tiles at a time; bands of up to eight row tiles,
// walked feature by feature, make them about 8 x 4 (12 operand panels in its
// L2) however many rows the expert has. (One expert of 16384 rows, 16384 x
// 16384: bands of all 64 row tiles make it 32 x 1 and 33 panels.)
__device__ __forceinline__ void place_tile(int local, int mt, int nt, int* m, int* n) {
  const int bands = (mt + 7) / 8;
  const int height = (mt + bands - 1) / bands;  // of a band; the last may be lower
  const int band = local / (height * nt), in = local - band * (height * nt);
  const int own = mt - band * height < height ? mt - band * height : height;
  *n = in / own;
  *m = band * height + in % own;
}

// Where a tile's operands live; uniform.
template <int kScaleLoads>
struct TileSrc {
  __amdgpu_buffer_rsrc_t rw, ra;
  __amdgpu_buffer_rsrc_t rs[kScaleLoads > 0 ? kScaleLoads : 1];
};

template <typename Op, int WI, int WJ, int SPB, bool kTransW, typename Job>
__device__ __forceinline__ void ring(Job& job) {
  const auto& p = job.p;
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
  static_assert(kSlotBytes >= 4 * Job::kStaging, "the epilogue stages in slot 3");

  __shared__ __attribute__((aligned(1024))) char slot0[kSlotBytes];
  __shared__ __attribute__((aligned(1024))) char slot1[kSlotBytes];
  __shared__ __attribute__((aligned(1024))) char slot2[kSlotBytes];
  __shared__ __attribute__((aligned(1024))) char slot3[kSlotBytes];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wn = wave & 1, wm = wave >> 1;
  const int half = lane >> 5, l32 = lane & 31;

  const int total = job.setup(wave, lane);

  // XCD-contiguous walk: workgroup b runs on XCD b % 8.
  const int G = gridDim.x;
  int tile = (int)(blockIdx.x % 8) * (G / 8) + (int)(blockIdx.x / 8);
  if (tile >= total) return;

  typedef typename Job::Tile Tile;
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
    job.template operands<kTransW>(T, exists, &S.rw, &S.ra);
    if constexpr (kScaled) {
#pragma unroll
      for (int j = 0; j < kScaleLoads; ++j) {
        // piece j 4 + wave: 64 positions of the weight rows, then of the tokens'
        const int piece = j * 4 + wave;
        S.rs[j] = job.scale_rows(T, piece < kWPasses, exists && piece < kPasses);
      }
    }
    return S;
  };

  const uint32_t lds_wave = (uint32_t)wave * 1024u;
  // Scale dwords: position l32 W + r of a wavefront's 32 W rows is row 32 r
  // + l32, so that one LDS read brings a lane the scales of its W blocks.
  uint32_t vo_s[kScaleLoads > 0 ? kScaleLoads : 1];
#pragma unroll
  for (int j = 0; j < kScaleLoads; ++j) {
    const int piece = j * 4 + wave;
    const bool w = piece < kWPasses;
    const int pos = (w ? piece : piece - kWPasses) * 64 + lane, W = w ? WI : WJ;
    const int in = pos % (32 * W);
    const int row = pos / (32 * W) * (32 * W) + in % W * 32 + in / W;
    vo_s[j] = (uint32_t)row * (uint32_t)p.lds;
  }
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
      lds_load4(S.rs[j], vo_s[j], o.t[sub] == kOutOfRange ? kOutOfRange : o.t[sub] / 16,
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
  // Scales of a stage. The lane's two blocks are bytes half and 2 + half of
  // its rows' dwords: shifted to bytes 0 and 2. A block past K holds no codes,
  // but its scale byte may be anything: in the stage that ends K it becomes 0
  // (`keep`).
  const int nb = tail / 16;  // blocks of the last stage
  const int keep_last = kScaled ? (half < nb ? 255 : 0) | (2 + half < nb ? 255 << 16 : 0) : 0;
  auto read_scales = [&](int (&raw)[WI + WJ], const char* stage) {
    const char* sc = stage + (BN + BM) * kRowBytes;
    typedef int wi_t __attribute__((ext_vector_type(WI)));
    typedef int wj_t __attribute__((ext_vector_type(WJ)));
    const wi_t a = *reinterpret_cast<const wi_t*>(sc + (wn * 32 + l32) * 4 * WI);
    const wj_t b = *reinterpret_cast<const wj_t*>(sc + BN * 4 + (wm * 32 + l32) * 4 * WJ);
#pragma unroll
    for (int i = 0; i < WI; ++i) raw[i] = a[i];
#pragma unroll
    for (int j = 0; j < WJ; ++j) raw[WI + j] = b[j];
  };
  auto set_scales = [&](Scales<WI, WJ>& sc, const int (&raw)[WI + WJ], int g) {
    const int keep = g == KT - 1 ? keep_last : 0x00ff00ff;
#pragma unroll
    for (int i = 0; i < WI; ++i) sc.a[i] = (int)((uint32_t)raw[i] >> (8 * half)) & keep;
#pragma unroll
    for (int j = 0; j < WJ; ++j) sc.b[j] = (int)((uint32_t)raw[WI + j] >> (8 * half)) & keep;
  };
  Frags<WI, WJ> f0, f1;
  Scales<WI, WJ> sc;
  int raw[WI + WJ];
  auto read_one = [&](Frags<WI, WJ>& f, const char* stage, int s, int r) {
    if (r < WI)
      f.a[r] = wfrag(stage, r, s);
    else
      f.b[r - WI] = tfrag(stage, r - WI, s);
  };
  // what a stage's first step needs
  auto read_first = [&](const char* stage) {
    if constexpr (kScaled) read_scales(raw, stage);
#pragma unroll
    for (int r = 0; r < kReads; ++r) read_one(f0, stage, 0, r);
    if constexpr (kScaled) set_scales(sc, raw, 0);
  };

  Tile T = job.locate(tile);
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
  read_first(slot0);

  typename Op::acc_t acc[WI][WJ];
  while (true) {
    const int tile_n = tile + G;
    const bool has_next = tile_n < total;
    Tile Tn = T;
    if (has_next) Tn = job.locate(tile_n);
    const src_t nxt = sources(Tn, has_next);

#pragma unroll
    for (int i = 0; i < WI; ++i)
#pragma unroll
      for (int j = 0; j < WJ; ++j)
#pragma unroll
        for (int v = 0; v < 16; ++v) acc[i][j][v] = 0;

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
      mma_step<Op, 0, WI, WJ, kReads + kLoadsPerStep>(acc, f0, sc, [&](int x) {         \
        const int lb = loads_before(x, kReads, kLoadsPerStep);                          \
        if (loads_before(x + 1, kReads, kLoadsPerStep) == lb) {                         \
          read_one(f1, cs, 1, x - lb);                                                  \
        } else {                                                                        \
          const int li = 2 * sub * kLoadsPerStep + lb;                                  \
          if (li < kLoads) fetch_one(FSLOT, SO, F, li);                                 \
        }                                                                               \
      });                                                                               \
      if (sub + 1 == SPB) wait_vmem_barrier<kWait>();                                   \
      if constexpr (kScaled) read_scales(raw, ns);                                      \
      mma_step<Op, 1, WI, WJ, kReads + kLoadsPerStep>(acc, f1, sc, [&](int x) {         \
        const int lb = loads_before(x, kReads, kLoadsPerStep);                          \
        if (loads_before(x + 1, kReads, kLoadsPerStep) == lb) {                         \
          read_one(f0, ns, 0, x - lb);                                                  \
        } else {                                                                        \
          const int li = (2 * sub + 1) * kLoadsPerStep + lb;                            \
          if (li < kLoads) fetch_one(FSLOT, SO, F, li);                                 \
        }                                                                               \
      });                                                                               \
      if constexpr (kScaled) set_scales(sc, raw, g + 1 == KS4 * SPB ? 0 : g + 1);       \
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

    // Epilogue, staged in slot 3 (consumed by the last step; next filled
    // after the barrier below). Non-temporal: the output is next read when
    // this launch has ended and should not displace operands in L2. (The
    // accumulators are read by asm: the nops are the wait states the compiler
    // cannot see.)
    asm volatile("s_nop 7\n\ts_nop 7\n\ts_nop 7\n\ts_nop 7" ::: "memory");
    job.store(T, acc, slot3 + wave * Job::kStaging, wn, wm, lane);
    // every wavefront's staging reads are done before the next tile's ring
    // writes slot 3
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    if (!has_next) break;
    // slot 0 holds the next tile's first stage
    read_first(slot0);
    tile = tile_n;
    T = Tn;
    cur = nxt;
  }
  // the loads that ran past the last tile read nothing but still write LDS
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
}

// The 256 x 256 tile on wide slots: 128 bytes of c per row, so that every
// load reads whole 128-byte lines (a 64-byte stage asks the L2 for each line
// twice, and the L2's request rate is what the tile is nearest to). A slot is
// 64 KiB, two fit; a slot's last fragments are read a step before its last
// MFMAs, so the loads of the slot after the next one start there: half in
// the slot's last step, half in the first step of the next, and have two
// steps (1024 MFMA cycles) and more to land.
template <typename Op, bool kTransW, typename Job>
__device__ __forceinline__ void wide_ring(Job& job) {
  const auto& p = job.p;
  constexpr bool kScaled = Op::kScaled;
  static_assert(!kScaled || !kTransW, "MXFP4: forward only");
  constexpr int WI = 4, WJ = 4, BN = 256;
  constexpr int kWide = 128;                 // bytes of c per row and slot
  constexpr int kOpBytes = 256 * kWide;      // one operand's share of a slot
  constexpr int kSlotBytes = 2 * kOpBytes;
  constexpr int kPasses = 16;                // 16-byte loads per slot and thread
  constexpr int kReads = WI + WJ;

  __shared__ __attribute__((aligned(1024))) char slots[2][kSlotBytes];
  __shared__ __attribute__((aligned(1024))) char staging[4][Job::kStaging];
  // scales of two slots: 16 bytes a row
  __shared__ __attribute__((aligned(1024))) char scales[kScaled ? 512 * 16 : 16];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wn = wave & 1, wm = wave >> 1;
  const int half = lane >> 5, l32 = lane & 31;

  const int total = job.setup(wave, lane);

  const int G = gridDim.x;
  int tile = (int)(blockIdx.x % 8) * (G / 8) + (int)(blockIdx.x / 8);
  if (tile >= total) return;

  typedef typename Job::Tile Tile;
  const uint32_t lda = (uint32_t)p.lda, ldw = (uint32_t)p.ldw;
  // c along the rows: a load moves 32 rows by 128 bytes, lane tid 16 bytes of
  // row tid / 8, to chunk tid % 8; logical chunk q of row r sits at q ^ (r /
  // 2) % 8, so that the 16 rows of a fragment read's cycle cover all banks.
  const int lr = tid >> 3, lc = (tid & 7) ^ ((lr >> 1) & 7);
  const uint32_t vo_t = (uint32_t)lr * lda + (uint32_t)lc * 16;
  // c down the columns: 32 rows c by 128 features are eight pieces of 1 KiB
  // (four rows by 256 bytes); a slot holds 64 rows c
  const uint32_t vo_w =
      kTransW ? (uint32_t)(lane >> 4) * ldw + (uint32_t)((lane & 15) ^ (4 * (lane >> 4))) * 16
              : (uint32_t)lr * ldw + (uint32_t)lc * 16;
  const int KP = (p.cbytes + kWide - 1) / kWide;  // slots of a tile that hold any c
  const int KP2 = (KP + 1) / 2 * 2;
  const bool dead = (KP - 1) * kWide + lc * 16 >= p.cbytes;
  const uint32_t vo_t_last = dead ? kOutOfRange : vo_t;
  const uint32_t vo_w_last = !kTransW && dead ? kOutOfRange : vo_w;
  const uint32_t wstep = kTransW ? 64u * ldw : (uint32_t)kWide;
  const uint32_t vo_s = (uint32_t)((wave & 1) * 128 + lane) * (uint32_t)p.lds;

  struct Src {
    __amdgpu_buffer_rsrc_t rw, ra, rs;
  };
  auto sources = [&](const Tile& T, bool exists) {
    Src S;
    job.template operands<kTransW>(T, exists, &S.rw, &S.ra);
    S.rs = S.ra;
    // wavefronts 0-1 fetch the weights' scales, 2-3 the tokens'
    if constexpr (kScaled) S.rs = job.scale_lines(T, wave < 2, exists);
    return S;
  };

  // Load x of slot position ks into slot c.
  struct Off {
    uint32_t w, t, s, vw, vt;
  };
  auto offsets_of = [&](int ks) {
    Off o;
    const bool in = ks < KP, last = ks == KP - 1;
    o.w = in ? (uint32_t)ks * wstep : kOutOfRange;
    o.t = in ? (uint32_t)ks * (uint32_t)kWide : kOutOfRange;
    o.s = in ? (uint32_t)ks * 8u : kOutOfRange;  // ks even: 16 bytes per two slots
    o.vw = last ? vo_w_last : vo_w;
    o.vt = last ? vo_t_last : vo_t;
    return o;
  };
  const uint32_t lds0 = (uint32_t)(uintptr_t)(lds_char*)&slots[0][0];
  const uint32_t lds_scales = (uint32_t)(uintptr_t)(lds_char*)&scales[0];
  const uint32_t lds_wave = (uint32_t)wave * 1024u;
  auto fetch = [&](int c, const Off& o, const Src& S, int x) {
    const uint32_t at = lds0 + (uint32_t)c * kSlotBytes;
    if (x < 8) {
      if constexpr (kTransW) {
        // sub-stage x / 4 (32 rows c), piece wave 4 + x % 4 of its 16
        const int piece = wave * 4 + (x & 3);
        lds_load16(S.rw, o.vw,
                   o.w + (uint32_t)((x >> 2) * 32 + 4 * (piece & 7)) * ldw +
                       (uint32_t)(piece >> 3) * 256u,
                   at + (uint32_t)((x >> 2) * 16384 + piece * 1024));
      } else {
        lds_load16(S.rw, o.vw, o.w + (uint32_t)(32 * x) * ldw, at + x * 4096 + lds_wave);
      }
    } else if (x < 16) {
      lds_load16(S.ra, o.vt, o.t + (uint32_t)(32 * (x - 8)) * lda, at + x * 4096 + lds_wave);
    } else if constexpr (kScaled) {
      // scale rows 128 (wave % 2) + 64 (x - 16) + lane of the operand
      lds_load16(S.rs, vo_s, o.s + (uint32_t)(64 * (x - 16)) * (uint32_t)p.lds,
                 lds_scales + (uint32_t)(wave * 2 + x - 16) * 1024u);
    }
  };

  const int grp = lane >> 4, gj = (lane >> 2) & 3, gq = lane & 3;
  const int tr_row = (2 * (grp >> 1)) * 1024 + gj * 256 + (gq & 1) * 8;
  const char* const slots0 = &slots[0][0];
  // fragment r (weight blocks, then token blocks) of step s of slot c
  Frags<WI, WJ> f0, f1;
  auto read_one = [&](Frags<WI, WJ>& f, int c, int s, int r) {
    const char* at = slots0 + c * kSlotBytes;
    if (kTransW && r < WI) {
      const int blk = wn * WI + r;
      const int chunk = ((blk & 3) * 4 + 2 * (grp & 1) + (gq >> 1)) ^ (4 * gj);
      const char* q = at + (s >> 1) * 16384 + (blk >> 2) * 8192 + (s & 1) * 4096 + tr_row +
                      chunk * 16;
      const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(lds_char*)q);
      const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(lds_char*)(q + 1024));
      f.a[r] = __builtin_bit_cast(u32x4, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    } else {
      const int row = r < WI ? wn * 128 + r * 32 + l32 : BN + wm * 128 + (r - WI) * 32 + l32;
      const u32x4 v = *reinterpret_cast<const u32x4*>(
          at + row * kWide + (((2 * s + half) ^ ((row >> 1) & 7)) << 4));
      if (r < WI)
        f.a[r] = v;
      else
        f.b[r - WI] = v;
    }
  };
  // Scales: raw holds two slots' (four stages of two steps) for the lane's
  // rows; stage q's bytes half and 2 + half, shifted to bytes 0 and 2, are
  // the lane's blocks. A block past K holds no codes, but its scale byte may
  // be anything: it becomes 0.
  const int KT = (p.cbytes + 63) / 64;
  const int nb = (p.cbytes - (KT - 1) * 64) / 16;
  const int keep_last = (half < nb ? 255 : 0) | (2 + half < nb ? 255 << 16 : 0);
  u32x4 raw[kScaled ? 8 : 1];
  Scales<WI, WJ> sc;
  auto read_scales = [&]() {
#pragma unroll
    for (int r = 0; r < kReads; ++r) {
      const int row = r < WI ? wn * 128 + r * 32 + l32 : BN + wm * 128 + (r - WI) * 32 + l32;
      raw[r] = *reinterpret_cast<const u32x4*>(scales + row * 16);
    }
  };
  auto set_scales = [&](int q, int g) {  // stage g (q = g % 4)
    const int keep = g < KT - 1 ? 0x00ff00ff : g == KT - 1 ? keep_last : 0;
#pragma unroll
    for (int i = 0; i < WI; ++i) sc.a[i] = (int)(raw[i][q] >> (8 * half)) & keep;
#pragma unroll
    for (int j = 0; j < WJ; ++j) sc.b[j] = (int)(raw[WI + j][q] >> (8 * half)) & keep;
  };

  // loads of a slot: 16, and 2 of scales into even ones; kFirst of them in
  // the step that frees the slot, the rest in the next
  constexpr int kFirst = 8;
  constexpr int kEven = kPasses + (kScaled ? 2 : 0);

  Tile T = job.locate(tile);
  Src cur = sources(T, true);
  {
    const Off o0 = offsets_of(0), o1 = offsets_of(1);
#pragma unroll
    for (int x = 0; x < kEven; ++x) fetch(0, o0, cur, x);
#pragma unroll
    for (int x = 0; x < kFirst; ++x) fetch(1, o1, cur, x);
  }
  wait_vmem_barrier<kFirst>();
  auto read_first = [&]() {
    if constexpr (kScaled) read_scales();
#pragma unroll
    for (int r = 0; r < kReads; ++r) read_one(f0, 0, 0, r);
    if constexpr (kScaled) set_scales(0, 0);
  };
  read_first();

  typename Op::acc_t acc[WI][WJ];
  while (true) {
    const int tile_n = tile + G;
    const bool has_next = tile_n < total;
    Tile Tn = T;
    if (has_next) Tn = job.locate(tile_n);
    const Src nxt = sources(Tn, has_next);

#pragma unroll
    for (int i = 0; i < WI; ++i)
#pragma unroll
      for (int j = 0; j < WJ; ++j)
#pragma unroll
        for (int v = 0; v < 16; ++v) acc[i][j][v] = 0;

    // Position ks in slot C. Step 0 issues the rest of position ks + 1's
    // loads (slot 1 - C); the barrier before step 3 waits for them; step 3
    // issues the first of ks + 2's into slot C.
#define MOE_WIDE(C, KS_, F0, K0, F3, K3)                                                \
  {                                                                                     \
    constexpr int kL0 = (C) == 1 ? kEven - kFirst : kPasses - kFirst;                   \
    {                                                                                   \
      const Off SO = offsets_of(K0);                                                    \
      mma_step<Op, 0, WI, WJ, kReads + kL0>(acc, f0, sc, [&](int x) {                   \
        const int lb = loads_before(x, kReads, kL0);                                    \
        if (loads_before(x + 1, kReads, kL0) == lb)                                     \
          read_one(f1, C, 1, x - lb);                                                   \
        else                                                                            \
          fetch(1 - (C), SO, F0, kFirst + lb);                                          \
      });                                                                               \
    }                                                                                   \
    mma_step<Op, 1, WI, WJ, kReads>(acc, f1, sc, [&](int x) { read_one(f0, C, 2, x); }); \
    if constexpr (kScaled) set_scales(2 * (C) + 1, 2 * (KS_) + 1);                      \
    mma_step<Op, 0, WI, WJ, kReads>(acc, f0, sc, [&](int x) { read_one(f1, C, 3, x); }); \
    wait_vmem_barrier<0>();                                                             \
    if constexpr (kScaled && (C) == 1) read_scales();                                   \
    {                                                                                   \
      const Off SO = offsets_of(K3);                                                    \
      mma_step<Op, 1, WI, WJ, kReads + kFirst>(acc, f1, sc, [&](int x) {                \
        const int lb = loads_before(x, kReads, kFirst);                                 \
        if (loads_before(x + 1, kReads, kFirst) == lb)                                  \
          read_one(f0, 1 - (C), 0, x - lb);                                             \
        else                                                                            \
          fetch(C, SO, F3, lb);                                                         \
      });                                                                               \
    }                                                                                   \
    if constexpr (kScaled)                                                              \
      set_scales((2 * (C) + 2) & 3, (KS_) + 1 == KP2 ? 0 : 2 * (KS_) + 2);              \
  }
    Src F = cur;
    int fofs = 0;
    for (int ks = 0; ks < KP2; ks += 2) {
      if (ks + 2 == KP2) {
        F = nxt;
        fofs = KP2;
      }
      // position ks + 1 is this tile's; from ks + 2 on the next tile's at
      // the end
      MOE_WIDE(0, ks, cur, ks + 1, F, ks + 2 - fofs)
      MOE_WIDE(1, ks + 1, F, ks + 2 - fofs, F, ks + 3 - fofs)
    }
#undef MOE_WIDE

    // Epilogue, as the narrow ring's, through a staging area of its own.
    asm volatile("s_nop 7\n\ts_nop 7\n\ts_nop 7\n\ts_nop 7" ::: "memory");
    job.store(T, acc, &staging[wave][0], wn, wm, lane);
    if (!has_next) break;
    read_first();
    tile = tile_n;
    T = Tn;
    cur = nxt;
  }
  // the loads that ran past the last tile read nothing but still write LDS
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
}

}  // namespace moe
