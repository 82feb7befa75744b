// Products over rows sorted by expert where the experts have few rows each:
// a serving batch, or one token. The time is that of reading the weights
// once, so nothing is staged: every lane loads its share of the operands
// straight into the registers of the matrix instruction.
//
// A workgroup takes 16 FB features and 16 MT rows of one expert. Its four
// wavefronts take the batches of K steps in turn (16 rows x 64 bytes a step
// and operand: 16x16x32 for 16-bit types, 16x16x128 for MXFP4) and their sums
// are joined in LDS, in wavefront order: the order of the sum is fixed. A
// batch's loads are issued while the one before is multiplied.
//
// Splitting K over the wavefronts makes four times as many loads in flight as
// one wavefront a tile would, and row blocks are workgroups of their own: the
// weights come from the L2 after the first. One token through four of 32
// experts, N = K = 2048, bf16: 8.4 us for 33.6 MB (4.0 TB/s; 7.6 us, 4.4 TB/s
// back to back), of which about 3 us are the launch. One expert of 64 rows,
// N = K = 4096: 20 us bf16, 8 us MXFP4.
#include "ragged_device.hpp"
#include "ragged_ring.hpp"

namespace moe {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));

constexpr int kRsrcWord3 = 0x00020000;          // raw buffer
constexpr uint32_t kOutOfRange = 0x80000000u;   // loads return zeros
constexpr int kNonTemporal = 2;
constexpr int kBatch = 4;  // K steps: the 16 scale bytes a lane loads at once

struct SkinnyBf16 {
  static constexpr bool kScaled = false;
  __device__ static __forceinline__ f32x4 mma(u32x4 a, u32x4 b, int, int, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  }
};
struct SkinnyF16 {
  static constexpr bool kScaled = false;
  __device__ static __forceinline__ f32x4 mma(u32x4 a, u32x4 b, int, int, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a),
                                                  __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  }
};
// 4-bit values: lane l supplies row l % 16, block l / 16 of the step's four,
// and the block's scale byte.
struct SkinnyMx {
  static constexpr bool kScaled = true;
  __device__ static __forceinline__ f32x4 mma(u32x4 a, u32x4 b, int sa, int sb, f32x4 c) {
    const i32x8 av = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
    const i32x8 bv = {(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(av, bv, c, 4, 4, 0, sa, 0, sb);
  }
};

// What a lane holds of a batch: 16 bytes a step of FB feature blocks and MT
// token blocks, and for MXFP4 the 16 scale bytes of each block's row.
template <typename Op, int FB, int MT>
struct Batch {
  u32x4 w[FB][kBatch], t[MT][kBatch];
  u32x4 sw[Op::kScaled ? FB : 1], st[Op::kScaled ? MT : 1];
};

template <typename Op, typename Out, int FB, int MT>
__device__ __forceinline__ void skinny_rows(const RingParams& p, const ExpertUnit& u, int n0,
                                            int m0, float* joined) {
  constexpr bool kScaled = Op::kScaled;
  constexpr int kFeatures = 16 * FB, kPitch = kFeatures + 4;  // floats
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l16 = lane & 15, blk = lane >> 4;
  const uint32_t lda = (uint32_t)p.lda, ldw = (uint32_t)p.ldw, lds = (uint32_t)p.lds;
  const int fw = p.B - n0 < kFeatures ? p.B - n0 : kFeatures;
  const int mr = u.rows - m0 < 16 * MT ? u.rows - m0 : 16 * MT;
  const int64_t w_row = (int64_t)u.e * p.B + n0, t_row = (int64_t)u.start + m0;
  // rows past the features or the expert's rows lie past the ranges
  const __amdgpu_buffer_rsrc_t rw = __builtin_amdgcn_make_buffer_rsrc(
      (void*)(p.w + (int64_t)u.e * p.wbytes + (int64_t)n0 * p.ldw), 0,
      (int)((uint32_t)(fw - 1) * ldw + (uint32_t)p.cbytes), kRsrcWord3);
  const __amdgpu_buffer_rsrc_t rt = __builtin_amdgcn_make_buffer_rsrc(
      (void*)(p.act + t_row * p.lda), 0, (int)((uint32_t)(mr - 1) * lda + (uint32_t)p.cbytes),
      kRsrcWord3);
  __amdgpu_buffer_rsrc_t rsw = rw, rst = rt;
  if constexpr (kScaled) {
    // a row's last 16 scale bytes may reach past it, into the next row or
    // past the array, which the range ends (dword by dword)
    const int64_t wl = ((int64_t)p.E * p.B - w_row) * lds, wm = (int64_t)fw * lds + 12;
    const int64_t tl = (p.rows - t_row) * (int64_t)lds, tm = (int64_t)mr * lds + 12;
    rsw = __builtin_amdgcn_make_buffer_rsrc((void*)(p.w_scales + w_row * lds), 0,
                                            (int)(wl < wm ? wl : wm), kRsrcWord3);
    rst = __builtin_amdgcn_make_buffer_rsrc((void*)(p.act_scales + t_row * lds), 0,
                                            (int)(tl < tm ? tl : tm), kRsrcWord3);
  }
  const int KT = (p.cbytes + 63) / 64;
  const bool dead = (KT - 1) * 64 + blk * 16 >= p.cbytes;  // of the last step
  const uint32_t vw = (uint32_t)l16 * ldw + (uint32_t)blk * 16;
  const uint32_t vt = (uint32_t)l16 * lda + (uint32_t)blk * 16;

  auto load = [&](Batch<Op, FB, MT>& b, int s0) {
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int s = s0 + k;
      const bool none = s >= KT || (s == KT - 1 && dead);
      const uint32_t at = (uint32_t)s * 64u;
#pragma unroll
      for (int i = 0; i < FB; ++i)
        b.w[i][k] = __builtin_bit_cast(
            u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                       rw, (int)(none ? kOutOfRange : vw + (uint32_t)(16 * i) * ldw + at), 0,
                       kNonTemporal));
#pragma unroll
      for (int j = 0; j < MT; ++j)
        b.t[j][k] = __builtin_bit_cast(
            u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                       rt, (int)(none ? kOutOfRange : vt + (uint32_t)(16 * j) * lda + at), 0, 0));
    }
    if constexpr (kScaled) {
      const bool none = s0 >= KT;
#pragma unroll
      for (int i = 0; i < FB; ++i)
        b.sw[i] = __builtin_bit_cast(
            u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                       rsw,
                       (int)(none ? kOutOfRange
                                  : (uint32_t)(16 * i + l16) * lds + (uint32_t)s0 * 4u),
                       0, 0));
#pragma unroll
      for (int j = 0; j < MT; ++j)
        b.st[j] = __builtin_bit_cast(
            u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                       rst,
                       (int)(none ? kOutOfRange
                                  : (uint32_t)(16 * j + l16) * lds + (uint32_t)s0 * 4u),
                       0, 0));
    }
  };
  f32x4 acc[FB][MT];
#pragma unroll
  for (int i = 0; i < FB; ++i)
#pragma unroll
    for (int j = 0; j < MT; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  auto multiply = [&](const Batch<Op, FB, MT>& b, int s0) {
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      int sw[FB] = {}, st[MT] = {};
      if constexpr (kScaled) {
        // a block past K holds no codes, but its scale byte may be anything
        const int s = s0 + k;
        const uint32_t keep = s >= KT || (s == KT - 1 && dead) ? 0u : 255u;
#pragma unroll
        for (int i = 0; i < FB; ++i) sw[i] = (int)((b.sw[i][k] >> (8 * blk)) & keep);
#pragma unroll
        for (int j = 0; j < MT; ++j) st[j] = (int)((b.st[j][k] >> (8 * blk)) & keep);
      }
#pragma unroll
      for (int i = 0; i < FB; ++i)
#pragma unroll
        for (int j = 0; j < MT; ++j)
          acc[i][j] = Op::mma(b.w[i][k], b.t[j][k], sw[i], st[j], acc[i][j]);
    }
  };

  const int step = 4 * kBatch;
  Batch<Op, FB, MT> b0, b1;
  int s = wave * kBatch;
  load(b0, s);
  for (; s < KT; s += 2 * step) {
    load(b1, s + step);
    multiply(b0, s);
    load(b0, s + 2 * step);
    multiply(b1, s + step);
  }

  // Lane: token l % 16 of a block, features 4 (l / 16) + 0..3 of a block.
  // joined[wave][token][feature], a token's features padded by four floats
#pragma unroll
  for (int j = 0; j < MT; ++j)
#pragma unroll
    for (int i = 0; i < FB; ++i)
      *reinterpret_cast<f32x4*>(joined + ((wave * MT + j) * 16 + l16) * kPitch +
                                16 * i + 4 * blk) =
          acc[i][j];
  __syncthreads();
  Out* y = reinterpret_cast<Out*>(p.out + t_row * p.ldo) + n0;
  const int64_t ldo = p.ldo / (int64_t)sizeof(Out);
#pragma unroll
  for (int k = 0; k < FB * MT; ++k) {
    const int token = tid / kFeatures + 256 / kFeatures * k, f = tid % kFeatures;
    if (token < mr && f < fw) {
      float r = 0.f;
#pragma unroll
      for (int w = 0; w < 4; ++w) r += joined[(w * MT * 16 + token) * kPitch + f];
      y[token * ldo + f] = from_f32<Out>(r);
    }
  }
}

template <typename Op, typename Out, int FB, int MT>
__global__ __launch_bounds__(256) void skinny_kernel(RingParams p) {
  __shared__ __attribute__((aligned(16))) float joined[4 * MT * 16 * (16 * FB + 4)];
  const int nb = (p.B + 16 * FB - 1) / (16 * FB);
  ExpertUnit u;
  const int t = blockIdx.x;
  if (!find_unit(p.offsets, p.E, p.rows, t,
                 [&](int rows) { return (rows + 16 * MT - 1) / (16 * MT) * nb; }, &u))
    return;
  const int local = t - u.first;
  skinny_rows<Op, Out, FB, MT>(p, u, local % nb * 16 * FB, local / nb * 16 * MT, joined);
}

// 32 features a workgroup, or 16 where that leaves CUs without one.
template <typename Op, typename Out, int MT>
hipError_t launch_rows(const RingParams& p, int num_cus, hipStream_t st) {
  const int64_t active = p.rows < p.E ? p.rows : p.E;
  const int64_t parts = p.rows / (16 * MT) + active;  // row blocks at most
  // and with experts of the mean number of rows
  const int64_t mean = (p.rows + active - 1) / active;
  const int64_t likely = active * ((mean + 16 * MT - 1) / (16 * MT));
  const int64_t wide = parts * ((p.B + 31) / 32);
  if (likely * ((p.B + 31) / 32) >= num_cus)
    hipLaunchKernelGGL((skinny_kernel<Op, Out, 2, MT>), dim3((unsigned)wide), dim3(256), 0, st, p);
  else
    hipLaunchKernelGGL((skinny_kernel<Op, Out, 1, MT>),
                       dim3((unsigned)(parts * ((p.B + 15) / 16))), dim3(256), 0, st, p);
  return hipGetLastError();
}

// Rows a workgroup, by the experts' mean (whose number is uneven: 64 rows of
// four experts take 11.8 us with 32, 14.4 with 16).
template <typename Op, typename Out>
hipError_t launch(const RingParams& p, int num_cus, hipStream_t st) {
  const int64_t active = p.rows < p.E ? p.rows : p.E;
  return p.rows <= 8 * active ? launch_rows<Op, Out, 1>(p, num_cus, st)
                              : launch_rows<Op, Out, 2>(p, num_cus, st);
}

}  // namespace

hipError_t launch_skinny(RingKind kind, const RingParams& p, int num_cus, hipStream_t st) {
  switch (kind) {
    case RingKind::kForwardBF16: return launch<SkinnyBf16, bf16>(p, num_cus, st);
    case RingKind::kForwardF16: return launch<SkinnyF16, f16>(p, num_cus, st);
    case RingKind::kMxBF16: return launch<SkinnyMx, bf16>(p, num_cus, st);
    case RingKind::kMxF16: return launch<SkinnyMx, f16>(p, num_cus, st);
    case RingKind::kMxF32: return launch<SkinnyMx, float>(p, num_cus, st);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace moe
