// Microscaled 4-bit floating point: quantisation, its inverse, and the
// product over rows sorted by expert with both operands in that format.
//
// A row of K values is K / 32 blocks. A block's scale is the power of two
// 2^e, e = floor(log2 max|x|) - 2, stored as the byte e + 127 (e at least
// -127; 255 means that the block has no values: it held an infinity or a
// NaN). Its values are x / 2^e rounded to nearest, ties to even, among 0,
// 0.5, 1, 1.5, 2, 3, 4 and 6 (a sign bit, two bits of exponent, one of
// mantissa), ending at 6; the block's largest magnitude lies in [4, 8).
#include "ragged_device.hpp"
#include "ragged_ring.hpp"

namespace moe {
namespace {

// Code (0 .. 7) of a magnitude in [0, 8): the number of borders it has
// passed. A border between an odd and an even code belongs to the even one.
__device__ __forceinline__ uint32_t code_of(float a) {
  return (uint32_t)(a > 0.25f) + (a >= 0.75f) + (a > 1.25f) + (a >= 1.75f) + (a > 2.5f) +
         (a >= 3.5f) + (a > 5.0f);
}

struct QuantParams {
  const void* x;
  int64_t ld_x, src_rows;
  const int32_t* index;
  int index_div;
  const int32_t* n_rows;
  int64_t rows, K;
  uint8_t* codes;
  uint8_t* scales;
  int64_t stride;  // bytes of a scale row
};

// A lane takes V = 16 bytes of a row (kVec: the row's addresses are
// 16-byte aligned), 32 / V lanes a block: its maximum is exchanged between
// them, and each stores V / 2 bytes of codes.
template <typename T, bool kVec>
__global__ __launch_bounds__(256) void mx_quantize_kernel(QuantParams p) {
  constexpr int V = 16 / sizeof(T);
  constexpr int kLanes = kMxBlock / V;
  const uint32_t per = (uint32_t)(p.K / V);
  const int64_t rows = live_rows(p.rows, p.n_rows);
  const int64_t total = rows * per;  // a multiple of kLanes
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total;
       i += (int64_t)gridDim.x * 256) {
    const int64_t row = i / per;
    const int c = (int)(i - row * per) * V;
    int64_t src = row;
    bool real = true;
    if (p.index) {
      const int32_t a = p.index[row];
      src = a < 0 ? -1 : a / p.index_div;
      real = src >= 0 && src < p.src_rows;
    }
    union {
      T e[V];
      u32x4 v;
    } x;
    x.v = u32x4{0, 0, 0, 0};
    if (real) {
      const T* at = static_cast<const T*>(p.x) + src * p.ld_x + c;
      if constexpr (kVec) {
        x.v = *reinterpret_cast<const u32x4*>(at);
      } else {
#pragma unroll
        for (int v = 0; v < V; ++v) x.e[v] = at[v];
      }
    }
    // largest magnitude, as the bits of an fp32 (their order is that of the
    // values, with infinity and then NaN above every number)
    uint32_t top = 0;
    float f[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      f[v] = to_f32(x.e[v]);
      const uint32_t b = __builtin_bit_cast(uint32_t, f[v]) & 0x7fffffffu;
      top = top > b ? top : b;
    }
#pragma unroll
    for (int m = 1; m < kLanes; m <<= 1) {
      const uint32_t o = (uint32_t)__shfl_xor((int)top, m, kWave);
      top = top > o ? top : o;
    }
    const bool bad = top >= 0x7f800000u;
    // e + 127 = exponent field - 2; below 2^-124 the scale stays at 2^-127
    const int byte = bad ? 255 : ((int)(top >> 23) > 2 ? (int)(top >> 23) - 2 : 0);
    uint32_t packed = 0;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const uint32_t sign = __builtin_bit_cast(uint32_t, f[v]) >> 31;
      const uint32_t q =
          bad ? 0 : (sign << 3) | code_of(ldexpf(__builtin_fabsf(f[v]), 127 - byte));
      packed |= q << (4 * v);
    }
    uint8_t* out = p.codes + row * (p.K / 2) + c / 2;
    if constexpr (V == 8)
      *reinterpret_cast<uint32_t*>(out) = packed;
    else
      *reinterpret_cast<uint16_t*>(out) = (uint16_t)packed;
    if (c % kMxBlock == 0) {
      uint8_t* s = p.scales + row * p.stride + c / kMxBlock;
      *s = (uint8_t)byte;
      // the padding of the scale row: blocks that hold nothing
      if (c + kMxBlock == p.K)
        for (int64_t k = p.K / kMxBlock; k < p.stride; ++k) *++s = 0;
    }
  }
}

struct DequantParams {
  const uint8_t* codes;
  const uint8_t* scales;
  void* y;
  int64_t ld_y, rows, K, stride;
  const int32_t* n_rows;
};

template <typename T, bool kVec>
__global__ __launch_bounds__(256) void mx_dequantize_kernel(DequantParams p) {
  constexpr int V = 16 / sizeof(T);
  const uint32_t per = (uint32_t)(p.K / V);
  const int64_t total = live_rows(p.rows, p.n_rows) * per;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total;
       i += (int64_t)gridDim.x * 256) {
    const int64_t row = i / per;
    const int c = (int)(i - row * per) * V;
    const uint8_t* at = p.codes + row * (p.K / 2) + c / 2;
    const uint32_t q = V == 8 ? *reinterpret_cast<const uint32_t*>(at)
                              : *reinterpret_cast<const uint16_t*>(at);
    const int s = p.scales[row * p.stride + c / kMxBlock];
    union {
      T e[V];
      u32x4 v;
    } y;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const uint32_t m = (q >> (4 * v)) & 7;
      // magnitude: 0 and 0.5, then (1 + mantissa / 2) 2^(exponent - 1)
      const float a = m < 2 ? 0.5f * (float)m
                            : ldexpf(1.0f + 0.5f * (float)(m & 1), (int)(m >> 1) - 1);
      float r = ldexpf((q >> (4 * v)) & 8 ? -a : a, s - 127);
      if (s == 255) r = __builtin_nanf("");
      y.e[v] = from_f32<T>(r);
    }
    T* out = static_cast<T*>(p.y) + row * p.ld_y + c;
    if constexpr (kVec) {
      *reinterpret_cast<u32x4*>(out) = y.v;
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) out[v] = y.e[v];
    }
  }
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

unsigned grid_of(int64_t lanes, int num_cus) {
  const int64_t blocks = (lanes + 255) / 256, most = (int64_t)num_cus * 16;
  return (unsigned)(blocks < most ? blocks : most);
}

template <typename T>
hipError_t quantize(const QuantParams& p, int num_cus, hipStream_t st) {
  constexpr int V = 16 / sizeof(T);
  const unsigned grid = grid_of(p.rows * (p.K / V), num_cus);
  if (p.ld_x % V == 0 && aligned16(p.x))
    hipLaunchKernelGGL((mx_quantize_kernel<T, true>), dim3(grid), dim3(256), 0, st, p);
  else
    hipLaunchKernelGGL((mx_quantize_kernel<T, false>), dim3(grid), dim3(256), 0, st, p);
  return hipGetLastError();
}

template <typename T>
hipError_t dequantize(const DequantParams& p, int num_cus, hipStream_t st) {
  constexpr int V = 16 / sizeof(T);
  const unsigned grid = grid_of(p.rows * (p.K / V), num_cus);
  if (p.ld_y % V == 0 && aligned16(p.y))
    hipLaunchKernelGGL((mx_dequantize_kernel<T, true>), dim3(grid), dim3(256), 0, st, p);
  else
    hipLaunchKernelGGL((mx_dequantize_kernel<T, false>), dim3(grid), dim3(256), 0, st, p);
  return hipGetLastError();
}

typedef int i32x8 __attribute__((ext_vector_type(8)));

struct MxParams {
  const uint8_t* xq;
  const uint8_t* xs;
  const uint8_t* wq;
  const uint8_t* ws;
  void* y;
  const int32_t* offsets;
  int64_t ld_y;
  int rows, E, N, K;
  int stride;  // bytes of a scale row
  int tiles_n;
};

// v_mfma_scale_f32_16x16x128_f8f6f4 on 4-bit operands: lane l supplies row
// l % 16 and block l / 16 (32 values, 16 bytes) of 128 values of c, and its
// block's scale byte.
__device__ __forceinline__ f32x4 mx_mma16(u32x4 a, int sa, u32x4 b, int sb, f32x4 c) {
  const i32x8 av = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
  const i32x8 bv = {(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(av, bv, c, 4, 4, 0, sa, 0, sb);
}

// One wavefront per 16 rows x 16 features.
template <typename T>
__global__ __launch_bounds__(64) void mx_gemm_kernel(MxParams p) {
  ExpertUnit u;
  const int t = blockIdx.x;
  if (!find_unit(p.offsets, p.E, p.rows, t,
                 [&](int rows) { return (rows + 15) / 16 * p.tiles_n; }, &u))
    return;
  const int local = t - u.first;
  const int m0 = local / p.tiles_n * 16, n0 = local % p.tiles_n * 16;
  const int lane = threadIdx.x, l16 = lane & 15, blk = lane >> 4;
  const int row = m0 + l16, feat = n0 + l16;
  const bool xin = row < u.rows, win = feat < p.N;
  const int64_t xr = (int64_t)u.start + (xin ? row : 0);
  const int64_t wr = (int64_t)u.e * p.N + (win ? feat : 0);
  const int64_t kb = p.K / 2;
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  const u32x4 none = {0, 0, 0, 0};
  for (int k = blk * kMxBlock; k < (p.K + 127) / 128 * 128; k += 128) {
    const bool in = k < p.K;
    const u32x4 x = xin && in ? *reinterpret_cast<const u32x4*>(p.xq + xr * kb + k / 2) : none;
    const u32x4 w = win && in ? *reinterpret_cast<const u32x4*>(p.wq + wr * kb + k / 2) : none;
    const int sx = xin && in ? p.xs[xr * p.stride + k / kMxBlock] : 127;
    const int sw = win && in ? p.ws[wr * p.stride + k / kMxBlock] : 127;
    acc = mx_mma16(x, sx, w, sw, acc);
  }
  // lane: feature l % 16, rows 4 (l / 16) + v
  if (!win) return;
#pragma unroll
  for (int v = 0; v < 4; ++v) {
    const int r = m0 + 4 * blk + v;
    if (r < u.rows)
      static_cast<T*>(p.y)[((int64_t)u.start + r) * p.ld_y + feat] = from_f32<T>(acc[v]);
  }
}

template <typename T>
hipError_t mx_gemm(MxParams p, int num_cus, hipStream_t st) {
  (void)num_cus;
  p.tiles_n = (p.N + 15) / 16;
  const int64_t jobs =
      ((int64_t)p.rows / 16 + (p.rows < p.E ? p.rows : p.E)) * p.tiles_n;
  hipLaunchKernelGGL((mx_gemm_kernel<T>), dim3((unsigned)jobs), dim3(64), 0, st, p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_mx_quantize(ElemType t, int64_t rows, int64_t K, const void* x, int64_t ld_x,
                              int64_t src_rows, const int32_t* index, int index_div,
                              const int32_t* n_rows, uint8_t* codes, uint8_t* scales,
                              int num_cus, hipStream_t st) {
  if (rows == 0) return hipSuccess;
  const QuantParams p{x,    ld_x, src_rows, index,  index_div,         n_rows,
                      rows, K,    codes,    scales, mx_scale_stride(K)};
  switch (t) {
    case ElemType::kF32: return quantize<float>(p, num_cus, st);
    case ElemType::kBF16: return quantize<bf16>(p, num_cus, st);
    default: return quantize<f16>(p, num_cus, st);
  }
}

hipError_t launch_mx_dequantize(ElemType t, int64_t rows, int64_t K, const uint8_t* codes,
                                const uint8_t* scales, void* y, int64_t ld_y,
                                const int32_t* n_rows, int num_cus, hipStream_t st) {
  if (rows == 0) return hipSuccess;
  const DequantParams p{codes, scales, y, ld_y, rows, K, mx_scale_stride(K), n_rows};
  switch (t) {
    case ElemType::kF32: return dequantize<float>(p, num_cus, st);
    case ElemType::kBF16: return dequantize<bf16>(p, num_cus, st);
    default: return dequantize<f16>(p, num_cus, st);
  }
}

hipError_t launch_mx_gemm(const RaggedShape& s, const int32_t* offsets, const uint8_t* xq,
                          const uint8_t* xs, const uint8_t* wq, const uint8_t* ws, void* y,
                          int num_cus, hipStream_t st) {
  if (s.rows == 0) return hipSuccess;
  const int64_t es = elem_bytes(s.type);
  if (s.rows > 16 * (int64_t)s.E) {
    RingParams r{};
    r.act = reinterpret_cast<const char*>(xq);
    r.w = reinterpret_cast<const char*>(wq);
    r.act_scales = reinterpret_cast<const char*>(xs);
    r.w_scales = reinterpret_cast<const char*>(ws);
    r.out = static_cast<char*>(y);
    r.offsets = offsets;
    r.lda = r.ldw = s.K / 2;
    r.ldo = s.ld_y * es;
    r.lds = mx_scale_stride(s.K);
    r.wbytes = (int64_t)s.N * s.K / 2;
    r.rows = (int)s.rows;
    r.E = s.E;
    r.B = s.N;
    r.cbytes = s.K / 2;
    r.out_vec = s.N % (16 / es) == 0 && s.ld_y % (16 / es) == 0 && aligned16(y);
    return launch_ring(s.type == ElemType::kBF16  ? RingKind::kMxBF16
                       : s.type == ElemType::kF16 ? RingKind::kMxF16
                                                  : RingKind::kMxF32,
                       r, num_cus, st);
  }
  const MxParams p{xq,     xs,          wq,  ws,  y,   offsets,
                   s.ld_y, (int)s.rows, s.E, s.N, s.K, (int)mx_scale_stride(s.K), 0};
  switch (s.type) {
    case ElemType::kF32: return mx_gemm<float>(p, num_cus, st);
    case ElemType::kBF16: return mx_gemm<bf16>(p, num_cus, st);
    default: return mx_gemm<f16>(p, num_cus, st);
  }
}

}  // namespace moe
