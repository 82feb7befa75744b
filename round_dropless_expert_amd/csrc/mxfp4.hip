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

// 16-byte vectors a lane has in flight. 98304 rows of 7168 bf16, to 4 bits and
// back: 581 us with 4, 557 with 8.
constexpr int kUnroll = 8;

// gfx950 converts two values at a time to and from the 4-bit format with a
// scale (an fp32 power of two, of which it uses the exponent): to nearest,
// ties to even, ending at 6, fp32 subnormals included.
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ float scale_of(int byte) {
  return __builtin_bit_cast(float, (uint32_t)byte << 23);
}

template <typename T>
struct Codec;
template <>
struct Codec<bf16> {
  typedef bf16x2 pair_t;
  // largest magnitude of 16 bytes, as bits in the order of the values
  __device__ static __forceinline__ uint32_t top(u32x4 v) { return top16(v); }
  // and its fp32 bits
  __device__ static __forceinline__ uint32_t bits(uint32_t t) { return t << 16; }
  __device__ static __forceinline__ uint32_t top16(u32x4 v) {
    typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
    u16x2 m = {0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, v[i] & 0x7fff7fffu));
    return m[0] > m[1] ? m[0] : m[1];
  }
  template <int kByte>
  __device__ static __forceinline__ uint32_t encode(uint32_t old, u32x4 v, float s) {
    const uint32_t two = v[kByte];
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(old, __builtin_bit_cast(pair_t, two), s, kByte);
  }
  template <int kByte>
  __device__ static __forceinline__ pair_t decode(uint32_t q, float s) {
    return __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, s, kByte);
  }
};
template <>
struct Codec<f16> {
  typedef f16x2 pair_t;
  __device__ static __forceinline__ uint32_t top(u32x4 v) { return Codec<bf16>::top16(v); }
  __device__ static __forceinline__ uint32_t bits(uint32_t t) {
    return __builtin_bit_cast(uint32_t, (float)__builtin_bit_cast(f16, (uint16_t)t));
  }
  template <int kByte>
  __device__ static __forceinline__ uint32_t encode(uint32_t old, u32x4 v, float s) {
    const uint32_t two = v[kByte];
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(old, __builtin_bit_cast(pair_t, two), s, kByte);
  }
  template <int kByte>
  __device__ static __forceinline__ pair_t decode(uint32_t q, float s) {
    return __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(q, s, kByte);
  }
};
template <>
struct Codec<float> {
  typedef f32x2 pair_t;
  __device__ static __forceinline__ uint32_t top(u32x4 v) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t b = v[i] & 0x7fffffffu;
      m = m > b ? m : b;
    }
    return m;
  }
  __device__ static __forceinline__ uint32_t bits(uint32_t t) { return t; }
  template <int kByte>
  __device__ static __forceinline__ uint32_t encode(uint32_t old, u32x4 v, float s) {
    const uint32_t a = v[2 * kByte], b = v[2 * kByte + 1];
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(old, __builtin_bit_cast(float, a),
                                                    __builtin_bit_cast(float, b), s, kByte);
  }
  template <int kByte>
  __device__ static __forceinline__ pair_t decode(uint32_t q, float s) {
    return __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, s, kByte);
  }
};

// Largest of the values of a block's lanes, 4 or 8 neighbours.
template <int kLanes>
__device__ __forceinline__ uint32_t block_max(uint32_t v) {
#define MOE_MAX_STEP(ctrl)                                                                \
  {                                                                                       \
    const uint32_t o = (uint32_t)__builtin_amdgcn_mov_dpp((int)v, ctrl, 0xf, 0xf, true);  \
    v = v > o ? v : o;                                                                    \
  }
  MOE_MAX_STEP(0xb1)  // lanes 1, 0, 3, 2 of each four
  MOE_MAX_STEP(0x4e)  // lanes 2, 3, 0, 1
  if constexpr (kLanes == 8) MOE_MAX_STEP(0x141)  // each eight mirrored
#undef MOE_MAX_STEP
  return v;
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
  int log_lanes;   // lanes per row
};

// A lane takes V = 16 bytes of a row at a time (kVec: the row's addresses
// are 16-byte aligned), 32 / V neighbours a block: their maximum is exchanged
// by DPP, and each stores V / 2 bytes of codes. kUnroll vectors of a row are
// in flight per lane.
//
// Bound by memory: 98304 rows of 7168 bf16 gathered from 16384 tokens, 237-243
// us (1.41 GB asked for and 0.37 GB stored, 7.4 TB/s: a token's later reads come
// from the caches; read once it would be 0.6 GB in all).
template <typename T, bool kVec>
__global__ __launch_bounds__(256) void mx_quantize_kernel(QuantParams p) {
  constexpr int V = 16 / sizeof(T);
  constexpr int kLanes = kMxBlock / V;
  const int per = (int)(p.K / V);
  const int64_t rows = live_rows(p.rows, p.n_rows);
  const int lanes = 1 << p.log_lanes, c0 = threadIdx.x & (lanes - 1);
  const int64_t row0 = (int64_t)blockIdx.x * (256 >> p.log_lanes) + (threadIdx.x >> p.log_lanes);
  for (int64_t row = row0; row < rows; row += (int64_t)gridDim.x * (256 >> p.log_lanes)) {
    int64_t src = row;
    bool real = true;
    if (p.index) {
      const int32_t a = p.index[row];
      src = a < 0 ? -1 : a / p.index_div;
      real = src >= 0 && src < p.src_rows;
    }
    const T* in = static_cast<const T*>(p.x) + (real ? src : 0) * p.ld_x;
    uint8_t* out = p.codes + row * (p.K / 2);
    uint8_t* sc = p.scales + row * p.stride;
    for (int c = c0; c < per; c += lanes * kUnroll) {
      u32x4 x[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        x[u] = u32x4{0, 0, 0, 0};
        const int v = c + u * lanes;
        if (v < per && real) {
          if constexpr (kVec) {
            x[u] = *reinterpret_cast<const u32x4*>(in + (int64_t)v * V);
          } else {
            __builtin_memcpy(&x[u], in + (int64_t)v * V, 16);
          }
        }
      }
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int v = c + u * lanes;
        if (v >= per) break;  // a block's lanes go together
        const uint32_t top = Codec<T>::bits(block_max<kLanes>(Codec<T>::top(x[u])));
        // The scale's byte is the exponent field - 2, at least 0; infinities
        // and NaN have the largest exponent field.
        const int field = (int)(top >> 23);
        const bool bad = field == 255;
        const int byte = bad ? 255 : (field > 2 ? field - 2 : 0);
        const float s = scale_of(byte);
        uint32_t q = Codec<T>::template encode<0>(0u, x[u], s);
        q = Codec<T>::template encode<1>(q, x[u], s);
        if constexpr (V == 8) {
          q = Codec<T>::template encode<2>(q, x[u], s);
          q = Codec<T>::template encode<3>(q, x[u], s);
          *reinterpret_cast<uint32_t*>(out + v * 4) = bad ? 0 : q;
        } else {
          *reinterpret_cast<uint16_t*>(out + v * 2) = (uint16_t)(bad ? 0 : q);
        }
        if (v % kLanes == 0) sc[v / kLanes] = (uint8_t)byte;
      }
    }
    // the padding of the scale row: blocks that hold nothing
    if (c0 < p.stride - p.K / kMxBlock) sc[p.K / kMxBlock + c0] = 0;
  }
}

struct DequantParams {
  const uint8_t* codes;
  const uint8_t* scales;
  void* y;
  int64_t ld_y, rows, K, stride;
  const int32_t* n_rows;
  int log_lanes;
};

// The inverse: a lane reads V / 2 bytes of codes and stores 16 bytes of
// values, past the caches. Bound by the stores: 98304 rows of 7168 bf16, 317-320
// us (0.37 GB read, 1.41 GB stored, 5.6 TB/s).
template <typename T, bool kVec>
__global__ __launch_bounds__(256) void mx_dequantize_kernel(DequantParams p) {
  constexpr int V = 16 / sizeof(T);
  const int per = (int)(p.K / V);
  const int64_t rows = live_rows(p.rows, p.n_rows);
  const int lanes = 1 << p.log_lanes, c0 = threadIdx.x & (lanes - 1);
  const int64_t row0 = (int64_t)blockIdx.x * (256 >> p.log_lanes) + (threadIdx.x >> p.log_lanes);
  for (int64_t row = row0; row < rows; row += (int64_t)gridDim.x * (256 >> p.log_lanes)) {
    const uint8_t* in = p.codes + row * (p.K / 2);
    const uint8_t* sc = p.scales + row * p.stride;
    T* out = static_cast<T*>(p.y) + row * p.ld_y;
    for (int c = c0; c < per; c += lanes * kUnroll) {
      uint32_t q[kUnroll];
      int s[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int v = c + u * lanes;
        q[u] = s[u] = 0;
        if (v < per) {
          q[u] = V == 8 ? *reinterpret_cast<const uint32_t*>(in + v * 4)
                        : *reinterpret_cast<const uint16_t*>(in + v * 2);
          s[u] = sc[v * V / kMxBlock];
        }
      }
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int v = c + u * lanes;
        if (v >= per) break;
        const float f = scale_of(s[u]);
        union {
          typename Codec<T>::pair_t e[V / 2];
          T t[V];
          u32x4 v;
        } y;
        y.e[0] = Codec<T>::template decode<0>(q[u], f);
        y.e[1] = Codec<T>::template decode<1>(q[u], f);
        if constexpr (V == 8) {
          y.e[2] = Codec<T>::template decode<2>(q[u], f);
          y.e[3] = Codec<T>::template decode<3>(q[u], f);
        }
        if (s[u] == 255) {
#pragma unroll
          for (int k = 0; k < V; ++k) y.t[k] = from_f32<T>(__builtin_nanf(""));
        }
        if constexpr (kVec)
          __builtin_nontemporal_store(y.v, reinterpret_cast<u32x4*>(out + (int64_t)v * V));
        else
          __builtin_memcpy(out + (int64_t)v * V, &y.v, 16);
      }
    }
  }
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// Lanes per row: a power of two that leaves a lane about kUnroll vectors of
// the row, 8 (a block's lanes) to 256.
int log_lanes_of(int64_t per) {
  int l = 3;
  while (l < 8 && ((int64_t)kUnroll << l) < per) ++l;
  return l;
}

unsigned grid_of(int64_t rows, int log_lanes, int num_cus) {
  const int64_t at_once = 256 >> log_lanes, blocks = (rows + at_once - 1) / at_once;
  const int64_t most = (int64_t)num_cus * 64;
  return (unsigned)(blocks < most ? blocks : most);
}

template <typename T>
hipError_t quantize(QuantParams p, int num_cus, hipStream_t st) {
  constexpr int V = 16 / sizeof(T);
  p.log_lanes = log_lanes_of(p.K / V);
  const unsigned grid = grid_of(p.rows, p.log_lanes, num_cus);
  if (p.ld_x % V == 0 && aligned16(p.x))
    hipLaunchKernelGGL((mx_quantize_kernel<T, true>), dim3(grid), dim3(256), 0, st, p);
  else
    hipLaunchKernelGGL((mx_quantize_kernel<T, false>), dim3(grid), dim3(256), 0, st, p);
  return hipGetLastError();
}

template <typename T>
hipError_t dequantize(DequantParams p, int num_cus, hipStream_t st) {
  constexpr int V = 16 / sizeof(T);
  p.log_lanes = log_lanes_of(p.K / V);
  const unsigned grid = grid_of(p.rows, p.log_lanes, num_cus);
  if (p.ld_y % V == 0 && aligned16(p.y))
    hipLaunchKernelGGL((mx_dequantize_kernel<T, true>), dim3(grid), dim3(256), 0, st, p);
  else
    hipLaunchKernelGGL((mx_dequantize_kernel<T, false>), dim3(grid), dim3(256), 0, st, p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_mx_quantize(ElemType t, int64_t rows, int64_t K, const void* x, int64_t ld_x,
                              int64_t src_rows, const int32_t* index, int index_div,
                              const int32_t* n_rows, uint8_t* codes, uint8_t* scales,
                              int num_cus, hipStream_t st) {
  if (rows == 0) return hipSuccess;
  const QuantParams p{x,    ld_x, src_rows, index,  index_div,         n_rows,
                      rows, K,    codes,    scales, mx_scale_stride(K), 0};
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
  const DequantParams p{codes, scales, y, ld_y, rows, K, mx_scale_stride(K), n_rows, 0};
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

}  // namespace moe
