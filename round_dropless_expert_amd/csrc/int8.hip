// Rows in 8-bit integers with a scale each, and the product over rows sorted
// by expert of such rows and weights.
//
//   scale = max|x| / 127     q = 127 x / max|x| to nearest, ties to even
//
// The code is that of the exact quotient: 127 x / max|x| in fp32 is off by less
// than 127 2^-22, and a value nearer than that to the middle of two codes is
// divided in fp64 (127 x is exact there, and a quotient that is no tie lies at
// least 2^-33 from one).
#include "ragged_device.hpp"
#include "ragged_ring.hpp"
#include "router.hpp"

namespace moe {
namespace {

typedef signed char i8;

// 16-byte vectors of a row that a lane holds.
constexpr int kHeld = 8;

struct QuantParams {
  const void* x;
  int64_t ld_x, src_rows;
  const int32_t* index;
  int index_div;
  const int32_t* n_rows;
  int64_t rows, K, stride;
  i8* codes;
  float* scales;
};

template <typename T>
struct Vec {
  static constexpr int V = 16 / sizeof(T);
  union {
    T e[V];
    u32x4 v;
  };
};

template <typename T, bool kVec>
__device__ __forceinline__ Vec<T> load_row(const T* row, int64_t c, int64_t K, bool real) {
  constexpr int V = Vec<T>::V;
  Vec<T> r;
  r.v = u32x4{0, 0, 0, 0};
  if (!real) return r;
  if (c + V <= K) {
    if constexpr (kVec)
      r.v = *reinterpret_cast<const u32x4*>(row + c);
    else
      __builtin_memcpy(&r.v, row + c, 16);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (c + i < K) r.e[i] = row[c + i];
  }
  return r;
}

// Largest magnitude, as fp32 bits (NaN above infinity above numbers).
template <typename T>
__device__ __forceinline__ uint32_t top_of(const Vec<T>& x, uint32_t top) {
#pragma unroll
  for (int i = 0; i < Vec<T>::V; ++i) {
    const uint32_t b = __builtin_bit_cast(uint32_t, to_f32(x.e[i])) & 0x7fffffffu;
    top = top > b ? top : b;
  }
  return top;
}

struct Quant {
  float top, inv;  // max|x|, 127 / max|x|
  bool exact;      // too small for inv
};
__device__ __forceinline__ int code_of(float x, const Quant& q) {
  const float r = x * q.inv;
  const float n = __builtin_rintf(r);
  // |r - n| <= 1/2; near 1/2 the quotient decides
  if (q.exact || __builtin_fabsf(__builtin_fabsf(r - n) - 0.5f) < 0x1p-14f)
    return (int)__builtin_rint(127.0 * (double)x / (double)q.top);
  return (int)n;
}

// kLanes lanes a row, kHeld vectors of it in each lane's registers; what a
// longer row has beyond them is read a second time.
template <typename T, int kLanes, bool kVec>
__global__ __launch_bounds__(256) void int8_quantize_kernel(QuantParams p) {
  constexpr int V = Vec<T>::V;
  __shared__ uint32_t tops[2][4];
  const int lane = threadIdx.x % kLanes;
  const int per = (int)(p.stride / V);  // vectors of a row, its padding included
  const int64_t rows = live_rows(p.rows, p.n_rows);
  int turn = 0;
  for (int64_t row = (int64_t)blockIdx.x * (256 / kLanes) + threadIdx.x / kLanes; row < rows;
       row += (int64_t)gridDim.x * (256 / kLanes)) {
    int64_t src = row;
    bool real = true;
    if (p.index) {
      const int32_t a = p.index[row];
      src = a < 0 ? -1 : a / p.index_div;
      real = src >= 0 && src < p.src_rows;
    }
    const T* in = static_cast<const T*>(p.x) + (real ? src : 0) * p.ld_x;
    Vec<T> x[kHeld];
    uint32_t top = 0;
#pragma unroll
    for (int u = 0; u < kHeld; ++u)
      x[u] = load_row<T, kVec>(in, (int64_t)(lane + u * kLanes) * V, p.K,
                               real && lane + u * kLanes < per);
#pragma unroll
    for (int u = 0; u < kHeld; ++u) top = top_of<T>(x[u], top);
    for (int v = lane + kHeld * kLanes; v < per; v += kLanes)
      top = top_of<T>(load_row<T, kVec>(in, (int64_t)v * V, p.K, real), top);
#pragma unroll
    for (int s = 1; s < (kLanes < kWave ? kLanes : kWave); s <<= 1) {
      const uint32_t o = __shfl_xor(top, s);
      top = top > o ? top : o;
    }
    if constexpr (kLanes > kWave) {
      // (two sets: a wavefront may be a row ahead of another's reads)
      static_assert(kLanes == 256, "a row a workgroup");
      if (threadIdx.x % kWave == 0) tops[turn][threadIdx.x / kWave] = top;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < 4; ++w) top = top > tops[turn][w] ? top : tops[turn][w];
      turn ^= 1;
    }
    const bool bad = top >= 0x7f800000u;
    Quant q;
    q.top = __builtin_bit_cast(float, top);
    q.exact = top < 0x0d800000u && top != 0;  // 2^-100
    q.inv = top == 0 || bad || q.exact ? 0.f : 127.f / q.top;
    i8* out = p.codes + row * p.stride;
    auto put = [&](const Vec<T>& xv, int v) {
      union {
        i8 b[V];
        uint32_t w[V / 4];
      } o;
#pragma unroll
      for (int i = 0; i < V; ++i) o.b[i] = bad ? (i8)0 : (i8)code_of(to_f32(xv.e[i]), q);
#pragma unroll
      for (int i = 0; i < V / 4; ++i)
        __builtin_nontemporal_store(o.w[i], reinterpret_cast<uint32_t*>(out + (int64_t)v * V) + i);
    };
#pragma unroll
    for (int u = 0; u < kHeld; ++u)
      if (lane + u * kLanes < per) put(x[u], lane + u * kLanes);
    for (int v = lane + kHeld * kLanes; v < per; v += kLanes)
      put(load_row<T, kVec>(in, (int64_t)v * V, p.K, real), v);
    if (lane == 0) p.scales[row] = bad ? __builtin_nanf("") : q.top / 127.f;
  }
}

struct DequantParams {
  const i8* codes;
  const float* scales;
  void* y;
  int64_t ld_y, rows, K, stride;
  const int32_t* n_rows;
  int strips;
};

// A wavefront takes 64 16-byte vectors of values of a row.
template <typename T, bool kVec>
__global__ __launch_bounds__(256) void int8_dequantize_kernel(DequantParams p) {
  constexpr int V = Vec<T>::V;
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int64_t units = live_rows(p.rows, p.n_rows) * p.strips;
  for (int64_t u = (int64_t)blockIdx.x * 4 + wave; u < units; u += (int64_t)gridDim.x * 4) {
    const int64_t row = u / p.strips;
    const int64_t c = ((u - row * p.strips) * kWave + lane) * V;
    if (c >= p.K) continue;
    union {
      i8 b[V];
      uint32_t w[V / 4];
    } q;
    const uint32_t* in = reinterpret_cast<const uint32_t*>(p.codes + row * p.stride + c);
#pragma unroll
    for (int i = 0; i < V / 4; ++i) q.w[i] = in[i];
    const float s = p.scales[row];
    Vec<T> o;
#pragma unroll
    for (int i = 0; i < V; ++i) o.e[i] = from_f32<T>((float)q.b[i] * s);
    T* out = static_cast<T*>(p.y) + row * p.ld_y + c;
    if (c + V <= p.K) {
      if constexpr (kVec)
        __builtin_nontemporal_store(o.v, reinterpret_cast<u32x4*>(out));
      else
        __builtin_memcpy(out, &o.v, 16);
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (c + i < p.K) out[i] = o.e[i];
    }
  }
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

template <typename T, int kLanes>
hipError_t quantize_lanes(const QuantParams& p, int num_cus, hipStream_t st) {
  const int64_t blocks = (p.rows + 256 / kLanes - 1) / (256 / kLanes);
  const int64_t most = (int64_t)num_cus * 256;
  const dim3 grid((unsigned)(blocks < most ? blocks : most));
  if (p.ld_x % Vec<T>::V == 0 && aligned16(p.x))
    hipLaunchKernelGGL((int8_quantize_kernel<T, kLanes, true>), grid, dim3(256), 0, st, p);
  else
    hipLaunchKernelGGL((int8_quantize_kernel<T, kLanes, false>), grid, dim3(256), 0, st, p);
  return hipGetLastError();
}

template <typename T>
hipError_t quantize(const QuantParams& p, int num_cus, hipStream_t st) {
  const int64_t per = p.stride / Vec<T>::V;
  if (per <= 16 * kHeld) return quantize_lanes<T, 16>(p, num_cus, st);
  if (per <= kWave * kHeld) return quantize_lanes<T, kWave>(p, num_cus, st);
  return quantize_lanes<T, 256>(p, num_cus, st);
}

template <typename T>
hipError_t dequantize(DequantParams p, int num_cus, hipStream_t st) {
  constexpr int V = Vec<T>::V;
  p.strips = (int)((p.K + kWave * V - 1) / (kWave * V));
  const int64_t blocks = (p.rows * p.strips + 3) / 4, most = (int64_t)num_cus * 1024;
  const dim3 grid((unsigned)(blocks < most ? blocks : most));
  if (p.ld_y % V == 0 && aligned16(p.y))
    hipLaunchKernelGGL((int8_dequantize_kernel<T, true>), grid, dim3(256), 0, st, p);
  else
    hipLaunchKernelGGL((int8_dequantize_kernel<T, false>), grid, dim3(256), 0, st, p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_int8_quantize(ElemType t, int64_t rows, int64_t K, const void* x, int64_t ld_x,
                                int64_t src_rows, const int32_t* index, int index_div,
                                const int32_t* n_rows, int8_t* codes, float* scales, int num_cus,
                                hipStream_t st) {
  if (rows == 0) return hipSuccess;
  const QuantParams p{x,    ld_x, src_rows,       index, index_div, n_rows,
                      rows, K,    int8_stride(K), reinterpret_cast<i8*>(codes), scales};
  switch (t) {
    case ElemType::kF32: return quantize<float>(p, num_cus, st);
    case ElemType::kBF16: return quantize<bf16>(p, num_cus, st);
    default: return quantize<f16>(p, num_cus, st);
  }
}

hipError_t launch_int8_dequantize(ElemType t, int64_t rows, int64_t K, const int8_t* codes,
                                  const float* scales, void* y, int64_t ld_y,
                                  const int32_t* n_rows, int num_cus, hipStream_t st) {
  if (rows == 0) return hipSuccess;
  const DequantParams p{reinterpret_cast<const i8*>(codes), scales, y, ld_y, rows, K,
                        int8_stride(K), n_rows, 0};
  switch (t) {
    case ElemType::kF32: return dequantize<float>(p, num_cus, st);
    case ElemType::kBF16: return dequantize<bf16>(p, num_cus, st);
    default: return dequantize<f16>(p, num_cus, st);
  }
}

hipError_t launch_int8_gemm(const RaggedShape& s, const int32_t* offsets, const int8_t* xq,
                            const float* xs, const int8_t* wq, const float* ws, void* y,
                            int num_cus, hipStream_t st) {
  if (s.rows == 0) return hipSuccess;
  const int64_t es = elem_bytes(s.type), stride = int8_stride(s.K);
  RingParams r{};
  r.act = reinterpret_cast<const char*>(xq);
  r.w = reinterpret_cast<const char*>(wq);
  r.act_scales = reinterpret_cast<const char*>(xs);
  r.w_scales = reinterpret_cast<const char*>(ws);
  r.out = static_cast<char*>(y);
  r.offsets = offsets;
  r.lda = r.ldw = stride;
  r.ldo = s.ld_y * es;
  r.wbytes = (int64_t)s.N * stride;
  r.rows = (int)s.rows;
  r.E = s.E;
  r.B = s.N;
  r.cbytes = (int)stride;
  r.out_vec = s.N % (16 / es) == 0 && s.ld_y % (16 / es) == 0 && aligned16(y);
  return launch_ring(s.type == ElemType::kBF16  ? RingKind::kI8BF16
                     : s.type == ElemType::kF16 ? RingKind::kI8F16
                                                : RingKind::kI8F32,
                     r, num_cus, st);
}

}  // namespace moe
