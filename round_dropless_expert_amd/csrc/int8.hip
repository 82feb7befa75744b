// Rows in 8-bit integers with a scale each, and the product over rows sorted
// by expert of such rows and weights.
//
//   scale = max|x| / 127     q = 127 x / max|x| to nearest, ties to even
//
// The code is that of the exact quotient. With v = 127 / max|x| in fp32, x v lies
// within 127 2^-24 of it, and one fma with 1.5 2^23 rounds x v to an integer; an
// x v nearer than 2^-16 to the middle of two is divided in fp64 (127 x is exact
// there, and a quotient that is no tie lies at least 2^-33 from one). Seven
// instructions an element, which is what keeps the quantisation at the memory's
// rate.
//
// 98304 rows of 7168 bf16 gathered from 16384 tokens: 340-345 us (1.41 GB asked for,
// 0.70 GB stored, 6.2 TB/s). A token is read, its maximum found and its codes rounded
// for each of its six rows anew: the tokens once and the codes are 184 us at a copy's
// rate. Back to bf16 343-370 us (2.1 GB, 5.7-6.1 TB/s).
#include "ragged_device.hpp"
#include "ragged_ring.hpp"
#include "router.hpp"

namespace moe {
namespace {

typedef signed char i8;

constexpr int kRsrcWord3 = 0x00020000;  // raw buffer
constexpr int kNonTemporal = 2;

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

// From any address, values past K zero.
template <typename T>
__device__ __forceinline__ Vec<T> load_row(const T* row, int64_t c, int64_t K, bool real) {
  constexpr int V = Vec<T>::V;
  Vec<T> r;
  r.v = u32x4{0, 0, 0, 0};
  if (!real) return r;
  if (c + V <= K) {
    __builtin_memcpy(&r.v, row + c, 16);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (c + i < K) r.e[i] = row[c + i];
  }
  return r;
}

// Largest magnitude of a vector, as bits in the order of the values (NaN above
// infinity above numbers), and its fp32 bits.
template <typename T>
__device__ __forceinline__ uint32_t top_of(const Vec<T>& x, uint32_t top) {
  if constexpr (sizeof(T) == 2) {
    typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
    u16x2 m = __builtin_bit_cast(u16x2, top);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, x.v[i] & 0x7fff7fffu));
    return __builtin_bit_cast(uint32_t, m);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t b = x.v[i] & 0x7fffffffu;
      top = top > b ? top : b;
    }
    return top;
  }
}
template <typename T>
__device__ __forceinline__ uint32_t top_bits(uint32_t top) {
  if constexpr (sizeof(T) == 2) {
    const uint32_t lo = top & 0xffffu, hi = top >> 16, m = lo > hi ? lo : hi;
    return __builtin_bit_cast(uint32_t, to_f32(__builtin_bit_cast(T, (uint16_t)m)));
  } else {
    return top;
  }
}

// Codes of a vector, four a word; true if one of them needs the quotient.
template <typename T>
__device__ __forceinline__ bool codes_of(const Vec<T>& x, float inv,
                                         uint32_t (&out)[Vec<T>::V / 4]) {
  constexpr int V = Vec<T>::V;
  constexpr float kMagic = 0x1.8p23f;  // its neighbours are integers apart
  float worst = 0.f;
  uint32_t code[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const float f = to_f32(x.e[i]);
    const float t = __builtin_fmaf(f, inv, kMagic);
    code[i] = __builtin_bit_cast(uint32_t, t);
    worst = fmaxf(worst, __builtin_fabsf(__builtin_fmaf(f, inv, -(t - kMagic))));
  }
#pragma unroll
  for (int i = 0; i < V / 4; ++i) {
    const uint32_t lo = __builtin_amdgcn_perm(code[4 * i + 1], code[4 * i], 0x0c0c0400u);
    const uint32_t hi = __builtin_amdgcn_perm(code[4 * i + 3], code[4 * i + 2], 0x04000c0cu);
    out[i] = lo | hi;
  }
  return worst > 0.5f - 0x1p-16f;
}
// The codes by fp64 quotients, an element at a time: rare, and no reason to hold
// registers.
template <typename T>
__device__ __forceinline__ void exact_codes_of(const Vec<T>& x, float top,
                                               uint32_t (&out)[Vec<T>::V / 4]) {
  constexpr int V = Vec<T>::V;
  uint64_t all = 0;
#pragma unroll 1
  for (int i = V - 1; i >= 0; --i) {
    const int w = sizeof(T) == 2 ? i / 2 : i;
    const uint32_t word = w == 0 ? x.v[0] : w == 1 ? x.v[1] : w == 2 ? x.v[2] : x.v[3];
    float f;
    if constexpr (sizeof(T) == 2)
      f = to_f32(__builtin_bit_cast(T, (uint16_t)(i & 1 ? word >> 16 : word)));
    else
      f = __builtin_bit_cast(float, word);
    const int c = (int)__builtin_rint(127.0 * (double)f / (double)top);
    all = all << 8 | (uint32_t)(c & 255);
  }
  out[0] = (uint32_t)all;
  if constexpr (V == 8) out[1] = (uint32_t)(all >> 32);
}

// A row that is read and written. kVec: its wavefronts share it and its addresses
// are 16-byte aligned and hold whole 4-byte words; loads and stores then go through
// buffer ranges, with no branch at its end. (With branches each load waited for the
// one before: 98304 rows of 7168 bf16 took 560 us.)
template <typename T, bool kVec>
struct Row {
  const T* in;
  i8* out;
  int64_t K;
  int per;  // vectors, the padding included
  bool real;
  __amdgpu_buffer_rsrc_t src, dst;

  __device__ __forceinline__ void set(const QuantParams& p, int64_t row) {
    int64_t from = row;
    real = true;
    if (p.index) {
      const int32_t a = p.index[row];
      from = a < 0 ? -1 : a / p.index_div;
      real = from >= 0 && from < p.src_rows;
    }
    in = static_cast<const T*>(p.x) + (real ? from : 0) * p.ld_x;
    out = p.codes + row * p.stride;
    K = p.K;
    per = (int)(p.stride / Vec<T>::V);
    if constexpr (kVec) {
      src = __builtin_amdgcn_make_buffer_rsrc(
          (void*)in, 0, real ? (int)(K * sizeof(T)) : 0, kRsrcWord3);
      dst = __builtin_amdgcn_make_buffer_rsrc((void*)out, 0, (int)p.stride, kRsrcWord3);
    }
  }
  __device__ __forceinline__ Vec<T> load(int v) const {
    if constexpr (kVec) {
      Vec<T> r;
      r.v = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(src, v * 16, 0, 0));
      return r;
    } else {
      return load_row(in, (int64_t)v * Vec<T>::V, K, real && v < per);
    }
  }
  __device__ __forceinline__ void store(const uint32_t (&w)[Vec<T>::V / 4], int v) const {
    typedef uint32_t words_t __attribute__((ext_vector_type(Vec<T>::V / 4)));
    words_t o;
#pragma unroll
    for (int i = 0; i < Vec<T>::V / 4; ++i) o[i] = w[i];
    if constexpr (kVec) {
      if constexpr (sizeof(T) == 2)
        __builtin_amdgcn_raw_buffer_store_b64(o, dst, v * 8, 0, kNonTemporal);
      else
        __builtin_amdgcn_raw_buffer_store_b32(w[0], dst, v * 4, 0, kNonTemporal);
    } else if (v < per) {
      __builtin_nontemporal_store(o, reinterpret_cast<words_t*>(out + (int64_t)v * Vec<T>::V));
    }
  }
};

// kLanes lanes a row, kHeld 16-byte vectors of it in each lane's registers; what a
// longer row has beyond them is read a second time, and so are the vectors that
// need quotients.
template <typename T, int kLanes, int kHeld, bool kVec>
__global__ __launch_bounds__(256) void int8_quantize_kernel(QuantParams p) {
  constexpr int V = Vec<T>::V;
  static_assert(kLanes >= kWave || !kVec, "a wavefront's row is one");
  __shared__ uint32_t tops[2][4];
  const int lane = threadIdx.x % kLanes;
  const int64_t rows = live_rows(p.rows, p.n_rows);
  int turn = 0;
  int64_t row = (int64_t)blockIdx.x * (256 / kLanes) + threadIdx.x / kLanes;
  if constexpr (kLanes >= kWave)  // uniform
    row = (int64_t)blockIdx.x * (256 / kLanes) +
          __builtin_amdgcn_readfirstlane(threadIdx.x / kLanes);
  for (; row < rows; row += (int64_t)gridDim.x * (256 / kLanes)) {
    Row<T, kVec> r;
    r.set(p, row);
    Vec<T> x[kHeld];
    uint32_t top = 0;
#pragma unroll
    for (int u = 0; u < kHeld; ++u) x[u] = r.load(lane + u * kLanes);
#pragma unroll
    for (int u = 0; u < kHeld; ++u) top = top_of<T>(x[u], top);
    for (int v = lane + kHeld * kLanes; v < r.per; v += kLanes) top = top_of<T>(r.load(v), top);
    top = top_bits<T>(top);
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
    const float most = bad ? 0.f : __builtin_bit_cast(float, top);
    const bool exact = most < 0x1p-100f && most > 0.f;  // too small for 127 / most
    const float inv = most == 0.f || exact ? 0.f : 127.f / most;
    uint32_t redo = 0;  // bit u: of the vectors held
#pragma unroll
    for (int u = 0; u < kHeld; ++u) {
      uint32_t w[V / 4];
      redo |= (uint32_t)codes_of<T>(x[u], inv, w) << u;
#pragma unroll
      for (int i = 0; i < V / 4; ++i) w[i] = bad ? 0 : w[i];
      r.store(w, lane + u * kLanes);
    }
    redo = bad ? 0 : exact ? (1u << kHeld) - 1 : redo;
    while (redo) {
      const int v = lane + __builtin_ctz(redo) * kLanes;
      redo &= redo - 1;
      uint32_t w[V / 4];
      exact_codes_of<T>(r.load(v), most, w);
      r.store(w, v);
    }
    for (int v = lane + kHeld * kLanes; v < r.per; v += kLanes) {
      const Vec<T> again = r.load(v);
      uint32_t w[V / 4];
      if ((codes_of<T>(again, inv, w) || exact) && !bad) exact_codes_of<T>(again, most, w);
#pragma unroll
      for (int i = 0; i < V / 4; ++i) w[i] = bad ? 0 : w[i];
      r.store(w, v);
    }
    if (lane == 0) p.scales[row] = bad ? __builtin_nanf("") : most / 127.f;
  }
}

struct DequantParams {
  const i8* codes;
  const float* scales;
  void* y;
  int64_t ld_y, rows, K, stride;
  const int32_t* n_rows;
  int strips, log_lanes;
};

// A unit is 64 16-byte vectors of values of a row for a wavefront, or a row of few
// vectors for a power of two of its lanes.
template <typename T, bool kVec>
__global__ __launch_bounds__(256) void int8_dequantize_kernel(DequantParams p) {
  constexpr int V = Vec<T>::V;
  const int lane = threadIdx.x & ((1 << p.log_lanes) - 1);
  const int at_once = 256 >> p.log_lanes;
  const int64_t units = live_rows(p.rows, p.n_rows) * p.strips;
  for (int64_t u = (int64_t)blockIdx.x * at_once + (threadIdx.x >> p.log_lanes); u < units;
       u += (int64_t)gridDim.x * at_once) {
    const int64_t row = p.strips == 1 ? u : u / p.strips;
    const int64_t c = (((u - row * p.strips) << p.log_lanes) + lane) * V;
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

template <typename T, int kLanes, int kHeld>
hipError_t quantize_lanes(const QuantParams& p, int num_cus, hipStream_t st) {
  const int64_t blocks = (p.rows + 256 / kLanes - 1) / (256 / kLanes);
  const int64_t most = (int64_t)num_cus * 64;
  const dim3 grid((unsigned)(blocks < most ? blocks : most));
  if constexpr (kLanes >= kWave) {
    if (p.ld_x % Vec<T>::V == 0 && aligned16(p.x) && p.K * sizeof(T) % 4 == 0) {
      hipLaunchKernelGGL((int8_quantize_kernel<T, kLanes, kHeld, true>), grid, dim3(256), 0, st,
                         p);
      return hipGetLastError();
    }
  }
  hipLaunchKernelGGL((int8_quantize_kernel<T, kLanes, kHeld, false>), grid, dim3(256), 0, st, p);
  return hipGetLastError();
}

// A wavefront a row while its registers hold one: no barrier, and the row's loads
// are all in flight. A few lanes where a row has few vectors, a workgroup where
// it has many; no more vectors held than the row has. bf16, by lanes and vectors
// held: 200000 rows of 512 61 us with 16 x 4, 108 with 64 x 4; 100000 of 1024 65 with
// 64 x 4, 92 with 64 x 8; 30000 of 4096 65 with 64 x 8, 69 with 64 x 16, 109 with 256 x
// 8; 10000 of 16384 87 with 256 x 8, 138 with 64 x 16.
template <typename T>
hipError_t quantize(const QuantParams& p, int num_cus, hipStream_t st) {
  const int64_t per = p.stride / Vec<T>::V;
  if (per <= 16) return quantize_lanes<T, 16, 1>(p, num_cus, st);
  if (per <= 16 * 4) return quantize_lanes<T, 16, 4>(p, num_cus, st);
  if (per <= kWave * 4) return quantize_lanes<T, kWave, 4>(p, num_cus, st);
  if (per <= kWave * 8) return quantize_lanes<T, kWave, 8>(p, num_cus, st);
  if (per <= kWave * 16) return quantize_lanes<T, kWave, 16>(p, num_cus, st);
  return quantize_lanes<T, 256, 8>(p, num_cus, st);
}

template <typename T>
hipError_t dequantize(DequantParams p, int num_cus, hipStream_t st) {
  constexpr int V = Vec<T>::V;
  p.log_lanes = 0;
  while (p.log_lanes < 6 && ((int64_t)V << p.log_lanes) < p.K) ++p.log_lanes;
  p.strips = (int)((p.K + kWave * V - 1) / (kWave * V));
  const int64_t at_once = 256 >> p.log_lanes;
  const int64_t blocks = (p.rows * p.strips + at_once - 1) / at_once;
  const int64_t most = (int64_t)num_cus * 1024;
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
                        int8_stride(K), n_rows, 0, 0};
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
