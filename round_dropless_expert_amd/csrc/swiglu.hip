// SwiGLU between the experts' products, and its gradient, on rows [g, u]:
//
//   h = g s(g) u        s = 1 / (1 + e^-g)
//   du = dh g s
//   dg = dh u s (1 + g (1 - s))
//
// All arithmetic is fp32; h, dg and du are rounded once, to their type.
//
// Bound by memory: one pass, 3 and 5 values moved a feature. 98304 rows of
// 2048 features, bf16: 191 us forward (1.21 GB, 6.3 TB/s), 323 us backward
// (2.01 GB, 6.2 TB/s); a 4 GiB copy moves 4.8 TB/s. A row's lanes are a power
// of two, so no lane divides, and outputs are stored past the caches, which
// leaves those to the inputs (648 us for both passes without either, 514
// with). Rows that 16-byte vectors do not fit (2047 features, or 4099 elements
// apart) go element by element: 231 and 440 us.
#include "ragged_device.hpp"

namespace moe {
namespace {

// s(g) and 1 - s(g), both to a few ulp for every g of at least kTail: with a =
// e^-|g| they are 1 / (1 + a) and a / (1 + a), in the order of g's sign, so
// neither cancels and no exponential overflows.
struct Gate {
  float s, rest;
};
// For 16-bit types the hardware's base-2 exponential and reciprocal (1 ulp
// each; the product |g| log2 e is off by at most |g| 2^-24 relative, far
// below half a step of fp16); for fp32 the full-precision functions.
template <typename T>
__device__ __forceinline__ Gate gate(float g) {
  float a, r;
  if constexpr (sizeof(T) == 2) {
    a = __builtin_amdgcn_exp2f(__builtin_fabsf(g) * -1.44269504088896341f);
    r = __builtin_amdgcn_rcpf(1.0f + a);
  } else {
    a = expf(-__builtin_fabsf(g));
    r = 1.0f / (1.0f + a);
  }
  const float q = a * r;
  return g >= 0.f ? Gate{r, q} : Gate{q, r};
}

// Below kTail s(g) leaves fp32's normal numbers (e^-87.3 = 2^-126; the hardware
// exponential returns 0 there), while its products with u and dh need not. It
// is e^g to 2^-124 then, kept as a value and a power of two, and so are the
// products (Scaled). Below kZero every product is 0 in fp32, and fp16 values are
// too small for one to reach fp16's least subnormal. One comparison per vector
// finds these features; their outputs are stored a second time, from operands
// that are read again behind the row's others, so that those hold no registers
// for them. The comparison costs nothing that can be measured (191 and 325 us
// with and without it); with such a feature in every row the passes above take
// 486 and 706 us.
constexpr float kTail = -86.f, kZero = -1024.f;
template <typename T>
constexpr bool kHasTail = !__is_same(T, f16);

struct Scaled {  // m 2^e
  float m;
  int e;
  __device__ __forceinline__ Scaled times(float v) const {
    return Scaled{m * __builtin_amdgcn_frexp_mantf(v), e + __builtin_amdgcn_frexp_expf(v)};
  }
  __device__ __forceinline__ float value() const { return __builtin_ldexpf(m, e); }
};
// e^g for kZero < g < 0: g log2 e less its nearest integer to fp32's precision
// by log2 e in two parts.
__device__ __forceinline__ Scaled scaled_exp(float g) {
  constexpr double kLog2e = 1.44269504088896340736;
  constexpr float kHigh = (float)kLog2e, kLow = (float)(kLog2e - kHigh);
  const float n = __builtin_rintf(g * kHigh);
  const float r = __builtin_fmaf(g, kLow, __builtin_fmaf(g, kHigh, -n));
  return Scaled{__builtin_amdgcn_exp2f(r), (int)n};
}

template <typename T, int V>
struct Vec {
  T e[V];
};

// Whether any g may lie below kTail: of negative values, as unsigned numbers
// the larger are further from zero (and of NaN, which store_tail leaves out).
template <typename T, int V>
__device__ __forceinline__ bool in_tail(const Vec<T, V>& g) {
  if constexpr (!kHasTail<T>) return false;
  constexpr uint32_t kBits = __builtin_bit_cast(uint32_t, kTail);
  if constexpr (sizeof(T) == 4) {
    typedef uint32_t uint_t __attribute__((ext_vector_type(V)));
    return __builtin_reduce_max(__builtin_bit_cast(uint_t, g)) > kBits;
  } else {
    typedef uint16_t uint_t __attribute__((ext_vector_type(V)));
    return __builtin_reduce_max(__builtin_bit_cast(uint_t, g)) > kBits >> 16;
  }
}

template <typename T, int V>
__device__ __forceinline__ Vec<T, V> load(const T* p) {
  if constexpr (V == 1) {
    return Vec<T, 1>{{*p}};
  } else {
    return __builtin_bit_cast(
        Vec<T, V>, __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p)));
  }
}
template <typename T, int V>
__device__ __forceinline__ void store(T* p, const Vec<T, V>& v) {
  if constexpr (V == 1)
    *p = v.e[0];
  else
    __builtin_nontemporal_store(__builtin_bit_cast(u32x4, v), reinterpret_cast<u32x4*>(p));
}

template <typename T, int V, bool kBackward>
__device__ __forceinline__ void store_tail(const T* gu, const T* dh, T* out, int64_t f,
                                           int64_t at) {
#pragma unroll 1
  for (int v = 0; v < V; ++v, ++at) {
    const float g = to_f32(gu[at]);
    if (!(g < kTail && g > kZero)) continue;
    const Scaled s = scaled_exp(g), gs = s.times(g);
    const float u = to_f32(gu[f + at]);
    if constexpr (!kBackward) {
      out[at] = from_f32<T>(gs.times(u).value());
    } else {  // 1 - s is 1
      const float d = to_f32(dh[at]);
      out[at] = from_f32<T>(s.times(1.0f + g).times(u).times(d).value());
      out[f + at] = from_f32<T>(gs.times(d).value());
    }
  }
}

struct SwigluParams {
  const void* gu;
  const void* dh;
  void* out;  // h or dgu
  int64_t ld_gu, ld_dh, ld_out;
  const int32_t* n_rows;
  int64_t rows;
  int64_t f;
  int log_lanes;  // lanes per row
};

constexpr int kUnroll = 2;  // vectors a lane has in flight per operand

// 2^log_lanes lanes a row, each V features at a time. All of it is read and
// written once: non-temporal.
template <typename T, int V, bool kBackward>
__global__ __launch_bounds__(256) void swiglu_kernel(SwigluParams p) {
  const int64_t rows = live_rows(p.rows, p.n_rows);
  const int per = (int)(p.f / V);
  const int lanes = 1 << p.log_lanes, c0 = threadIdx.x & (lanes - 1);
  const int64_t row0 = (int64_t)blockIdx.x * (256 >> p.log_lanes) + (threadIdx.x >> p.log_lanes);
  for (int64_t row = row0; row < rows; row += (int64_t)gridDim.x * (256 >> p.log_lanes)) {
    const T* gu = static_cast<const T*>(p.gu) + row * p.ld_gu;
    const T* dh = static_cast<const T*>(p.dh) + row * p.ld_dh;
    T* out = static_cast<T*>(p.out) + row * p.ld_out;
    bool tail = false;
    for (int c = c0; c < per; c += lanes * kUnroll) {
      Vec<T, V> g[kUnroll], u[kUnroll], d[kUnroll];
#pragma unroll
      for (int k = 0; k < kUnroll; ++k) {
        const int64_t at = (int64_t)(c + k * lanes) * V;
        if (c + k * lanes < per) {
          g[k] = load<T, V>(gu + at);
          u[k] = load<T, V>(gu + p.f + at);
          if constexpr (kBackward) d[k] = load<T, V>(dh + at);
        }
      }
#pragma unroll
      for (int k = 0; k < kUnroll; ++k) {
        if (c + k * lanes >= per) break;
        const int64_t at = (int64_t)(c + k * lanes) * V;
        tail |= in_tail(g[k]);
        if constexpr (!kBackward) {
          Vec<T, V> h;
#pragma unroll
          for (int v = 0; v < V; ++v) {
            const float gf = to_f32(g[k].e[v]);
            h.e[v] = from_f32<T>(gf * gate<T>(gf).s * to_f32(u[k].e[v]));
          }
          store<T, V>(out + at, h);
        } else {
          Vec<T, V> dg, du;
#pragma unroll
          for (int v = 0; v < V; ++v) {
            const float gf = to_f32(g[k].e[v]), df = to_f32(d[k].e[v]);
            const Gate q = gate<T>(gf);
            dg.e[v] = from_f32<T>(df * (q.s * (1.0f + gf * q.rest)) * to_f32(u[k].e[v]));
            du.e[v] = from_f32<T>(df * (gf * q.s));
          }
          store<T, V>(out + at, dg);
          store<T, V>(out + p.f + at, du);
        }
      }
    }
    if (tail) {
#pragma unroll 1
      for (int c = c0; c < per; c += lanes)
        store_tail<T, V, kBackward>(gu, dh, out, p.f, (int64_t)c * V);
    }
  }
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

template <typename T, bool kBackward>
hipError_t run(SwigluParams p, int num_cus, hipStream_t st) {
  constexpr int kV = 16 / sizeof(T);
  // 16-byte vectors where every row of every buffer starts at one
  const bool vec = p.f % kV == 0 && p.ld_gu % kV == 0 && p.ld_out % kV == 0 &&
                   (!kBackward || p.ld_dh % kV == 0) && aligned16(p.gu) && aligned16(p.out) &&
                   (!kBackward || aligned16(p.dh));
  const int64_t per = vec ? p.f / kV : p.f;
  // lanes per row: a power of two that leaves a lane about kUnroll vectors
  p.log_lanes = 3;
  while (p.log_lanes < 8 && ((int64_t)kUnroll << p.log_lanes) < per) ++p.log_lanes;
  const int64_t at_once = 256 >> p.log_lanes, blocks = (p.rows + at_once - 1) / at_once;
  const int64_t most = (int64_t)num_cus * 64;
  const unsigned grid = (unsigned)(blocks < most ? blocks : most);
  if (vec)
    hipLaunchKernelGGL((swiglu_kernel<T, kV, kBackward>), dim3(grid), dim3(256), 0, st, p);
  else
    hipLaunchKernelGGL((swiglu_kernel<T, 1, kBackward>), dim3(grid), dim3(256), 0, st, p);
  return hipGetLastError();
}

template <bool kBackward>
hipError_t dispatch(ElemType t, const SwigluParams& p, int num_cus, hipStream_t st) {
  if (p.rows == 0) return hipSuccess;
  switch (t) {
    case ElemType::kF32: return run<float, kBackward>(p, num_cus, st);
    case ElemType::kBF16: return run<bf16, kBackward>(p, num_cus, st);
    default: return run<f16, kBackward>(p, num_cus, st);
  }
}

}  // namespace

hipError_t launch_swiglu(ElemType t, int64_t rows, int64_t f, const void* gu, int64_t ld_gu,
                         void* h, int64_t ld_h, const int32_t* n_rows, int num_cus,
                         hipStream_t st) {
  return dispatch<false>(t, SwigluParams{gu, nullptr, h, ld_gu, 0, ld_h, n_rows, rows, f, 0},
                         num_cus, st);
}

hipError_t launch_swiglu_backward(ElemType t, int64_t rows, int64_t f, const void* gu,
                                  int64_t ld_gu, const void* dh, int64_t ld_dh, void* dgu,
                                  int64_t ld_dgu, const int32_t* n_rows, int num_cus,
                                  hipStream_t st) {
  return dispatch<true>(t, SwigluParams{gu, dh, dgu, ld_gu, ld_dh, ld_dgu, n_rows, rows, f, 0},
                        num_cus, st);
}

}  // namespace moe
