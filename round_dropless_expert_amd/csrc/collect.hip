// The experts' outputs back to tokens, and the gradients of that sum.
//
//   y[t] = sum_j w[t][j] z[pos[t][j]]
//   dz[pos[t][j]] = w[t][j] dy[t]      dw[t][j] = <z[pos[t][j]], dy[t]>
//
// Sums are fp32 over ascending j; y and dz are rounded once.
//
// Bound by memory. Every row is read and written once, in strips of 64
// 16-byte vectors: a wavefront takes a strip of a token and has the k rows'
// loads in flight together, so that one token of a wide layer is spread over
// many CUs and any d and k keep the same loop. With the weights' gradient a
// wavefront takes a whole row instead, one (t, j) each: its dot product then
// stays in the wavefront, and the k reads of dy[t] by neighbouring wavefronts
// come from the caches.
//
// 16384 tokens, 6 experts each, d = 7168, bf16: the sum 282-294 us (1.64 GB, 5.7
// TB/s; 354 with a branch at each load), both gradients
// 585-590 us (3.05 GB, 5.2 TB/s), dz alone, the gather into expert order, 263 us (1.64
// GB, 6.2 TB/s: a strip is read once and stored past the caches); a device copy moves
// 5.1 TB/s. 5 tokens of 1001 values: 3.3 us each.
#include "ragged_device.hpp"
#include "router.hpp"

namespace moe {
namespace {

// V elements of a row from column c on, of which n exist.
template <typename T>
struct Vec {
  static constexpr int V = 16 / sizeof(T);
  union {
    T e[V];
    u32x4 v;
  };
};
template <typename T, bool kVec>
__device__ __forceinline__ Vec<T> load_vec(const T* p, int n) {
  constexpr int V = Vec<T>::V;
  Vec<T> r;
  if (n >= V) {
    if constexpr (kVec)
      r.v = *reinterpret_cast<const u32x4*>(p);
    else
      __builtin_memcpy(&r.v, p, 16);
  } else {
    r.v = u32x4{0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i < n) r.e[i] = p[i];
  }
  return r;
}

// Stored past the caches, which leaves those to the rows that are read.
template <typename T, bool kVec>
__device__ __forceinline__ void store_vec(T* p, int n, const float* v) {
  constexpr int V = 16 / sizeof(T);
  union {
    T e[V];
    u32x4 v;
  } r;
#pragma unroll
  for (int i = 0; i < V; ++i) r.e[i] = from_f32<T>(v[i]);
  if (n >= V) {
    if constexpr (kVec)
      __builtin_nontemporal_store(r.v, reinterpret_cast<u32x4*>(p));
    else
      __builtin_memcpy(p, &r.v, 16);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i < n) p[i] = r.e[i];
  }
}

constexpr int kAtOnce = 4;  // rows of a token in flight (eight are no faster)

// kWhole: every strip is whole (d is a multiple of 64 vectors), so that no load
// depends on a branch.
template <typename T, bool kVec, bool kWhole>
__global__ __launch_bounds__(256) void collect_kernel(CollectParams p, int strips) {
  constexpr int V = Vec<T>::V;
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int64_t units = p.T * strips;
  for (int64_t u = (int64_t)blockIdx.x * 4 + wave; u < units; u += (int64_t)gridDim.x * 4) {
    const int64_t t = u / strips;
    const int64_t c = ((u - t * strips) * kWave + lane) * V;
    const int n = kWhole ? V : (int)(p.d - c < V ? p.d - c : V);
    const T* z = static_cast<const T*>(p.z) + c;
    float acc[V] = {};
    for (int j0 = 0; j0 < p.k; j0 += kAtOnce) {
      Vec<T> v[kAtOnce];
      float w[kAtOnce];
      bool real[kAtOnce];  // uniform
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j) {
        const bool in = j0 + j < p.k;
        const int64_t a = t * p.k + (in ? j0 + j : 0);
        const int64_t row = in ? p.pos[a] : -1;
        real[j] = row >= 0 && row < p.rows;
        w[j] = p.weight ? p.weight[a] : 1.f;
        if (real[j])
          v[j] = load_vec<T, kVec>(z + row * p.ld_z, n);
      }
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j)
        if (real[j])
#pragma unroll
          for (int i = 0; i < V; ++i) acc[i] = fmaf(w[j], to_f32(v[j].e[i]), acc[i]);
    }
    if (n > 0) store_vec<T, kVec>(static_cast<T*>(p.y) + t * p.ld_y + c, n, acc);
  }
}

// dz alone: a strip of dy is read once and stored k times.
template <typename T, bool kVec>
__global__ __launch_bounds__(256) void spread_kernel(CollectParams p, int strips) {
  constexpr int V = 16 / sizeof(T);
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int64_t units = p.T * strips;
  for (int64_t u = (int64_t)blockIdx.x * 4 + wave; u < units; u += (int64_t)gridDim.x * 4) {
    const int64_t t = u / strips;
    const int64_t c = ((u - t * strips) * kWave + lane) * V;
    const int n = (int)(p.d - c < V ? p.d - c : V);
    if (n <= 0) continue;
    const Vec<T> g = load_vec<T, kVec>(static_cast<const T*>(p.dy) + t * p.ld_y + c, n);
    for (int j = 0; j < p.k; ++j) {
      const int64_t a = t * p.k + j;
      const int64_t row = p.pos[a];
      if (row < 0 || row >= p.rows) continue;
      const float w = p.weight ? p.weight[a] : 1.f;
      float v[V];
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] = w * to_f32(g.e[i]);
      store_vec<T, kVec>(static_cast<T*>(p.dz) + row * p.ld_dz + c, n, v);
    }
  }
}

// U vectors of both rows in flight.
template <typename T, bool kVec, int U>
__global__ __launch_bounds__(256) void collect_grad_kernel(CollectParams p) {
  constexpr int V = Vec<T>::V;
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int64_t units = p.T * p.k;
  for (int64_t a = (int64_t)blockIdx.x * 4 + wave; a < units; a += (int64_t)gridDim.x * 4) {
    const int64_t t = a / p.k;
    const int64_t row = p.pos[a];
    if (row < 0 || row >= p.rows) {
      if (lane == 0) p.dweight[a] = 0.f;
      continue;
    }
    const float w = p.weight ? p.weight[a] : 1.f;
    const T* dy = static_cast<const T*>(p.dy) + t * p.ld_y;
    const T* z = static_cast<const T*>(p.z) + row * p.ld_z;
    T* dz = static_cast<T*>(p.dz) + row * p.ld_dz;
    float dot = 0.f;
    // whole turns of U vectors a lane without a check, then vector by vector
    int64_t c0 = (int64_t)lane * V;
    auto use = [&](const Vec<T>& g, const Vec<T>& v, int64_t c, int n) {
      float o[V];
#pragma unroll
      for (int i = 0; i < V; ++i) {
        dot = fmaf(to_f32(v.e[i]), to_f32(g.e[i]), dot);
        o[i] = w * to_f32(g.e[i]);
      }
      if (p.dz) store_vec<T, kVec>(dz + c, n, o);
    };
    for (; c0 - (int64_t)lane * V + U * kWave * V <= p.d; c0 += U * kWave * V) {
      Vec<T> g[U], v[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        g[u] = load_vec<T, kVec>(dy + c0 + u * kWave * V, V);
        v[u] = load_vec<T, kVec>(z + c0 + u * kWave * V, V);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) use(g[u], v[u], c0 + u * kWave * V, V);
    }
    for (; c0 < p.d; c0 += kWave * V) {
      const int n = (int)(p.d - c0 < V ? p.d - c0 : V);
      use(load_vec<T, kVec>(dy + c0, n), load_vec<T, kVec>(z + c0, n), c0, n);
    }
#pragma unroll
    for (int x = 1; x < kWave; x <<= 1) dot += __shfl_xor(dot, x);
    if (lane == 0) p.dweight[a] = dot;
  }
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

unsigned grid_of(int64_t units, int num_cus) {
  const int64_t blocks = (units + 3) / 4, most = (int64_t)num_cus * 1024;
  return (unsigned)(blocks < most ? blocks : most);
}

template <typename T>
hipError_t collect(const CollectParams& p, int num_cus, hipStream_t st) {
  constexpr int V = 16 / sizeof(T);
  const int strips = (int)((p.d + kWave * V - 1) / (kWave * V));
  const bool vec = p.ld_z % V == 0 && p.ld_y % V == 0 && aligned16(p.z) && aligned16(p.y);
  const dim3 grid(grid_of(p.T * strips, num_cus));
  const bool whole = p.d % (kWave * V) == 0;
  if (vec && whole)
    hipLaunchKernelGGL((collect_kernel<T, true, true>), grid, dim3(256), 0, st, p, strips);
  else if (vec)
    hipLaunchKernelGGL((collect_kernel<T, true, false>), grid, dim3(256), 0, st, p, strips);
  else
    hipLaunchKernelGGL((collect_kernel<T, false, false>), grid, dim3(256), 0, st, p, strips);
  return hipGetLastError();
}

template <typename T>
hipError_t collect_backward(const CollectParams& p, int num_cus, hipStream_t st) {
  constexpr int V = 16 / sizeof(T);
  bool vec = p.ld_y % V == 0 && aligned16(p.dy);
  if (p.dz) vec = vec && p.ld_dz % V == 0 && aligned16(p.dz);
  if (!p.dweight) {
    const int strips = (int)((p.d + kWave * V - 1) / (kWave * V));
    const dim3 grid(grid_of(p.T * strips, num_cus));
    if (vec)
      hipLaunchKernelGGL((spread_kernel<T, true>), grid, dim3(256), 0, st, p, strips);
    else
      hipLaunchKernelGGL((spread_kernel<T, false>), grid, dim3(256), 0, st, p, strips);
    return hipGetLastError();
  }
  vec = vec && p.ld_z % V == 0 && aligned16(p.z);
  const dim3 grid(grid_of(p.T * p.k, num_cus));
  if (vec)
    hipLaunchKernelGGL((collect_grad_kernel<T, true, 4>), grid, dim3(256), 0, st, p);
  else
    hipLaunchKernelGGL((collect_grad_kernel<T, false, 4>), grid, dim3(256), 0, st, p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_collect(ElemType t, const CollectParams& p, int num_cus, hipStream_t st) {
  if (p.T == 0) return hipSuccess;
  switch (t) {
    case ElemType::kF32: return collect<float>(p, num_cus, st);
    case ElemType::kBF16: return collect<bf16>(p, num_cus, st);
    default: return collect<f16>(p, num_cus, st);
  }
}

hipError_t launch_collect_backward(ElemType t, const CollectParams& p, int num_cus,
                                   hipStream_t st) {
  if (p.T == 0 || (!p.dz && !p.dweight)) return hipSuccess;
  switch (t) {
    case ElemType::kF32: return collect_backward<float>(p, num_cus, st);
    case ElemType::kBF16: return collect_backward<bf16>(p, num_cus, st);
    default: return collect_backward<f16>(p, num_cus, st);
  }
}

}  // namespace moe
