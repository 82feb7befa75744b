// Routing with scores, a bias for balance, and groups of experts, and the
// gradient of its weights.
//
//   s = softmax(l) or 1 / (1 + e^-l)     c = s + bias
//   group score = sum of the group's best one or two c; the best groups stay
//   idx = experts of the k largest c     w = scale s_idx (/ sum s_idx)
//
// The choice is the one that fp64 arithmetic makes. That is dear for every
// expert and needed for few tokens: the fast kernel scores in fp32, with a
// bound on its error, and a token in which two values that decide something
// lie closer than the bound is chosen again by the exact routine.
//
// The weights are fp32 functions of the chosen logits, computed so that they
// neither overflow nor vanish together: a softmax over the chosen logits, or
// sigmoids with a common factor where all of them are small.
#include "ragged_device.hpp"
#include "router.hpp"

namespace moe {
namespace {

__device__ __forceinline__ bool no_number(float l) { return !(l > -INFINITY); }  // -inf, NaN

template <typename T>
__device__ __forceinline__ float load_f32(const T* p) {
  return to_f32(*p);
}

// Maximum and sum over the kLanes neighbouring lanes of a segment.
template <int kLanes>
__device__ __forceinline__ float seg_max(float v) {
#pragma unroll
  for (int x = 1; x < kLanes; x <<= 1) v = fmaxf(v, __shfl_xor(v, x));
  return v;
}
template <int kLanes>
__device__ __forceinline__ float seg_sum(float v) {
#pragma unroll
  for (int x = 1; x < kLanes; x <<= 1) v += __shfl_xor(v, x);
  return v;
}

// e^(l - top), 1 where both are infinite.
__device__ __forceinline__ float exp_below(float l, float top) {
  return no_number(l) ? 0.f : l == top ? 1.f : expf(l - top);
}

// 1 / (1 + e^-l) times e^-m for m = min(0, top), top >= l: the sigmoids of a
// token's chosen logits, with a common factor that keeps the largest near 1.
__device__ __forceinline__ float sigmoid_above(float l, float top) {
  if (no_number(l)) return 0.f;
  if (l >= 0.f) return 1.f / (1.f + expf(-l));
  return expf(l - fminf(top, 0.f)) / (1.f + expf(l));
}

// Weights of a token: kLanes lanes hold its chosen logits (use: this lane
// holds one). top, sum: the maximum of all the token's logits and the sum of
// e^(l - top), for the softmax over all experts.
template <int kLanes>
__device__ __forceinline__ float weight_of(float l, bool use, float top, float sum, bool sigmoid,
                                           bool renormalize, float scale) {
  if (!renormalize) {
    if (sigmoid) return scale * sigmoid_above(l, 0.f);
    return sum > 0.f ? scale * (exp_below(l, top) / sum) : 0.f;
  }
  const float best = seg_max<kLanes>(use && !no_number(l) ? l : -INFINITY);
  const float e = !use ? 0.f : sigmoid ? sigmoid_above(l, best) : exp_below(l, best);
  const float all = seg_sum<kLanes>(e);
  return all > 0.f ? scale * (e / all) : 0.f;
}

// A token's choice in fp64, by one wavefront. Lane l holds experts l + 64 m.
// `c` is the wavefront's share of LDS, E doubles (used with groups).
template <typename T, int M>
__device__ __forceinline__ void route_exact(const RouterParams& p, int64_t t, double* c) {
  const int lane = threadIdx.x & (kWave - 1);
  const T* row = static_cast<const T*>(p.logits) + t * p.ld;
  float l[M];
  float top = -INFINITY;
#pragma unroll
  for (int m = 0; m < M; ++m) {
    const int e = lane + kWave * m;
    l[m] = e < p.E ? load_f32(row + e) : -INFINITY;
    if (!no_number(l[m])) top = fmaxf(top, l[m]);
  }
  top = seg_max<kWave>(top);
  float sum32 = 0.f;
  double s[M];
  double sum = 0.0;
  if (!p.sigmoid) {
#pragma unroll
    for (int m = 0; m < M; ++m) {
      s[m] = no_number(l[m]) ? 0.0 : l[m] == top ? 1.0 : exp((double)l[m] - (double)top);
      sum += s[m];
    }
#pragma unroll
    for (int x = 1; x < kWave; x <<= 1) sum += __shfl_xor(sum, x);
    sum32 = (float)sum;
#pragma unroll
    for (int m = 0; m < M; ++m) s[m] = s[m] / sum;
  } else {
#pragma unroll
    for (int m = 0; m < M; ++m) s[m] = 1.0 / (1.0 + exp(-(double)l[m]));
  }
  // what can be chosen: bit m of `open`
  uint32_t open = 0;
#pragma unroll
  for (int m = 0; m < M; ++m) {
    const int e = lane + kWave * m;
    if (e < p.E) {
      open |= 1u << m;
      if (p.bias) s[m] += (double)p.bias[e];
      if (no_number(l[m]) || !(s[m] == s[m])) s[m] = -INFINITY;
    }
  }
  if (p.groups > 1) {
#pragma unroll
    for (int m = 0; m < M; ++m)
      if (lane + kWave * m < p.E) c[lane + kWave * m] = s[m];
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    double first = -INFINITY, second = -INFINITY;
    if (lane < p.groups)
      for (int i = 0; i < p.per_group; ++i) {
        const double v = c[lane * p.per_group + i];
        second = v > first ? first : (v > second ? v : second);
        first = v > first ? v : first;
      }
    double g = p.group_top == 2 && p.per_group > 1 ? first + second : first;
    if (!(g == g)) g = -INFINITY;
    int ahead = 0;  // groups that come before this lane's
    for (int q = 0; q < p.groups; ++q) {
      const double o = __shfl(g, q);
      ahead += (o > g) | ((o == g) & (q < lane));
    }
    const uint64_t keep = __builtin_amdgcn_ballot_w64(lane < p.groups && ahead < p.top_groups);
#pragma unroll
    for (int m = 0; m < M; ++m) {
      const int e = lane + kWave * m;
      if (e < p.E && !((keep >> (e / p.per_group)) & 1)) open &= ~(1u << m);
    }
    __builtin_amdgcn_wave_barrier();
  }
  // without a bias experts rank by their logits
  if (!p.bias)
#pragma unroll
    for (int m = 0; m < M; ++m) s[m] = no_number(l[m]) ? -INFINITY : (double)l[m];

  float mine = 0.f;
  int chosen = 0;
  for (int j = 0; j < p.k; ++j) {
    double v = -INFINITY;
    int at = 0x7fffffff;
#pragma unroll
    for (int m = 0; m < M; ++m)
      if ((open >> m) & 1 && (at == 0x7fffffff || s[m] > v)) {
        v = s[m];
        at = lane + kWave * m;
      }
#pragma unroll
    for (int x = 1; x < kWave; x <<= 1) {
      const double ov = __shfl_xor(v, x);
      const int oa = __shfl_xor(at, x);
      if (ov > v || (ov == v && oa < at)) {
        v = ov;
        at = oa;
      }
    }
    // its logit, from the lane that holds it
    float lv = 0.f;
#pragma unroll
    for (int m = 0; m < M; ++m)
      if (at == lane + kWave * m) {
        lv = l[m];
        open &= ~(1u << m);
      }
    lv = __shfl(lv, at & (kWave - 1));
    if (lane == j) {
      mine = lv;
      chosen = at;
    }
  }
  const bool use = lane < p.k;
  const float w =
      weight_of<kWave>(mine, use, top, sum32, p.sigmoid, p.renormalize, p.scale);
  if (use) {
    p.idx[t * p.k + lane] = chosen;
    p.weight[t * p.k + lane] = w;
  }
}

template <typename T, int M>
__global__ __launch_bounds__(256) void router_exact_kernel(RouterParams p) {
  __shared__ double c[4][kWave * M];
  const int wave = threadIdx.x / kWave;
  for (int64_t t = (int64_t)blockIdx.x * 4 + wave; t < p.T; t += (int64_t)gridDim.x * 4)
    route_exact<T, M>(p, t, c[wave]);
}

template <typename T>
hipError_t route(const RouterParams& p, int num_cus, hipStream_t st) {
  const int64_t blocks = (p.T + 3) / 4, most = (int64_t)num_cus * 32;
  const dim3 grid((unsigned)(blocks < most ? blocks : most));
#define MOE_EXACT(M) \
  hipLaunchKernelGGL((router_exact_kernel<T, M>), grid, dim3(256), 0, st, p)
  if (p.E <= 64) MOE_EXACT(1);
  else if (p.E <= 128) MOE_EXACT(2);
  else if (p.E <= 256) MOE_EXACT(4);
  else if (p.E <= 512) MOE_EXACT(8);
  else MOE_EXACT(16);
#undef MOE_EXACT
  return hipGetLastError();
}

// ---------------------------------------------------------------- gradient
// With w_j = scale s_j (/ sum), g_j = scale dweight_j over the chosen j:
//   softmax, renormalised   dl_j = w_j (g_j - sum w g)      (w: without scale)
//   sigmoid, renormalised   dl_j = w_j (g_j - sum w g) (1 - s_j)
//   sigmoid                 dl_j = s_j (1 - s_j) g_j
//   softmax                 dl_e = s_e (g_e - sum s g)      for every expert
// kLanes lanes a token. What the chosen experts get is left in LDS, one value
// each; then every lane writes its experts' gradients, whole rows at once.
constexpr int kGradTokens = 32;  // of a workgroup at most

template <typename T, int kLanes, bool kVec>
__global__ __launch_bounds__(256) void router_grad_kernel(RouterGradParams p) {
  constexpr int V = kVec ? 16 / sizeof(T) : 1;
  constexpr int kTokens = 256 / kLanes;
  static_assert(kTokens <= kGradTokens, "share of LDS");
  __shared__ float val[kTokens][kRouterMaxTopK];
  __shared__ int32_t at[kTokens][kRouterMaxTopK];
  const int q = threadIdx.x % kLanes, seg = threadIdx.x / kLanes;
  const bool full = !p.sigmoid && !p.renormalize;
  const int64_t steps = (p.T + kTokens - 1) / kTokens;
  for (int64_t step = blockIdx.x; step < steps; step += gridDim.x) {
    const int64_t t = step * kTokens + seg;
    const bool live = t < p.T;
    const T* row = static_cast<const T*>(p.logits) + (live ? t : 0) * p.ld;
    T* out = static_cast<T*>(p.dlogits) + (live ? t : 0) * p.ld;
    // the softmax over all experts
    float top = -INFINITY, inv = 0.f;
    if (full) {
      if (live)
        for (int e = q; e < p.E; e += kLanes) {
          const float l = load_f32(row + e);
          if (!no_number(l)) top = fmaxf(top, l);
        }
      top = seg_max<kLanes>(top);
      float sum = 0.f;
      if (live)
        for (int e = q; e < p.E; e += kLanes) sum += exp_below(load_f32(row + e), top);
      sum = seg_sum<kLanes>(sum);
      inv = sum > 0.f ? 1.f / sum : 0.f;
    } else if (p.renormalize) {
      if (live)
        for (int j = q; j < p.k; j += kLanes) {
          const int e = p.idx[t * p.k + j];
          if (e >= 0 && e < p.E) {
            const float l = load_f32(row + e);
            if (!no_number(l)) top = fmaxf(top, l);
          }
        }
      top = seg_max<kLanes>(top);
    }
    // the chosen experts' scores, and the sums over them
    float sum = 0.f, dot = 0.f;
    if (live)
      for (int j = q; j < p.k; j += kLanes) {
        const int e = p.idx[t * p.k + j];
        const bool in = e >= 0 && e < p.E;
        const float l = in ? load_f32(row + e) : -INFINITY;
        const float g = p.scale * p.dweight[t * p.k + j];
        float s;
        if (full) s = exp_below(l, top) * inv;
        else if (!p.sigmoid) s = exp_below(l, top);
        else s = sigmoid_above(l, p.renormalize ? top : 0.f);
        sum += s;
        dot += s > 0.f ? s * g : 0.f;
        at[seg][j] = in ? e : -1;
        val[seg][j] = s;
      }
    sum = seg_sum<kLanes>(sum);
    dot = seg_sum<kLanes>(dot);
    if (p.renormalize) dot = sum > 0.f ? dot / sum : 0.f;
    if (live)
      for (int j = q; j < p.k; j += kLanes) {
        const float s = val[seg][j];
        const float g = p.scale * p.dweight[t * p.k + j];
        const int e = at[seg][j];
        float v = g;
        if (!full) {
          const float l = e >= 0 ? load_f32(row + e) : -INFINITY;
          v = p.renormalize ? s / sum * (g - dot) : s * g;
          // 1 - 1 / (1 + e^-l)
          if (p.sigmoid)
            v *= l >= 0.f ? expf(-l) / (1.f + expf(-l)) : 1.f / (1.f + expf(l));
          if (!(s > 0.f)) v = 0.f;
        }
        val[seg][j] = v;
      }
    __syncthreads();
    if (live)
      for (int e0 = q * V; e0 < p.E; e0 += kLanes * V) {
        const int n = p.E - e0 < V ? p.E - e0 : V;
        float d[V] = {};
        for (int j = 0; j < p.k; ++j) {
          const int e = at[seg][j] - e0;
          const float v = val[seg][j];
#pragma unroll
          for (int i = 0; i < V; ++i) d[i] += e == i ? v : 0.f;
        }
        if (full)
#pragma unroll
          for (int i = 0; i < V; ++i) {
            const float s = i < n ? exp_below(load_f32(row + e0 + i), top) * inv : 0.f;
            d[i] = s > 0.f ? s * (d[i] - dot) : 0.f;
          }
        union {
          T e[V];
          u32x4 v;
        } o;
#pragma unroll
        for (int i = 0; i < V; ++i) o.e[i] = from_f32<T>(d[i]);
        if (kVec && n == V) {
          *reinterpret_cast<u32x4*>(out + e0) = o.v;
        } else {
#pragma unroll
          for (int i = 0; i < V; ++i)
            if (i < n) out[e0 + i] = o.e[i];
        }
      }
    __syncthreads();
  }
}

template <typename T, int kLanes>
hipError_t grad_lanes(const RouterGradParams& p, int num_cus, hipStream_t st) {
  const int64_t steps = (p.T * kLanes + 255) / 256, most = (int64_t)num_cus * 16;
  const dim3 grid((unsigned)(steps < most ? steps : most));
  if (p.vec)
    hipLaunchKernelGGL((router_grad_kernel<T, kLanes, true>), grid, dim3(256), 0, st, p);
  else
    hipLaunchKernelGGL((router_grad_kernel<T, kLanes, false>), grid, dim3(256), 0, st, p);
  return hipGetLastError();
}

template <typename T>
hipError_t grad(const RouterGradParams& p, int num_cus, hipStream_t st) {
  const int per = p.vec ? p.E / (int)(16 / sizeof(T)) : p.E;
  if (per <= 8) return grad_lanes<T, 8>(p, num_cus, st);
  if (per <= 16) return grad_lanes<T, 16>(p, num_cus, st);
  if (per <= 32) return grad_lanes<T, 32>(p, num_cus, st);
  return grad_lanes<T, 64>(p, num_cus, st);
}

}  // namespace

hipError_t launch_router(ElemType t, const RouterParams& p, int num_cus, hipStream_t st) {
  if (p.T == 0) return hipSuccess;
  switch (t) {
    case ElemType::kF32: return route<float>(p, num_cus, st);
    case ElemType::kBF16: return route<bf16>(p, num_cus, st);
    default: return route<f16>(p, num_cus, st);
  }
}

hipError_t launch_router_backward(ElemType t, const RouterGradParams& p, int num_cus,
                                  hipStream_t st) {
  if (p.T == 0) return hipSuccess;
  switch (t) {
    case ElemType::kF32: return grad<float>(p, num_cus, st);
    case ElemType::kBF16: return grad<bf16>(p, num_cus, st);
    default: return grad<f16>(p, num_cus, st);
  }
}

}  // namespace moe
