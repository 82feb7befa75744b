// Routing with scores, a bias for balance, and groups of experts, and the
// gradient of its weights.
//
//   s = softmax(l) or 1 / (1 + e^-l)     c = s + bias
//   group score = sum of the group's best one or two c; the best groups stay
//   idx = experts of the k largest c     w = scale s_idx (/ sum s_idx)
//
// The choice is the one that fp64 arithmetic makes. That is dear for every
// expert and, with fp32 logits, needed for few tokens: the fast kernel scores in
// fp32, with a bound on its error, and a token in which two values that decide
// something lie closer than the bound is chosen again by the exact routine. Equal
// values count as close, though the keys order them already, so the time depends on
// the data: with 16-bit logits and a bias that is the same for all experts (normal
// logits of deviation 1.5, 8 of 256) 37% of the tokens hold equal values in bf16, 5% in
// fp16. 16384 tokens, us, with a bias of random values and with one of zeros: 8 of 256
// experts in eight groups, fp32 13.7 and 13.7, bf16 14.4 and 29.7, fp16 13.0 and 18.4;
// without groups 10.8 and 10.7, 10.9 and 24.5, 11.0 and 16.4; 6 of 64 in bf16 5.9 and
// 13.2.
//
// The weights are fp32 functions of the chosen logits, computed so that they
// neither overflow nor vanish together: a softmax over the chosen logits, or
// sigmoids with a common factor where all of them are small.
//
// Bound by instructions, not by the 19 MB that 16384 tokens of 256 experts have
// to move (4 us): 16384 x 256 in eight groups with a bias 13-14 us (44 when every token
// is chosen in fp64), without groups and bias 6; one token 4.3 and 2.7 us, of which
// 2.4 are the launch. A workgroup takes 16 or 32 tokens and ends: with a loop over
// more of them the compiler kept the loop's constants in 249 registers a lane, not
// 105, and the first case took 25 us.
#include "ragged_device.hpp"
#include "router.hpp"

namespace moe {
namespace {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ bool no_number(float l) { return !(l > -INFINITY); }  // -inf, NaN

template <typename T>
__device__ __forceinline__ float load_f32(const T* p) {
  return to_f32(*p);
}
// Element i of an array of type t.
__device__ __forceinline__ float load_as(const void* p, ElemType t, int64_t i) {
  if (t == ElemType::kF32) return static_cast<const float*>(p)[i];
  if (t == ElemType::kBF16) return to_f32(static_cast<const bf16*>(p)[i]);
  return to_f32(static_cast<const f16*>(p)[i]);
}

// The value of another lane of the segment: step x pairs lanes at xor distance 1
// and 2, then mirrored in eights and sixteens (whose fours, and eights, hold the
// same value by then), then at xor distance 16 and 32.
template <int x>
__device__ __forceinline__ int other_lane(int v) {
  if constexpr (x == 1) return __builtin_amdgcn_mov_dpp(v, 0xb1, 0xf, 0xf, true);
  else if constexpr (x == 2) return __builtin_amdgcn_mov_dpp(v, 0x4e, 0xf, 0xf, true);
  else if constexpr (x == 4) return __builtin_amdgcn_mov_dpp(v, 0x141, 0xf, 0xf, true);
  else if constexpr (x == 8) return __builtin_amdgcn_mov_dpp(v, 0x140, 0xf, 0xf, true);
  else return __shfl_xor(v, x);
}
template <int x>
__device__ __forceinline__ float other_lane(float v) {
  return __builtin_bit_cast(float, other_lane<x>(__builtin_bit_cast(int, v)));
}
template <int x>
__device__ __forceinline__ double other_lane(double v) {
  const u32x2 b = __builtin_bit_cast(u32x2, v);
  const u32x2 o = {(uint32_t)other_lane<x>((int)b[0]), (uint32_t)other_lane<x>((int)b[1])};
  return __builtin_bit_cast(double, o);
}
// f(value, other lane's value) over the kLanes neighbouring lanes of a segment;
// every lane ends with the same bits (f is commutative).
template <int kLanes, int x = 1, typename V, typename F>
__device__ __forceinline__ V over_segment(V v, F f) {
  if constexpr (x < kLanes) return over_segment<kLanes, 2 * x>(f(v, other_lane<x>(v)), f);
  else return v;
}
template <int kLanes>
__device__ __forceinline__ float seg_max(float v) {
  return over_segment<kLanes>(v, [](float a, float b) { return fmaxf(a, b); });
}
template <int kLanes, typename V>
__device__ __forceinline__ V seg_sum(V v) {
  return over_segment<kLanes>(v, [](V a, V b) { return a + b; });
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

__device__ __forceinline__ double read_lane(double v, int lane) {
  const u32x2 b = __builtin_bit_cast(u32x2, v);
  const u32x2 o = {(uint32_t)__builtin_amdgcn_readlane((int)b[0], lane),
                   (uint32_t)__builtin_amdgcn_readlane((int)b[1], lane)};
  return __builtin_bit_cast(double, o);
}
__device__ __forceinline__ void take_first(double& v, int& at, double ov, int oa) {
  const bool take = (ov > v) | ((ov == v) & (oa < at));
  v = take ? ov : v;
  at = take ? oa : at;
}
// The larger value of the wavefront, and of equal ones that of the lower index:
// over rows of 16 lanes by DPP, over the four rows by lane reads.
template <int x = 1>
__device__ __forceinline__ void first_of_wave(double& v, int& at) {
  if constexpr (x < 16) {
    take_first(v, at, other_lane<x>(v), other_lane<x>(at));
    first_of_wave<2 * x>(v, at);
  } else {
    double w[4];
    int a[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      w[r] = read_lane(v, 16 * r);
      a[r] = __builtin_amdgcn_readlane(at, 16 * r);
    }
    take_first(w[0], a[0], w[1], a[1]);
    take_first(w[2], a[2], w[3], a[3]);
    take_first(w[0], a[0], w[2], a[2]);
    v = w[0];
    at = a[0];
  }
}

// The group of expert e: e / per_group by the factor 2^20 / per_group, rounded up
// (exact for e < 1024: the excess is below e 2^-20 < 1 / per_group).
__device__ __forceinline__ int group_of(const RouterParams& p, int e) {
  return (int)((uint32_t)e * (uint32_t)p.group_factor >> 20);
}

// A wavefront's logits of token t, lane l's experts l + 64 m; -inf past E.
template <typename T, int M>
__device__ __forceinline__ void load_wave(const RouterParams& p, int64_t t, int lane,
                                          float (&l)[M]) {
  const T* row = static_cast<const T*>(p.logits) + t * p.ld;
  T v[M];
#pragma unroll
  for (int m = 0; m < M; ++m) {
    const int e = lane + kWave * m;
    v[m] = row[e < p.E ? e : p.E - 1];
  }
#pragma unroll
  for (int m = 0; m < M; ++m) l[m] = lane + kWave * m < p.E ? to_f32(v[m]) : -INFINITY;
}

// A token's choice in fp64, by one wavefront. Lane l holds experts l + 64 m.
// `c` is the wavefront's share of LDS, E doubles (used with groups). `least`: a
// bound below the k-th choice, -inf if none is known; where few experts reach it,
// each is placed by the number of them before it, which costs a few instructions
// an expert; otherwise the wavefront finds its largest k times.
template <int M>
__device__ __forceinline__ void route_exact(const RouterParams& p, int64_t t, double* c,
                                            double least) {
  const int lane = threadIdx.x & (kWave - 1);
  float l[M], b[M];
  if (p.type == ElemType::kF32) load_wave<float, M>(p, t, lane, l);
  else if (p.type == ElemType::kBF16) load_wave<bf16, M>(p, t, lane, l);
  else load_wave<f16, M>(p, t, lane, l);
  if (p.bias)
#pragma unroll
    for (int m = 0; m < M; ++m) {
      const int e = lane + kWave * m;
      b[m] = p.bias[e < p.E ? e : p.E - 1];
    }
  float top = -INFINITY;
#pragma unroll
  for (int m = 0; m < M; ++m)
    if (!no_number(l[m])) top = fmaxf(top, l[m]);
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
    sum = seg_sum<kWave>(sum);
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
    open |= (uint32_t)(lane + kWave * m < p.E) << m;
    if (p.bias) s[m] += (double)b[m];
    if (no_number(l[m]) || !(s[m] == s[m])) s[m] = -INFINITY;
  }
  if (p.groups > 1) {
#pragma unroll
    for (int m = 0; m < M; ++m)
      if (lane + kWave * m < p.E) c[lane + kWave * m] = s[m];
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    // a group by 64 / (groups, up to a power of two) lanes
    const int log_share = 6 - (32 - __builtin_clz(p.groups - 1)), share = 1 << log_share;
    const int id = lane >> log_share;
    double first = -INFINITY, second = -INFINITY;
    if (id < p.groups) {
      const double* mine = c + id * p.per_group;
      for (int i = lane & (share - 1); i < p.per_group; i += 4 * share) {
        double v[4];
#pragma unroll
        for (int u = 0; u < 4; ++u)
          v[u] = mine[i + u * share < p.per_group ? i + u * share : i];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const double x = i + u * share < p.per_group ? v[u] : -INFINITY;
          second = x > first ? first : (x > second ? x : second);
          first = x > first ? x : first;
        }
      }
    }
    for (int x = 1; x < share; x <<= 1) {
      const double f = __shfl_xor(first, x), o = __shfl_xor(second, x);
      const double less = f > first ? first : f;
      first = f > first ? f : first;
      second = o > second ? o : second;
      second = less > second ? less : second;
    }
    double g = p.group_top == 2 && p.per_group > 1 ? first + second : first;
    if (!(g == g)) g = -INFINITY;
    int ahead = 0;  // groups that come before this lane's
    for (int q = 0; q < p.groups; ++q) {
      const double o = read_lane(g, q << log_share);
      ahead += (o > g) | ((o == g) & (q < id));
    }
    const uint64_t keep = __builtin_amdgcn_ballot_w64(id < p.groups && ahead < p.top_groups);
#pragma unroll
    for (int m = 0; m < M; ++m) {
      const int at = group_of(p, lane + kWave * m) << log_share;
      if (!((keep >> (at & 63)) & 1)) open &= ~(1u << m);
    }
    __builtin_amdgcn_wave_barrier();
  }
  // without a bias experts rank by their logits
  if (!p.bias)
#pragma unroll
    for (int m = 0; m < M; ++m) s[m] = no_number(l[m]) ? -INFINITY : (double)l[m];

  float mine = 0.f;
  int chosen = 0;
  uint64_t reach[M];
  int reached = 0;
#pragma unroll
  for (int m = 0; m < M; ++m) {
    reach[m] = __builtin_amdgcn_ballot_w64(((open >> m) & 1) != 0 && s[m] >= least);
    reached += __builtin_popcountll(reach[m]);
  }
  if (least > -INFINITY && reached >= p.k && reached <= 2 * p.k) {
    int before[M];
#pragma unroll
    for (int m = 0; m < M; ++m) before[m] = 0;
#pragma unroll
    for (int h = 0; h < M; ++h)
      for (uint64_t left = reach[h]; left; left &= left - 1) {
        const int from = __builtin_ctzll(left);
        const double v = read_lane(s[h], from);
#pragma unroll
        for (int m = 0; m < M; ++m)
          before[m] +=
              (v > s[m]) | ((v == s[m]) & (from + kWave * h < lane + kWave * m));
      }
#pragma unroll
    for (int h = 0; h < M; ++h)
      for (uint64_t left = reach[h]; left; left &= left - 1) {
        const int from = __builtin_ctzll(left);
        const float v = __builtin_bit_cast(
            float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, l[h]), from));
        const bool here = lane == __builtin_amdgcn_readlane(before[h], from);
        mine = here ? v : mine;
        chosen = here ? from + kWave * h : chosen;
      }
  } else {
    for (int j = 0; j < p.k; ++j) {
      double v = -INFINITY;
      int at = 0x7fffffff;
#pragma unroll
      for (int m = 0; m < M; ++m)
        if ((open >> m) & 1 && (at == 0x7fffffff || s[m] > v)) {
          v = s[m];
          at = lane + kWave * m;
        }
      first_of_wave(v, at);
      // its logit, from the lane that holds it
      float lv = 0.f;
#pragma unroll
      for (int m = 0; m < M; ++m)
        if (at == lane + kWave * m) {
          lv = l[m];
          open &= ~(1u << m);
        }
      lv = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, lv),
                                                               at & (kWave - 1)));
      if (lane == j) {
        mine = lv;
        chosen = at;
      }
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

template <int M>
__global__ __launch_bounds__(256) void router_exact_kernel(RouterParams p) {
  __shared__ double c[4][kWave * M];
  const int wave = threadIdx.x / kWave;
  const int64_t t = (int64_t)blockIdx.x * 4 + wave;
  if (t < p.T) route_exact<M>(p, t, c[wave], -INFINITY);
}

// M logits of a token from expert e0 on; those from E on are any of the row's.
template <typename T, int M>
__device__ __forceinline__ void load_logits(const RouterParams& p, int64_t t, int e0,
                                            float (&l)[M]) {
  constexpr int V = 16 / sizeof(T);
  const T* row = static_cast<const T*>(p.logits) + t * p.ld;
  if constexpr (M % V == 0) {
    if (p.vec) {  // whole vectors: E is a multiple of V
      union {
        T e[V];
        u32x4 v;
      } r[M / V];
#pragma unroll
      for (int c = 0; c < M / V; ++c) {
        const int e = e0 + c * V;
        r[c].v = *reinterpret_cast<const u32x4*>(row + (e < p.E ? e : p.E - V));
      }
#pragma unroll
      for (int m = 0; m < M; ++m) l[m] = to_f32(r[m / V].e[m % V]);
      return;
    }
  }
#pragma unroll
  for (int m = 0; m < M; ++m) {
    const int e = e0 + m;
    l[m] = to_f32(row[e < p.E ? e : p.E - 1]);
  }
}

// Where expert e's choice lies in LDS: one word in 32 is skipped, against bank
// conflicts of the lanes that walk neighbouring groups.
__host__ __device__ constexpr int choice_at(int e) { return e + e / 32; }

// Larger and smaller of two keys (never NaN).
__device__ __forceinline__ void order_keys(double& a, double& b) {
  const double hi = __builtin_fmax(a, b), lo = __builtin_fmin(a, b);
  a = hi;
  b = lo;
}
// A bitonic list of K keys, into descending order.
template <int K>
__device__ __forceinline__ void sort_bitonic(double* v) {
#pragma unroll
  for (int s = K / 2; s > 0; s >>= 1)
#pragma unroll
    for (int i = 0; i < K; ++i)
      if ((i & s) == 0) order_keys(v[i], v[i + s]);
}
// K keys in any order.
template <int K>
__device__ __forceinline__ void sort_keys(double* v) {
  if constexpr (K > 1) {
    sort_keys<K / 2>(v);
    sort_keys<K / 2>(v + K / 2);
    // first half descending, second read backwards: compare across, then both
    // halves are bitonic
#pragma unroll
    for (int i = 0; i < K / 2; ++i) order_keys(v[i], v[K - 1 - i]);
    sort_bitonic<K / 2>(v);
    sort_bitonic<K / 2>(v + K / 2);
  }
}
// The K best of two descending lists, into a.
template <int K>
__device__ __forceinline__ void merge_keys(double (&a)[K], const double (&b)[K]) {
#pragma unroll
  for (int i = 0; i < K; ++i) a[i] = __builtin_fmax(a[i], b[K - 1 - i]);
  sort_bitonic<K>(a);
}
template <int kLanes, int K, int x = 1>
__device__ __forceinline__ void merge_segment(double (&a)[K]) {
  if constexpr (x < kLanes) {
    double b[K];
#pragma unroll
    for (int i = 0; i < K; ++i) b[i] = other_lane<x>(a[i]);
    merge_keys<K>(a, b);
    merge_segment<kLanes, K, 2 * x>(a);
  }
}

// An expert's key: its value, with the low bits of the fp64 mantissa (which fp32
// values leave empty) telling equal ones apart, the lower index first. One
// v_max_f64 then compares value and index. Values end at fp32's largest: a token
// that chooses one there is chosen again.
constexpr float kMost = 0x1.fffffep127f;
__device__ __forceinline__ double key_of(float v, int e) {
  u32x2 b = __builtin_bit_cast(u32x2, (double)__builtin_amdgcn_fmed3f(v + 0.f, -kMost, kMost));
  b[0] |= (uint32_t)e ^ (~(uint32_t)((int32_t)b[1] >> 31) & 1023u);  // e, or 1023 - e
  return __builtin_bit_cast(double, b);
}
__device__ __forceinline__ int expert_of(double key) {
  const u32x2 b = __builtin_bit_cast(u32x2, key);
  return (int)((b[0] ^ ~(uint32_t)((int32_t)b[1] >> 31)) & 1023u);
}

// The best two of the lanes of a group (1, 2, 4, 8 or 16 neighbours).
template <int x>
__device__ __forceinline__ void merge_two(float& first, float& second, int lanes) {
  if constexpr (x < 16) {
    if (x < lanes) {
      const float f = other_lane<x>(first), s = other_lane<x>(second);
      second = fmaxf(fminf(first, f), fmaxf(second, s));
      first = fmaxf(first, f);
    }
    merge_two<2 * x>(first, second, lanes);
  }
}

constexpr float kLog2e = 1.44269504088896341f;
constexpr int kGroupStep = 4;  // choices that a group's lane reads at once

// kLanes lanes a token, lane q holding experts q M .. q M + M - 1, k <= K. Each
// lane sorts its K best keys, and exchanges with the lanes of its segment merge
// them. Groups (16 lanes): where a group's experts are whole lanes their best two
// are merged like that, otherwise a lane a group reads them from LDS; rotations of
// the lanes count the groups before each. kScored: there is a bias or there are
// groups; otherwise experts rank by their logits alone.
//
// Scores are fp32, by the hardware's base-2 exponential and reciprocal (an ulp
// each). They are off by at most tol = 2^-24 (A pmax + |c|): a sigmoid by A = 8 (4
// by its steps: l log2 e is off by |l| 2^-23 and s (1 - s) |l| < 0.23), a softmax
// of M values a lane by A = 2 (M + 16) of its largest score; the sum with the bias
// by one of c. Where two chosen values, the last chosen and another, or two groups
// lie within the sum of their errors, the token goes to route_exact. Without a
// bias keys are the logits themselves.
//
// What cannot be chosen (masked, of a group left out, past E) is -inf; a token
// whose last choice is that low is chosen again too. The code has no branch an
// expert: conditions are selects.
template <int kLanes, int M, int K, bool kScored>
__global__ __launch_bounds__(256) void router_kernel(RouterParams p) {
  static_assert(K <= kLanes && kLanes <= 16, "a chosen expert a lane; DPP rows");
  constexpr int EP = kLanes * M, kTokens = 256 / kLanes;
  constexpr int kRow = choice_at(EP);
  extern __shared__ float choices[];  // with groups: [kTokens][kRow]
  const int q = threadIdx.x % kLanes, seg = threadIdx.x / kLanes, e0 = q * M;
  const bool biased = kScored && p.bias != nullptr;
  const int64_t t = (int64_t)blockIdx.x * kTokens + seg;
  const bool live = t < p.T;
  float l[M];
  if (p.type == ElemType::kF32) load_logits<float, M>(p, live ? t : 0, e0, l);
  else if (p.type == ElemType::kBF16) load_logits<bf16, M>(p, live ? t : 0, e0, l);
  else load_logits<f16, M>(p, live ? t : 0, e0, l);
  if (p.E < EP)
#pragma unroll
    for (int m = 0; m < M; ++m) l[m] = e0 + m < p.E ? l[m] : -INFINITY;

  float top = -INFINITY, sum = 0.f, c[M];
  float worst = 8.f;  // A pmax
  if (!p.sigmoid && (kScored || !p.renormalize)) {
#pragma unroll
    for (int m = 0; m < M; ++m) {
      l[m] = l[m] > -INFINITY ? l[m] : -INFINITY;  // NaN
      top = fmaxf(top, l[m]);
    }
    top = seg_max<kLanes>(top);
#pragma unroll
    for (int m = 0; m < M; ++m) {
      const float d = l[m] == top ? 0.f : l[m] - top;
      c[m] = __builtin_amdgcn_exp2f((l[m] > -INFINITY ? d : -INFINITY) * kLog2e);
      sum += c[m];
    }
    sum = seg_sum<kLanes>(sum);
    const float inv = sum > 0.f ? 1.f / sum : 0.f;
#pragma unroll
    for (int m = 0; m < M; ++m) c[m] *= inv;
    worst = (float)(2 * (M + 16)) * inv;
  }
  // what the choice goes by
  bool unsure = false;
  if constexpr (kScored) {
    if (p.sigmoid)
#pragma unroll
      for (int m = 0; m < M; ++m)
        c[m] = __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-kLog2e * l[m]));
    if (biased) {
      float b[M];
      if (M % 4 == 0 && p.bias_vec) {
#pragma unroll
        for (int m = 0; m < M; m += 4) {
          const float4 f = *reinterpret_cast<const float4*>(
              p.bias + (uint32_t)(e0 + m < p.E ? e0 + m : p.E - 4));
          b[m] = f.x;
          b[m + 1] = f.y;
          b[m + 2] = f.z;
          b[m + 3] = f.w;
        }
      } else {
#pragma unroll
        for (int m = 0; m < M; ++m) b[m] = p.bias[(uint32_t)(e0 + m < p.E ? e0 + m : p.E - 1)];
      }
#pragma unroll
      for (int m = 0; m < M; ++m) c[m] += b[m];
    }
#pragma unroll
    for (int m = 0; m < M; ++m) c[m] = l[m] > -INFINITY ? c[m] : -INFINITY;
  }
  if constexpr (kScored && kLanes == 16) {
    if (p.groups > 1) {
      // (a NaN among c leaves both as they are)
      float first = -INFINITY, second = -INFINITY;
      bool is_group;
      int id, share = 1;  // this lane's group, and the lanes that hold it
      if (p.lanes_per_group) {
#pragma unroll
        for (int m = 0; m < M; ++m) {
          second = __builtin_amdgcn_fmed3f(first, second, c[m]);
          first = fmaxf(first, c[m]);
        }
        merge_two<1>(first, second, p.lanes_per_group);
        share = p.lanes_per_group;
        id = q / share;
        is_group = e0 < p.E;
      } else {
        float* mine = choices + seg * kRow;
#pragma unroll
        for (int m = 0; m < M; ++m) mine[choice_at(e0 + m)] = c[m];
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        id = q;
        is_group = q < p.groups;
        for (int i = 0; i < p.per_group; i += kGroupStep) {
          float v[kGroupStep];
#pragma unroll
          for (int u = 0; u < kGroupStep; ++u) {
            const int e = q * p.per_group + i + u;
            v[u] = mine[choice_at(e < EP ? e : EP - 1)];
          }
#pragma unroll
          for (int u = 0; u < kGroupStep; ++u) {
            const float x = i + u < p.per_group ? v[u] : -INFINITY;
            second = __builtin_amdgcn_fmed3f(first, second, x);
            first = fmaxf(first, x);
          }
        }
      }
      const float g = p.group_top == 2 && p.per_group > 1 ? first + second : first;
      unsure = is_group & !(g == g);
      // two groups' sums of two choices each
      const float big = seg_max<kLanes>(
          is_group & (fabsf(g) < INFINITY) ? fmaxf(fabsf(first), fabsf(second)) : 0.f);
      const float near = 0x1p-24f * (4.f * worst + 16.f * big);
      // groups before this lane's, by rotations of the 16 lanes by multiples of
      // a group's lanes; a lane of no group holds -inf and an id behind all
      const float mark = is_group ? g : -INFINITY;
      const int name = is_group ? id : 64;
      int ahead = 0;
#define MOE_TURN(n)                                                                           \
{                                                                                           \
  const float v = __builtin_bit_cast(                                                       \
      float,                                                                                \
      __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, mark), 0x120 + n, 0xf, 0xf, true));  \
  const int o = __builtin_amdgcn_mov_dpp(name, 0x120 + n, 0xf, 0xf, true);                  \
  ahead += (v > mark) | ((v == mark) & (o < name));                                         \
  unsure |= (o != name) & (fabsf(v - mark) <= near);                                        \
}
      if (share == 1) {
        MOE_TURN(1) MOE_TURN(3) MOE_TURN(5) MOE_TURN(7) MOE_TURN(9) MOE_TURN(11) MOE_TURN(13)
        MOE_TURN(15)
      }
      if (share <= 2) { MOE_TURN(2) MOE_TURN(6) MOE_TURN(10) MOE_TURN(14) }
      if (share <= 4) { MOE_TURN(4) MOE_TURN(12) }
      if (share <= 8) MOE_TURN(8)
#undef MOE_TURN
      const bool chosen = is_group & (ahead < p.top_groups);
      if (!biased)
#pragma unroll
        for (int m = 0; m < M; ++m) c[m] = l[m];
      if (p.lanes_per_group) {
#pragma unroll
        for (int m = 0; m < M; ++m) c[m] = chosen ? c[m] : -INFINITY;
      } else {
        const uint64_t in = __builtin_amdgcn_ballot_w64(chosen);
        const uint32_t keep = (uint32_t)(in >> (threadIdx.x & 48)) & 0xffffu;
        int group = group_of(p, e0), left = (group + 1) * p.per_group - e0;
#pragma unroll
        for (int m = 0; m < M; ++m) {
          c[m] = ((keep >> (group & 31)) & 1) != 0 ? c[m] : -INFINITY;
          --left;
          group += left == 0;
          left = left == 0 ? p.per_group : left;
        }
      }
    }
  }
  double best[K];
  {
    // each lane's K best: blocks of K sorted and merged
    constexpr int kBlocks = (M + K - 1) / K;
#pragma unroll
    for (int b = 0; b < kBlocks; ++b) {
      double v[K];
#pragma unroll
      for (int i = 0; i < K; ++i) {
        const int m = b * K + i;
        v[i] = -INFINITY;
        if (m < M) v[i] = key_of(kScored ? c[m] : l[m], e0 + m);
      }
      sort_keys<K>(v);
      if (b == 0)
#pragma unroll
        for (int i = 0; i < K; ++i) best[i] = v[i];
      else
        merge_keys<K>(best, v);
    }
  }
  merge_segment<kLanes, K>(best);
  double mine = best[0], last = best[0];
#pragma unroll
  for (int j = 1; j < K; ++j) {
    last = j == p.k - 1 ? best[j] : last;
    mine = q == j ? best[j] : mine;
  }
  const bool use = q < p.k;
  const int e = use ? expert_of(mine) : 0;
  const float le =
      live && use ? load_as(p.logits, p.type, t * p.ld + (e < p.E ? e : 0)) : -INFINITY;
  // (an end's own value, index bits and all, is at least that far out)
  unsure |= !(last > -(double)kMost) | !(best[0] < (double)kMost);
  float least = (float)last;  // of the k-th choice
  if (biased) {
    const float c1 = (float)best[0];
    const float near = 0x1p-24f * (2.f * worst + 4.f * fmaxf(fabsf(least), fabsf(c1)));
#pragma unroll
    for (int j = 0; j + 1 < K; ++j)
      if (j + 1 < p.k) unsure |= !(best[j] - best[j + 1] > (double)near);
    least -= near;
    int over = 0;
#pragma unroll
    for (int m = 0; m < M; ++m) over += c[m] >= least;
    unsure |= seg_sum<kLanes>(over) != p.k;
  }
  const float w = weight_of<kLanes>(le, use, top, sum, p.sigmoid, p.renormalize, p.scale);
  if (live && use) {
    p.idx[t * p.k + q] = e;
    p.weight[t * p.k + q] = w;
  }
  // tokens to choose again: one wavefront each
  uint64_t again = __builtin_amdgcn_ballot_w64(live && unsure);
  double* share = reinterpret_cast<double*>(
      choices + (threadIdx.x / kWave) * (kWave / kLanes) * kRow);
  while (again) {
    const int at = __builtin_ctzll(again) / kLanes;  // a segment of the wavefront
    again &= ~(((1ull << (kLanes - 1) << 1) - 1) << (at * kLanes));
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    const float from = __builtin_bit_cast(
        float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, least), at * kLanes));
    route_exact<(EP + kWave - 1) / kWave>(
        p, (int64_t)blockIdx.x * kTokens + (threadIdx.x / kWave) * (kWave / kLanes) + at, share,
        from > -kMost ? (double)from : -INFINITY);
  }
}

// launch(p, grid) over ranges of the tokens: a grid has at most 2^32 threads.
template <typename F>
hipError_t in_grids(RouterParams p, int tokens, F launch) {
  const int64_t T = p.T, most = (int64_t)tokens << 23;
  for (int64_t t0 = 0; t0 < T; t0 += most) {
    p.T = T - t0 < most ? T - t0 : most;
    launch(p, dim3((unsigned)((p.T + tokens - 1) / tokens)));
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    p.logits = static_cast<const char*>(p.logits) + p.T * p.ld * elem_bytes(p.type);
    p.idx += p.T * p.k;
    p.weight += p.T * p.k;
  }
  return hipSuccess;
}

// kScored: with a bias or groups too.
template <int kLanes, int M, bool kScored = true>
hipError_t route_lanes(RouterParams p, hipStream_t st) {
  constexpr int kTokens = 256 / kLanes;
  // the lanes of a group, where they hold nothing else
  p.lanes_per_group = 0;
  if (p.groups > 1 && p.per_group % M == 0) {
    const int lanes = p.per_group / M;
    if ((lanes & (lanes - 1)) == 0 && lanes <= 16) p.lanes_per_group = lanes;
  }
  const size_t lds = p.groups > 1 ? sizeof(float) * kTokens * choice_at(kLanes * M) : 0;
  const bool scored = kScored && (p.bias || p.groups > 1);
  return in_grids(p, kTokens, [&](const RouterParams& p, dim3 grid) {
// (few choices of few experts without either are 8 lanes')
#define MOE_ROUTE(K)                                                                         \
  if (scored)                                                                                \
    hipLaunchKernelGGL((router_kernel<kLanes, M, K, kScored>), grid, dim3(256), lds, st, p); \
  else if constexpr (K > 8 || kLanes == 8 || M >= 16)                                        \
    hipLaunchKernelGGL((router_kernel<kLanes, M, K, false>), grid, dim3(256), lds, st, p)
    if (p.k <= 4) {
      MOE_ROUTE(4);
    } else if (kLanes == 8 || p.k <= 8) {
      MOE_ROUTE(8);
    } else {
      MOE_ROUTE(kLanes);
    }
#undef MOE_ROUTE
  });
}

// The fast kernel takes up to 16 of up to 512 experts with up to 16 groups (with
// neither bias nor groups, of up to 1024); the exact one, a wavefront a token, takes
// the rest. In us, fast and exact: 16384 tokens, 9 of 256 experts 8.2 and 38, with a
// bias 13 and 38, and groups 17 and 44; 16 of 512 with a bias 34 and 91; 8 of 1024 26
// and 104. More than 512 experts with a bias go to the exact one at every number of
// tokens, which is the slower one for many: 16384 tokens 67 and 91-105, one 14.5 and
// 10.4 (1024 tokens by the exact one 13.6). Eight lanes a token
// or sixteen, without groups: 65536 tokens, 6 of 64 experts 7.3 and 12, 8 of 128 9.6
// and 13.6, 4 of 256 15.3 and 14.5.
hipError_t route(const RouterParams& p, hipStream_t st) {
  if (p.groups == 1 && p.k <= 8) {
    if (p.E <= 16) return route_lanes<8, 2>(p, st);
    if (p.E <= 32) return route_lanes<8, 4>(p, st);
    if (p.E <= 64) return route_lanes<8, 8>(p, st);
    if (p.E <= 128) return route_lanes<8, 16>(p, st);
  }
  if (p.k <= 16 && p.groups <= 16) {
    if (p.E <= 64) return route_lanes<16, 4>(p, st);
    if (p.E <= 128) return route_lanes<16, 8>(p, st);
    if (p.E <= 256) return route_lanes<16, 16>(p, st);
    if (p.E <= 512) return route_lanes<16, 32>(p, st);
    if (p.groups == 1 && !p.bias) return route_lanes<16, 64, false>(p, st);
  }
  return in_grids(p, 4, [&](const RouterParams& p, dim3 grid) {
#define MOE_EXACT(M) hipLaunchKernelGGL((router_exact_kernel<M>), grid, dim3(256), 0, st, p)
    if (p.E <= 64) MOE_EXACT(1);
    else if (p.E <= 128) MOE_EXACT(2);
    else if (p.E <= 256) MOE_EXACT(4);
    else if (p.E <= 512) MOE_EXACT(8);
    else MOE_EXACT(16);
#undef MOE_EXACT
  });
}

// ---------------------------------------------------------------- gradient
// With w_j = scale s_j (/ sum), g_j = scale dweight_j over the chosen j:
//   softmax, renormalised   dl_j = w_j (g_j - sum w g)      (w: without scale)
//   sigmoid, renormalised   dl_j = w_j (g_j - sum w g) (1 - s_j)
//   sigmoid                 dl_j = s_j (1 - s_j) g_j
//   softmax                 dl_e = s_e (g_e - sum s g)      for every expert
// kLanes lanes a token, all of one wavefront. What the chosen experts get is added to
// a row of zeros in LDS; then every lane writes its experts' gradients, whole rows at
// once. With the softmax over all experts (kHeld > 0) a lane keeps its first kHeld
// vectors of the row, and of their exponentials. 16384 tokens of 64 experts, 6 chosen, full softmax,
// fp32: 4.3 us for 9.2 MB (1.8 us at a copy's rate, 2.5 the launch; 6.2 with the row
// read three times and the choices compared with every expert). Wide rows are bound by
// instructions: 65536 of 1024 in bf16, full softmax, 91 us for 268 MB (53 at a copy's
// rate), 711 vector instructions a token, the exponentials and the row in LDS, which
// keep the vector units busy 98% of the cycles.
constexpr int kGradTokens = 32;  // of a workgroup at most

template <typename T, int kLanes, bool kVec, int kHeld>
__global__ __launch_bounds__(256) void router_grad_kernel(RouterGradParams p) {
  constexpr int V = kVec ? 16 / sizeof(T) : 1;
  constexpr int kTokens = 256 / kLanes;
  constexpr bool kFull = kHeld > 0;
  static_assert(kTokens <= kGradTokens, "share of LDS");
  __shared__ float val[kTokens][kRouterMaxTopK];
  extern __shared__ float rows[];  // [kTokens][E]
  const int q = threadIdx.x % kLanes, seg = threadIdx.x / kLanes;
  const int64_t steps = (p.T + kTokens - 1) / kTokens;
  for (int64_t step = blockIdx.x; step < steps; step += gridDim.x) {
    const int64_t t = step * kTokens + seg;
    const bool live = t < p.T;
    const T* row = static_cast<const T*>(p.logits) + (live ? t : 0) * p.ld;
    T* out = static_cast<T*>(p.dlogits) + (live ? t : 0) * p.ld;
    // what comes from memory first, all at once: this lane's choice and its values
    // of the row (experts own(h, i))
    int own_e = -1;
    float own_g = 0.f;
    if (live && q < p.k) {
      own_e = p.idx[t * p.k + q];
      own_g = p.scale * p.dweight[t * p.k + q];
    }
    auto order = [] {  // (a token's lanes are of one wavefront)
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
    };
    auto choice = [&](int j) { return j == q ? own_e : p.idx[t * p.k + j]; };
    auto gradient = [&](int j) { return j == q ? own_g : p.scale * p.dweight[t * p.k + j]; };
    auto own = [&](int h, int i) { return (h * kLanes + q) * V + i; };
    float s[kHeld > 0 ? kHeld : 1][V];
    float top = -INFINITY, inv = 0.f;
    // the softmax over all experts
    if constexpr (kFull) {
#pragma unroll
      for (int h = 0; h < kHeld; ++h) {
        if (kVec && live && own(h, V) <= p.E) {
          union {
            T e[V];
            u32x4 v;
          } r;
          r.v = *reinterpret_cast<const u32x4*>(row + own(h, 0));
#pragma unroll
          for (int i = 0; i < V; ++i) s[h][i] = to_f32(r.e[i]);
        } else {
#pragma unroll
          for (int i = 0; i < V; ++i)
            s[h][i] = live && own(h, i) < p.E ? load_f32(row + own(h, i)) : -INFINITY;
        }
      }
#pragma unroll
      for (int h = 0; h < kHeld; ++h)
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (!no_number(s[h][i])) top = fmaxf(top, s[h][i]);
      if (live)
        for (int e = kHeld * kLanes * V + q; e < p.E; e += kLanes) {
          const float l = load_f32(row + e);
          if (!no_number(l)) top = fmaxf(top, l);
        }
      top = seg_max<kLanes>(top);
      float sum = 0.f;
#pragma unroll
      for (int h = 0; h < kHeld; ++h)
#pragma unroll
        for (int i = 0; i < V; ++i) {
          s[h][i] = exp_below(s[h][i], top);
          sum += s[h][i];
        }
      if (live)
        for (int e = kHeld * kLanes * V + q; e < p.E; e += kLanes)
          sum += exp_below(load_f32(row + e), top);
      sum = seg_sum<kLanes>(sum);
      inv = sum > 0.f ? 1.f / sum : 0.f;
    } else if (p.renormalize) {
      if (live)
        for (int j = q; j < p.k; j += kLanes) {
          const int e = choice(j);
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
        const int e = choice(j);
        const bool in = e >= 0 && e < p.E;
        const float l = in ? load_f32(row + e) : -INFINITY;
        const float g = gradient(j);
        float c;
        if (kFull) c = exp_below(l, top) * inv;
        else if (!p.sigmoid) c = exp_below(l, top);
        else c = sigmoid_above(l, p.renormalize ? top : 0.f);
        sum += c;
        dot += c > 0.f ? c * g : 0.f;
        val[seg][j] = c;
      }
    float* mine = rows + seg * p.E;
    for (int e = q; e < p.E; e += kLanes) mine[e] = 0.f;
    order();
    sum = seg_sum<kLanes>(sum);
    dot = seg_sum<kLanes>(dot);
    if (p.renormalize) dot = sum > 0.f ? dot / sum : 0.f;
    if (live)
      for (int j = q; j < p.k; j += kLanes) {
        const float c = val[seg][j];
        const float g = gradient(j);
        const int e = choice(j);
        const bool in = e >= 0 && e < p.E;
        float v = g;
        if (!kFull) {
          const float l = in ? load_f32(row + e) : -INFINITY;
          v = p.renormalize ? c / sum * (g - dot) : c * g;
          // 1 - 1 / (1 + e^-l)
          if (p.sigmoid)
            v *= l >= 0.f ? expf(-l) / (1.f + expf(-l)) : 1.f / (1.f + expf(l));
          if (!(c > 0.f)) v = 0.f;
        }
        if (in) atomicAdd(&mine[e], v);
      }
    order();
    // V experts from e0 on, whose shares before the division are c
    auto write = [&](int e0, const float (&c)[V]) {
      const int n = p.E - e0 < V ? p.E - e0 : V;
      float d[V];
#pragma unroll
      for (int i = 0; i < V; ++i) d[i] = mine[i < n ? e0 + i : e0];
      if (kFull)
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float share = c[i] * inv;
          d[i] = share > 0.f ? share * (d[i] - dot) : 0.f;
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
    };
#pragma unroll
    for (int h = 0; h < kHeld; ++h)
      if (live && own(h, 0) < p.E) write(own(h, 0), s[h]);
    if (live)
      for (int e0 = own(kHeld, 0); e0 < p.E; e0 += kLanes * V) {
        float c[V];
#pragma unroll
        for (int i = 0; i < V; ++i)
          c[i] = kFull && e0 + i < p.E ? exp_below(load_f32(row + e0 + i), top) : 0.f;
        write(e0, c);
      }
    order();
  }
}

template <typename T, int kLanes, int kVectors>
hipError_t grad_lanes(const RouterGradParams& p, int num_cus, hipStream_t st) {
  const int64_t steps = (p.T * kLanes + 255) / 256, most = (int64_t)num_cus * 16;
  const dim3 grid((unsigned)(steps < most ? steps : most));
  const bool full = !p.sigmoid && !p.renormalize;
  const size_t lds = sizeof(float) * (256 / kLanes) * p.E;
#define MOE_GRAD(V, H) \
  hipLaunchKernelGGL((router_grad_kernel<T, kLanes, V, H>), grid, dim3(256), lds, st, p)
  if (p.vec && full) MOE_GRAD(true, kVectors);
  else if (p.vec) MOE_GRAD(true, 0);
  else if (full) MOE_GRAD(false, 4 * kVectors);
  else MOE_GRAD(false, 0);
#undef MOE_GRAD
  return hipGetLastError();
}

// A vector a lane, or four scalars, up to 16 lanes; two of them above (us, by one and
// two: 16384 tokens of 64 experts in fp32 4.4 and 4.8, of 256 10.1 and 7.4, 65536 of
// 1024 in bf16 167 and 92).
template <typename T>
hipError_t grad(const RouterGradParams& p, int num_cus, hipStream_t st) {
  const int per = p.vec ? p.E / (int)(16 / sizeof(T)) : (p.E + 3) / 4;
  if (per <= 8) return grad_lanes<T, 8, 1>(p, num_cus, st);
  if (per <= 16) return grad_lanes<T, 16, 1>(p, num_cus, st);
  if (per <= 32) return grad_lanes<T, 16, 2>(p, num_cus, st);
  if (per <= 64) return grad_lanes<T, 32, 2>(p, num_cus, st);
  return grad_lanes<T, 64, 2>(p, num_cus, st);
}

}  // namespace

hipError_t launch_router(RouterParams p, hipStream_t st) {
  if (p.T == 0) return hipSuccess;
  p.group_factor = ((1 << 20) + p.per_group - 1) / p.per_group;
  return route(p, st);
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
