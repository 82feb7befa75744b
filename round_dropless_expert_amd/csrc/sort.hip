// Assignments into expert order: a stable counting sort of idx [n] by expert.
// Bucket E takes the assignments of no expert; it sorts behind the others.
//
// A chunk of assignments is one workgroup's, split into runs of its
// wavefronts. Every wavefront counts its run per bucket in LDS (a count does
// not depend on the order of its increments); prefixes over buckets, chunks
// and wavefronts give each wavefront's first place in every bucket; then it
// walks its run again, 64 assignments at a time: ballots over the bits of the
// bucket find the lanes with the same bucket, and the number of such lanes
// below is the rank. No atomic decides an order.
//
// Few assignments are one launch of one workgroup; more are a launch that
// counts the chunks and one that places them, in which each workgroup sums
// the counts of the chunks before its own.
//
// Latency: 8 assignments of 256 experts 4.4 us, 32768 (64 experts) 8.3, 131072 (256)
// 10.5 (4 and 9 us the launches, 1.6 MB moved), 524288 17. In one launch and in two:
// 2048 assignments of 64 experts 5.4 and 7.6 us, 4096 7.1 and 8.0, 8192 10.7 and 8.1.
#include "ragged_device.hpp"
#include "router.hpp"

namespace moe {
namespace {

constexpr int kSortWaves = 16;
constexpr int kMaxBuckets = kRaggedMaxExperts + 1;
constexpr int64_t kOneChunk = 4096;   // sorted by one workgroup
constexpr int64_t kChunkLeast = 2048;
constexpr int64_t kMaxChunks = 256;

int64_t chunk_of(int64_t n) {
  const int64_t c = (n + kMaxChunks - 1) / kMaxChunks;
  return c < kChunkLeast ? kChunkLeast : (c + 1023) / 1024 * 1024;
}

__device__ __forceinline__ int bucket_of(const int32_t* idx, int64_t a, int E) {
  const int e = idx[a];
  return e >= 0 && e < E ? e : E;
}

// counts[chunk][E + 1]
__global__ __launch_bounds__(256) void sort_count_kernel(const int32_t* __restrict__ idx,
                                                         int64_t n, int E, int64_t chunk,
                                                         int32_t* __restrict__ counts) {
  __shared__ int h[kMaxBuckets];
  for (int b = threadIdx.x; b <= E; b += 256) h[b] = 0;
  __syncthreads();
  const int64_t first = blockIdx.x * chunk, last = first + chunk < n ? first + chunk : n;
  for (int64_t a = first + threadIdx.x; a < last; a += 256 * 8) {
    int b[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) b[u] = bucket_of(idx, a + u * 256 < last ? a + u * 256 : a, E);
#pragma unroll
    for (int u = 0; u < 8; ++u)
      if (a + u * 256 < last) atomicAdd(&h[b[u]], 1);
  }
  __syncthreads();
  for (int b = threadIdx.x; b <= E; b += 256)
    counts[(int64_t)blockIdx.x * (E + 1) + b] = h[b];
}

// kOne: the only workgroup, which counts for itself.
template <bool kOne>
__global__ __launch_bounds__(1024) void sort_place_kernel(
    const int32_t* __restrict__ idx, int64_t n, int E, int bits, int64_t chunk, int chunks,
    const int32_t* __restrict__ counts, int32_t* __restrict__ perm, int32_t* __restrict__ pos,
    int32_t* __restrict__ offsets) {
  __shared__ int place[kSortWaves][kMaxBuckets];  // counts, then next places
  __shared__ int start[kMaxBuckets];              // totals, then first places
  __shared__ int parts[kSortWaves];
  __shared__ int shared_sum[kOne ? 1 : 1024], shared_pre[kOne ? 1 : 1024];
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
  const int B = E + 1;
  const int64_t first = blockIdx.x * chunk, last = first + chunk < n ? first + chunk : n;
  const int64_t run = (chunk + kSortWaves * kWave - 1) / (kSortWaves * kWave) * kWave;
  const int64_t r0 = first + wave * run, r1 = r0 + run < last ? r0 + run : last;
  for (int b = tid; b < kSortWaves * B; b += 1024) place[b / B][b % B] = 0;
  __syncthreads();
  for (int64_t a = r0 + lane; a < r1; a += kWave) atomicAdd(&place[wave][bucket_of(idx, a, E)], 1);
  __syncthreads();
  // per bucket: the wavefronts' counts become prefixes; the total of all
  // chunks, and of the chunks before this one
  const bool on = tid < B;
  int total = 0, before = 0;
  if (on) {
    int sum = 0;
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) {
      const int c = place[w][tid];
      place[w][tid] = sum;
      sum += c;
    }
    if (kOne) total = sum;
  }
  if constexpr (!kOne) {
    // groups of `width` threads share the chunks; 16 counts of each in flight
    const int width = B <= 128 ? 128 : B <= 256 ? 256 : B <= 512 ? 512 : 1024;
    const int b = tid & (width - 1), group = tid / width, groups = 1024 / width;
    int sum = 0, pre = 0;
    if (b < B) {
      int c = group;
      for (; c + 15 * groups < chunks; c += 16 * groups) {
        int v[16];
#pragma unroll
        for (int u = 0; u < 16; ++u) v[u] = counts[(int64_t)(c + u * groups) * B + b];
#pragma unroll
        for (int u = 0; u < 16; ++u) {
          sum += v[u];
          pre += c + u * groups < (int)blockIdx.x ? v[u] : 0;
        }
      }
      for (; c < chunks; c += groups) {
        const int v = counts[(int64_t)c * B + b];
        sum += v;
        pre += c < (int)blockIdx.x ? v : 0;
      }
    }
    shared_sum[tid] = sum;
    shared_pre[tid] = pre;
    __syncthreads();
    if (on)
      for (int g = 0; g < groups; ++g) {
        total += shared_sum[g * width + tid];
        before += shared_pre[g * width + tid];
      }
  }
  // exclusive prefix over the buckets (1024 of them here, the last one by
  // itself where there are 1025)
  const int incl = wave_inclusive_scan(total);
  if (lane == kWave - 1) parts[wave] = incl;
  __syncthreads();
  int base = 0;
  for (int w = 0; w < wave; ++w) base += parts[w];
  if (on) start[tid] = base + incl - total;
  if (B > 1024 && tid == 1023) start[1024] = base + incl;
  __syncthreads();
  if (blockIdx.x == 0)
    for (int b = tid; b <= E; b += 1024) offsets[b] = start[b];
  // (bucket 1024, of no expert: its prefixes are found here)
  if (B > 1024 && tid == 0) {
    int sum = 0, more = 0;
    for (int w = 0; w < kSortWaves; ++w) {
      const int c = place[w][1024];
      place[w][1024] = sum;
      sum += c;
    }
    if constexpr (!kOne)
      for (int c = 0; c < (int)blockIdx.x; ++c) more += counts[(int64_t)c * B + 1024];
    start[1024] += more;
  }
  __syncthreads();
  if (on) {
    const int s = start[tid] + before;
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) place[w][tid] += s;
  }
  if (B > 1024 && tid < kSortWaves) place[tid][1024] += start[1024];
  __syncthreads();
  const uint64_t below = ~(~0ull << lane);
  for (int64_t a0 = r0; a0 < r1; a0 += kWave) {
    const int64_t a = a0 + lane;
    const bool live = a < r1;
    const int b = live ? bucket_of(idx, a, E) : 0;
    uint64_t same = __builtin_amdgcn_ballot_w64(live);
    for (int bit = 0; bit < bits; ++bit) {
      const bool set = (b >> bit) & 1;
      const uint64_t v = __builtin_amdgcn_ballot_w64(set);
      same &= set ? v : ~v;
    }
    const int rank = __builtin_popcountll(same & below);
    int p = 0;
    if (live) p = place[wave][b] + rank;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    if (live) {
      if (rank == 0) place[wave][b] = p + __builtin_popcountll(same);
      perm[p] = b < E ? (int32_t)a : -1;
      pos[a] = b < E ? p : -1;
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  }
}

__global__ __launch_bounds__(256) void sort_nothing_kernel(int E, int32_t* offsets) {
  for (int b = threadIdx.x; b <= E; b += 256) offsets[b] = 0;
}

}  // namespace

size_t sort_bytes(int64_t n, int E) {
  if (n <= kOneChunk) return 0;
  const int64_t chunk = chunk_of(n);
  return (size_t)((n + chunk - 1) / chunk) * (size_t)(E + 1) * 4;
}

hipError_t launch_sort(int64_t n, int E, const int32_t* idx, int32_t* perm, int32_t* pos,
                       int32_t* offsets, int32_t* counts, hipStream_t st) {
  if (n == 0) {
    hipLaunchKernelGGL(sort_nothing_kernel, dim3(1), dim3(256), 0, st, E, offsets);
    return hipGetLastError();
  }
  int bits = 0;
  while (E >> bits) ++bits;  // buckets 0 .. E
  if (n <= kOneChunk) {
    hipLaunchKernelGGL(sort_place_kernel<true>, dim3(1), dim3(1024), 0, st, idx, n, E, bits, n, 1,
                       nullptr, perm, pos, offsets);
    return hipGetLastError();
  }
  const int64_t chunk = chunk_of(n);
  const int chunks = (int)((n + chunk - 1) / chunk);
  hipLaunchKernelGGL(sort_count_kernel, dim3((unsigned)chunks), dim3(256), 0, st, idx, n, E,
                     chunk, counts);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(sort_place_kernel<false>, dim3((unsigned)chunks), dim3(1024), 0, st, idx, n,
                     E, bits, chunk, chunks, counts, perm, pos, offsets);
  return hipGetLastError();
}

}  // namespace moe
