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
// Latency: 8 assignments of 256 experts 4.0 us, 32768 (64 experts) 7.8, 131072 (256)
// 10.0 (two launches and 1.6 MB moved; every workgroup sums the counts of 64 chunks),
// 524288 15. In one launch and in two: 2048 assignments of 64 experts 4.5 and 6.4 us,
// 4096 5.7 and 6.5.
#include "ragged_device.hpp"
#include "router.hpp"

namespace moe {
namespace {

constexpr int kSortWaves = 16;
constexpr int kMaxBuckets = kRaggedMaxExperts + 1;
constexpr int kHeld = 4;               // rounds of 64 assignments a wavefront keeps
constexpr int64_t kOneChunk = 4096;   // sorted by one workgroup

// 64 chunks while a chunk's assignments are held, then more of those, and at most 256
// (every workgroup reads the counts of all). 256 experts, us, by 64, 128 and 256
// chunks: 131072 assignments 10.0, 11.6, 11.7; 524288 17.5, 15.1, 17.8; 2000000 52, 37,
// 30.
int64_t chunk_of(int64_t n) {
  const int64_t held = (int64_t)kSortWaves * kWave * kHeld;
  int64_t c = (n + 63) / 64;
  if (c > held) c = held;
  if (c < (n + 255) / 256) c = (n + 255) / 256;
  return (c + 1023) / 1024 * 1024;
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

// kOne: the only workgroup, which counts for itself. What a wavefront does not hold of
// its run it reads twice.
template <bool kOne>
__global__ __launch_bounds__(1024) void sort_place_kernel(
    const int32_t* __restrict__ idx, int64_t n, int E, int bits, int64_t chunk, int chunks,
    const int32_t* __restrict__ counts, int32_t* __restrict__ perm, int32_t* __restrict__ pos,
    int32_t* __restrict__ offsets) {
  __shared__ int place[kSortWaves][kMaxBuckets];  // counts, then next places
  __shared__ int start[kMaxBuckets];              // totals, then first places
  __shared__ int parts[kSortWaves];
  __shared__ int shared_sum[kOne ? 1 : 1024], shared_pre[kOne ? 1 : 1024];
  const int tid = threadIdx.x, lane = tid & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int B = E + 1;
  const int64_t first = blockIdx.x * chunk, last = first + chunk < n ? first + chunk : n;
  const int64_t run = (chunk + kSortWaves * kWave - 1) / (kSortWaves * kWave) * kWave;
  const int64_t r0 = first + wave * run, r1 = r0 + run < last ? r0 + run : last;
  int held[kHeld];
#pragma unroll
  for (int u = 0; u < kHeld; ++u) {
    const int64_t a = r0 + u * kWave + lane;
    held[u] = r0 + u * kWave < r1 ? idx[a < r1 ? a : r0] : 0;
  }
  // counts of all chunks, and of those before this one
  int sum = 0, pre = 0, more = 0;
  // groups of `width` threads share the chunks; 16 counts of each in flight
  const int width = B <= 128 ? 128 : B <= 256 ? 256 : B <= 512 ? 512 : 1024;
  const int groups = 1024 / width;
  if constexpr (!kOne) {
    const int b = tid & (width - 1), group = tid / width;
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
    if (B > 1024 && wave == 0) {  // bucket 1024
      for (int c = lane; c < (int)blockIdx.x; c += kWave) more += counts[(int64_t)c * B + 1024];
      more = wave_inclusive_scan(more);
      more = __builtin_amdgcn_readlane(more, kWave - 1);
    }
  }
  for (int b = lane; b < B; b += kWave) place[wave][b] = 0;
#pragma unroll
  for (int u = 0; u < kHeld; ++u) held[u] = held[u] >= 0 && held[u] < E ? held[u] : E;
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
#pragma unroll
  for (int u = 0; u < kHeld; ++u)
    if (r0 + u * kWave + lane < r1) atomicAdd(&place[wave][held[u]], 1);
  for (int64_t a = r0 + kHeld * kWave + lane; a < r1; a += kWave)
    atomicAdd(&place[wave][bucket_of(idx, a, E)], 1);
  __syncthreads();
  // per bucket: the wavefronts' counts become prefixes
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
  if constexpr (!kOne)
    if (on)
      for (int g = 0; g < groups; ++g) {
        total += shared_sum[g * width + tid];
        before += shared_pre[g * width + tid];
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
    int sum = 0;
    for (int w = 0; w < kSortWaves; ++w) {
      const int c = place[w][1024];
      place[w][1024] = sum;
      sum += c;
    }
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
  auto put = [&](int64_t a0, int b) {
    const int64_t a = a0 + lane;
    const bool live = a < r1;
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
  };
#pragma unroll
  for (int u = 0; u < kHeld; ++u)
    if (r0 + u * kWave < r1) put(r0 + u * kWave, held[u]);
  for (int64_t a0 = r0 + kHeld * kWave; a0 < r1; a0 += kWave)
    put(a0, a0 + lane < r1 ? bucket_of(idx, a0 + lane, E) : 0);
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
