// Orthogonalised updates by Newton-Schulz products: for every matrix G [N][K],
// with m <= n its sides and X = G / |G| (or its transpose) [m][n],
//
//   A = X X^T        Q = a I + b A + c A A        X' = Q X
//
// a few times, which drives X's singular values towards 1.
//
// All products run in the LDS ring of the ragged products, both operands with
// the summed index along their rows: A from X twice, Q from A twice (A is
// symmetric, so its rows are its columns), and the last one as X'^T = X^T Q
// from X^T [n][m] and Q's rows. X is therefore kept in both orientations, and
// its product's tiles are stored twice, one of them turned around. A and Q are
// symmetric: the tiles on and below the diagonal are computed and stored to
// both places, which saves almost half of the first two products. a I is part
// of Q, so the last product needs no second operand and its rounding is
// relative to what X is multiplied by.
//
// Between products values are fp16: eight times finer than bf16 at the same
// rate of the matrix cores. X is kept times a power of two that makes its
// elements' root mean square 2^-5 to 2^-4 at first, far above fp16's subnormals;
// as |X| = 1 at the start no element passes 2^10. A and Q need no scale: Q's
// elements are near a on the diagonal, and an error of 2^-25 in A moves Q by b
// 2^-25 there.
#include "ragged_device.hpp"
#include "ring_body.hpp"
#include "router.hpp"

namespace moe {
namespace {

constexpr int kNormParts = 128;  // workgroups that sum a matrix's squares
constexpr double kNormFloor = 1e-20;

// Sums of squares of a matrix's parts, in fp64: no fp32 square overflows it.
template <typename T>
__global__ __launch_bounds__(256) void ortho_norm_kernel(const T* g, int64_t size,
                                                         double* parts) {
  __shared__ double sums[4];
  const T* x = g + blockIdx.y * size;
  constexpr int U = 8;
  double sum = 0.0;
  for (int64_t i = (int64_t)blockIdx.x * 256 * U + threadIdx.x; i < size;
       i += (int64_t)gridDim.x * 256 * U) {
    float v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) v[u] = i + u * 256 < size ? to_f32(x[i + u * 256]) : 0.f;
#pragma unroll
    for (int u = 0; u < U; ++u) sum += (double)v[u] * (double)v[u];
  }
#pragma unroll
  for (int s = 1; s < kWave; s <<= 1) sum += __shfl_xor(sum, s);
  if (threadIdx.x % kWave == 0) sums[threadIdx.x / kWave] = sum;
  __syncthreads();
  if (threadIdx.x == 0)
    parts[(int64_t)blockIdx.y * gridDim.x + blockIdx.x] = sums[0] + sums[1] + sums[2] + sums[3];
}

struct SplitParams {
  const void* g;
  const double* parts;
  int n_parts;
  int N, K;
  double scale;          // 2^s
  char* same;            // fp16 [N][K padded], ld_same elements apart
  char* turned;          // fp16 [K][N padded], ld_turned apart
  int64_t ld_same, ld_turned, same_batch, turned_batch;  // elements
};

// A matrix divided by its norm, in fp16, as it is and turned around: 64 x 64
// tiles through LDS. Columns are padded with zeros to whole 16 bytes.
template <typename T>
__global__ __launch_bounds__(256) void ortho_split_kernel(SplitParams p) {
  __shared__ f16 tile[64][64 + 2];
  __shared__ double factor;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int e = blockIdx.z;
  if (wave == 0) {
    double sum = 0.0;
    for (int i = lane; i < p.n_parts; i += kWave) sum += p.parts[(int64_t)e * p.n_parts + i];
#pragma unroll
    for (int s = 1; s < kWave; s <<= 1) sum += __shfl_xor(sum, s);
    const double norm = sqrt(sum);
    // an infinite norm divides by nothing: the matrix becomes NaN
    if (lane == 0)
      factor = norm < __builtin_inf() ? p.scale / (norm + kNormFloor) : __builtin_nan("");
  }
  __syncthreads();
  const double f = factor;
  const int r0 = blockIdx.y * 64, c0 = blockIdx.x * 64;
  const int Kp = (p.K + 7) & ~7, Np = (p.N + 7) & ~7;
  const T* g = static_cast<const T*>(p.g) + (int64_t)e * p.N * p.K;
  f16* same = reinterpret_cast<f16*>(p.same) + e * p.same_batch;
  f16* turned = reinterpret_cast<f16*>(p.turned) + e * p.turned_batch;
#pragma unroll 4
  for (int i = 0; i < 16; ++i) {
    const int r = wave * 16 + i, row = r0 + r, col = c0 + lane;
    float v = 0.f;
    if (row < p.N && col < p.K) v = (float)((double)to_f32(g[(int64_t)row * p.K + col]) * f);
    const f16 h = from_f32<f16>(v);
    tile[r][lane] = h;
    if (row < p.N && col < Kp) same[row * p.ld_same + col] = h;
  }
  __syncthreads();
#pragma unroll 4
  for (int i = 0; i < 16; ++i) {
    const int c = wave * 16 + i;
    if (c0 + c < p.K && r0 + lane < Np) turned[(c0 + c) * p.ld_turned + r0 + lane] = tile[lane][c];
  }
}

enum OrthoMode {
  kGram,       // A: scaled
  kPoly,       // Q from A
  kApply,      // X^T and X
  kLastTall,   // y [n][m]
  kLastWide    // y [m][n]
};

struct OrthoParams {
  const char* act;  // [rows] of cbytes, lda apart
  const char* w;    // [B] of cbytes, ldw apart
  int64_t lda, ldw, act_batch, w_batch;  // bytes
  int cbytes;
  int lds;          // (scales of other operands)
  int E, rows, B;
  char* out;        // 16-bit [rows][out_cols], ldo elements apart
  char* turned;     // 16-bit [B][turned_cols], ldt apart
  int64_t ldo, ldt, out_batch, turned_batch;  // elements
  int out_cols, turned_cols;
  // stored: alpha sum + beta A + diag I
  float alpha, beta, diag;
  bool vec;         // the last product's rows are 16-byte aligned
};

template <int BN, int BM, int kMode>
struct OrthoJob {
  struct Tile {
    int e, m0, n0;
  };
  static constexpr bool kSymmetric = kMode == kGram || kMode == kPoly;
  static constexpr bool kLast = kMode == kLastTall || kMode == kLastWide;
  const OrthoParams& p;

  __device__ __forceinline__ int tiles_of_matrix() const {
    const int mt = (p.rows + BM - 1) / BM, nt = (p.B + BN - 1) / BN;
    return kSymmetric ? mt * (mt + 1) / 2 : mt * nt;
  }
  __device__ __forceinline__ int setup(int, int) const { return p.E * tiles_of_matrix(); }

  __device__ __forceinline__ Tile locate(int t) const {
    static_assert(!kSymmetric || BN == BM, "square tiles");
    const int per = tiles_of_matrix();
    Tile T;
    T.e = t / per;
    const int local = t - T.e * per;
    int m, n;
    if constexpr (kSymmetric) {
      // row m of the lower triangle holds tiles m (m + 1) / 2 ..
      m = (int)((__builtin_sqrtf(8.f * (float)local + 1.f) - 1.f) * 0.5f);
      while (m * (m + 1) / 2 > local) --m;
      while ((m + 1) * (m + 2) / 2 <= local) ++m;
      n = local - m * (m + 1) / 2;
    } else {
      place_tile(local, (p.rows + BM - 1) / BM, (p.B + BN - 1) / BN, &m, &n);
    }
    T.m0 = __builtin_amdgcn_readfirstlane(m * BM);
    T.n0 = __builtin_amdgcn_readfirstlane(n * BN);
    return T;
  }

  template <bool kTransW>
  __device__ __forceinline__ void operands(const Tile& T, bool exists, __amdgpu_buffer_rsrc_t* rw,
                                           __amdgpu_buffer_rsrc_t* ra) const {
    const int fw = p.B - T.n0 < BN ? p.B - T.n0 : BN;
    const int mr = p.rows - T.m0 < BM ? p.rows - T.m0 : BM;
    *rw = __builtin_amdgcn_make_buffer_rsrc(
        (void*)(p.w + T.e * p.w_batch + (int64_t)T.n0 * p.ldw), 0,
        exists ? (int)((uint32_t)(fw - 1) * (uint32_t)p.ldw + (uint32_t)p.cbytes) : 0, kRsrcWord3);
    *ra = __builtin_amdgcn_make_buffer_rsrc(
        (void*)(p.act + T.e * p.act_batch + (int64_t)T.m0 * p.lda), 0,
        exists ? (int)((uint32_t)(mr - 1) * (uint32_t)p.lda + (uint32_t)p.cbytes) : 0, kRsrcWord3);
  }

  // 32 rows x 64 columns of 16 bits from LDS (chunk q of row r at q ^ r % 8) to
  // row r0 of a buffer and column c0.
  __device__ __forceinline__ void put(const char* stg, char* to, int64_t ld, int r0, int rows,
                                      int c0, int cols, int lane) const {
    const int rrow = lane >> 3, rchunk = lane & 7, col = c0 + rchunk * 8;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = i * 8 + rrow;
      const u32x4 v =
          *reinterpret_cast<const u32x4*>(stg + r * 128 + ((rchunk ^ (r & 7)) * 16));
      uint16_t* at = reinterpret_cast<uint16_t*>(to) + (int64_t)(r0 + r) * ld + col;
      if (r0 + r < rows && col < cols) {
        if (!kLast || (p.vec && col + 8 <= cols)) {
          *reinterpret_cast<u32x4*>(at) = v;
        } else if (col + 8 <= cols) {
          __builtin_memcpy(at, &v, 16);
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if (col + k < cols) at[k] = (uint16_t)(v[k / 2] >> (16 * (k & 1)));
        }
      }
    }
  }

  // Sums in 64 x 64 blocks: every lane (row l32 of a block of 32, columns 8 q + 4
  // half + 0..3) rounds its 64 values, which go out by rows and by columns.
  template <int WI, int WJ>
  __device__ __forceinline__ void store(const Tile& T, const f32x16 (&acc)[WI][WJ], char* stg,
                                        int wn, int wm, int lane) const {
    static_assert(WI % 2 == 0 && WJ % 2 == 0, "blocks of 64 x 64");
    const int half = lane >> 5, l32 = lane & 31;
    char* out = p.out + T.e * p.out_batch * 2;
    char* turned = p.turned + T.e * p.turned_batch * 2;
    const bool mirror = !kSymmetric || T.m0 != T.n0;
#pragma unroll
    for (int jp = 0; jp < WJ / 2; ++jp)
#pragma unroll
      for (int ip = 0; ip < WI / 2; ++ip) {
        const int row0 = T.m0 + wm * (BM / 2) + jp * 64, col0 = T.n0 + wn * (BN / 2) + ip * 64;
        uint16_t v[2][2][16];  // of block (jp, ip): rows, columns, values
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const int row = row0 + j * 32 + l32, col = col0 + i * 32 + 8 * q + 4 * half;
              f16 add[4] = {};
              if constexpr (kMode == kPoly)
                if (row < p.rows && col < p.out_cols)  // whole fours of padded columns
                  __builtin_memcpy(add,
                                   p.act + T.e * p.act_batch + (int64_t)row * p.lda + col * 2, 8);
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                float s = p.alpha * acc_read(acc[2 * ip + i][2 * jp + j][4 * q + k]);
                if constexpr (kMode == kPoly) {
                  s = fmaf(p.beta, to_f32(add[k]), s);
                  if (row == col + k) s += p.diag;
                }
                if constexpr (kLast)
                  v[j][i][4 * q + k] = __builtin_bit_cast(uint16_t, from_f32<bf16>(s));
                else
                  v[j][i][4 * q + k] = __builtin_bit_cast(uint16_t, from_f32<f16>(s));
              }
            }
        if constexpr (kMode != kLastWide)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                const u32x2 four = {v[j][i][4 * q] | (uint32_t)v[j][i][4 * q + 1] << 16,
                                    v[j][i][4 * q + 2] | (uint32_t)v[j][i][4 * q + 3] << 16};
                *reinterpret_cast<u32x2*>(stg + l32 * 128 + (((i * 4 + q) ^ (l32 & 7)) * 16) +
                                          half * 8) = four;
              }
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            put(stg, out, p.ldo, row0 + j * 32, p.rows, col0, p.out_cols, lane);
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
          }
        if constexpr (kMode != kLastTall)
          if (mirror)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
#pragma unroll
              for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int x = 0; x < 16; ++x) {
                  const int r = 8 * (x >> 2) + 4 * half + (x & 3);
                  *reinterpret_cast<uint16_t*>(
                      stg + r * 128 + (((j * 4 + (l32 >> 3)) ^ (r & 7)) * 16) + (l32 & 7) * 2) =
                      v[j][i][x];
                }
              __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
              put(stg, turned, p.ldt, col0 + i * 32, p.B, row0, p.turned_cols, lane);
              __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            }
      }
  }
};

template <int kMode>
__global__ __launch_bounds__(256, 1) void ortho_wide_kernel(OrthoParams p) {
  OrthoJob<256, 256, kMode> job{p};
  wide_ring<OpF16, false>(job);
}

template <int kMode>
__global__ __launch_bounds__(256, 1) void ortho_ring_kernel(OrthoParams p) {
  OrthoJob<128, 128, kMode> job{p};
  ring<OpF16, 2, 2, 2, false>(job);
}

// 256 x 256 tiles, or 128 x 128 where those keep more CUs at work: turns of the
// CUs times a tile's area over its relative speed.
template <int kMode>
hipError_t product(const OrthoParams& p, int num_cus, hipStream_t st) {
  auto cost = [&](int b, float speed) {
    const int64_t mt = (p.rows + b - 1) / b, nt = (p.B + b - 1) / b;
    const int64_t tiles =
        p.E * (kMode == kGram || kMode == kPoly ? mt * (mt + 1) / 2 : mt * nt);
    return (float)((tiles + num_cus - 1) / num_cus) * (float)b * (float)b / speed;
  };
  const dim3 grid((unsigned)(num_cus < 8 ? 8 : num_cus / 8 * 8));
  if (cost(256, 1.f) <= cost(128, 0.7f))
    hipLaunchKernelGGL((ortho_wide_kernel<kMode>), grid, dim3(256), 0, st, p);
  else
    hipLaunchKernelGGL((ortho_ring_kernel<kMode>), grid, dim3(256), 0, st, p);
  return hipGetLastError();
}

int64_t up64(int64_t v) { return (v + 63) / 64 * 64; }

// The workspace: sums of squares, X, X^T twice, A and Q.
struct Layout {
  int64_t m, n, ldm, ldn;                   // ldm, ldn: row strides of m and n values
  int64_t x_size, t_size, a_size;           // elements of one matrix
  size_t parts, x, t[2], a, q, total;       // bytes
  Layout(int E, int N, int K) {
    m = N < K ? N : K;
    n = N < K ? K : N;
    ldm = up64(m);
    ldn = up64(n);
    x_size = m * ldn;
    t_size = n * ldm;
    a_size = m * ldm;
    size_t at = 0;
    auto take = [&](int64_t bytes) {
      const size_t was = at;
      at += ((size_t)bytes + 255) & ~size_t(255);
      return was;
    };
    parts = take((int64_t)E * kNormParts * 8);
    x = take(E * x_size * 2);
    t[0] = take(E * t_size * 2);
    t[1] = take(E * t_size * 2);
    a = take(E * a_size * 2);
    q = take(E * a_size * 2);
    total = at;
  }
};

template <typename T>
hipError_t split(int E, int N, int K, const void* g, double scale, const Layout& L, char* ws,
                 hipStream_t st) {
  const int64_t size = (int64_t)N * K;
  int parts = (int)((size + 256 * 8 * 4 - 1) / (256 * 8 * 4));
  parts = parts < kNormParts ? parts : kNormParts;
  double* sums = reinterpret_cast<double*>(ws + L.parts);
  hipLaunchKernelGGL(ortho_norm_kernel<T>, dim3(parts, E), dim3(256), 0, st,
                     static_cast<const T*>(g), size, sums);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const bool wide = N <= K;
  SplitParams p{};
  p.g = g;
  p.parts = sums;
  p.n_parts = parts;
  p.N = N;
  p.K = K;
  p.scale = scale;
  p.same = ws + (wide ? L.x : L.t[0]);
  p.turned = ws + (wide ? L.t[0] : L.x);
  p.ld_same = wide ? L.ldn : L.ldm;
  p.ld_turned = wide ? L.ldm : L.ldn;
  p.same_batch = wide ? L.x_size : L.t_size;
  p.turned_batch = wide ? L.t_size : L.x_size;
  hipLaunchKernelGGL(ortho_split_kernel<T>, dim3((K + 63) / 64, (N + 63) / 64, E), dim3(256), 0, st,
                     p);
  return hipGetLastError();
}

}  // namespace

size_t orthogonalize_bytes(int E, int N, int K) { return Layout(E, N, K).total; }

hipError_t launch_orthogonalize(ElemType t, int E, int N, int K, const void* g, void* y, int steps,
                                const float* coefficients, float scale, char* ws, int num_cus,
                                hipStream_t st) {
  const Layout L(E, N, K);
  // the elements' root mean square is 1 / sqrt(m n) at first
  int s = 0;
  while ((int64_t)4 << (2 * s) <= L.m * L.n) ++s;  // 2^s <= sqrt(m n) < 2^(s + 1)
  s = s > 4 ? s - 4 : 0;
  const float up = (float)(1 << s);
  hipError_t e = t == ElemType::kF32    ? split<float>(E, N, K, g, up, L, ws, st)
                 : t == ElemType::kBF16 ? split<bf16>(E, N, K, g, up, L, ws, st)
                                        : split<f16>(E, N, K, g, up, L, ws, st);
  const int m = (int)L.m, n = (int)L.n, m8 = (m + 7) & ~7, n8 = (n + 7) & ~7;
  int cur = 0;
  for (int i = 0; i < steps && e == hipSuccess; ++i) {
    const float* c = coefficients + 3 * i;
    OrthoParams p{};
    p.E = E;
    // A = X X^T
    p.act = p.w = ws + L.x;
    p.lda = p.ldw = L.ldn * 2;
    p.act_batch = p.w_batch = L.x_size * 2;
    p.cbytes = n8 * 2;
    p.rows = p.B = m;
    p.out = p.turned = ws + L.a;
    p.ldo = p.ldt = L.ldm;
    p.out_batch = p.turned_batch = L.a_size;
    p.out_cols = p.turned_cols = m8;
    p.alpha = 1.f / (up * up);
    if ((e = product<kGram>(p, num_cus, st)) != hipSuccess) break;
    // Q = a I + b A + c A A
    p.act = p.w = ws + L.a;
    p.lda = p.ldw = L.ldm * 2;
    p.act_batch = p.w_batch = L.a_size * 2;
    p.cbytes = m8 * 2;
    p.out = p.turned = ws + L.q;
    p.alpha = c[2];
    p.beta = c[1];
    p.diag = c[0];
    if ((e = product<kPoly>(p, num_cus, st)) != hipSuccess) break;
    // X'^T = X^T Q
    p.act = ws + L.t[cur];
    p.act_batch = L.t_size * 2;
    p.w = ws + L.q;
    p.rows = n;
    p.alpha = 1.f;
    if (i + 1 < steps) {
      p.out = ws + L.t[1 - cur];
      p.out_batch = L.t_size;
      p.turned = ws + L.x;
      p.ldt = L.ldn;
      p.turned_batch = L.x_size;
      p.turned_cols = n8;
      e = product<kApply>(p, num_cus, st);
      cur = 1 - cur;
    } else {
      p.out = p.turned = static_cast<char*>(y);
      p.ldo = p.ldt = K;
      p.out_batch = p.turned_batch = (int64_t)N * K;
      p.out_cols = m;
      p.turned_cols = n;
      p.alpha = scale / up;
      p.vec = K % 8 == 0 && (reinterpret_cast<uintptr_t>(y) & 15) == 0;
      e = N <= K ? product<kLastWide>(p, num_cus, st) : product<kLastTall>(p, num_cus, st);
    }
  }
  return e;
}

}  // namespace moe
