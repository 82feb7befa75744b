// Orthogonalised updates by Newton-Schulz products: for every matrix G [N][K],
// with m <= n its sides and X = G / |G| (or its transpose) [m][n],
//
//   A = X X^T        P = (a - d) I + b A + c A A        X' = d X + P X
//
// a few times, which drives X's singular values towards 1.
//
// All products run in the LDS ring of the ragged products, both operands with
// the summed index along their rows: A from X twice, P from A twice (A is
// symmetric, so its rows are its columns), and the last one as X'^T = X^T P
// from X^T [n][m] and P's rows. X is therefore kept in both orientations, and
// its product's tiles are stored twice, one of them turned around. A and P are
// symmetric: the tiles on and below the diagonal are computed and stored to
// both places, which saves almost half of the first two products.
//
// The products' operands are fp16: eight times finer than bf16 at the same rate of
// the matrix cores. What an error does depends on where it lies. One of A or P is
// multiplied by X, so it keeps X's null spaces and stays of its size. One of X
// itself that lies in X's left and right null space is multiplied by about a in
// every step, by 485 in five: with fp16's 2^-12 a matrix of rank one, the gradient of
// an expert that got one token, is 0.15 of its norm off. So X has 22 bits, as hi + lo
// 2^-11 with two fp16 values (X^T alone has lo), and d X is added to the product in
// fp32; P X takes hi alone, which with d = a leaves the null spaces alone. Where what
// X's rounding still grows by is small (kGrowth), d is the middle of a + b s s + c s^4
// over singular values s from 0 to 1, so that P and its rounding are small. Distance
// of y from the fp64 iteration, of its norm, at full rank, rank 64, 8 and 1: 2048 x 2048
// 1.8e-3, 2.0e-3, 2.0e-3, 2.1e-3; 512 x 512 1.9e-3, 2.1e-3, 2.0e-3, 2.1e-3; 64 x 64 2.4e-3,
// -, 2.1e-3, 2.1e-3 (y's own rounding: 1.7e-3; X in fp16: 2e-3, 0.02, 0.04, 0.15).
//
// X is kept times a power of two that makes its elements' root mean square 2^-5 to
// 2^-4 at first, far above fp16's subnormals; as |X| = 1 at the start no element
// passes 2^10. A and P need no scale: an error of 2^-25 in A moves P by b 2^-25.
//
// 32 matrices of 2048 x 2048 from fp32, five steps: 6.55-6.6 ms, 5.50 TFLOP with half
// of the symmetric products, 0.84 PFLOP/s (a library product in fp16 reaches 1.19): 87 +
// 234 us to divide by the norm, then per step A 300-310, P 320 and X' 640 us (the last
// one 565). MFMA pipes are busy 47-67% of the cycles at 1.65-1.75 GHz, the chip's power
// limit; the ring's loop alone keeps them busy 76%. The rest is a tile's reads and
// stores between two tiles (256 KiB in and 384 out a workgroup and round, all at once)
// and, for A and P, the 4.5 rounds of 36 x 32 tiles over 256 CUs. (X in fp16 alone:
// 5.9-6.1 ms, X' 520.) Starting the workgroups a quarter of a tile apart did not help.
#include "ragged_device.hpp"
#include "ring_body.hpp"
#include "router.hpp"

namespace moe {
namespace {

typedef f16 f16x4 __attribute__((ext_vector_type(4)));

constexpr int kNormParts = 128;  // workgroups that sum a matrix's squares
constexpr double kNormFloor = 1e-20;

// Sums of squares of a matrix's parts, in fp64: no fp32 square overflows it.
template <typename T>
__global__ __launch_bounds__(256) void ortho_norm_kernel(const T* g, int64_t size,
                                                         double* parts) {
  __shared__ double sums[4];
  constexpr int V = 16 / sizeof(T), U = 4;  // vectors in flight
  const T* x = g + blockIdx.y * size;
  const int64_t vectors = size / V;
  double sum = 0.0;
  for (int64_t i = (int64_t)blockIdx.x * 256 * U + threadIdx.x; i < vectors;
       i += (int64_t)gridDim.x * 256 * U) {
    union {
      T e[V];
      u32x4 v;
    } r[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      // (the address need only be an element's)
      const int64_t at = i + u * 256 < vectors ? i + u * 256 : vectors - 1;
      __builtin_memcpy(&r[u].v, x + at * V, 16);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      double part = 0.0;
#pragma unroll
      for (int k = 0; k < V; ++k) {
        const double d = (double)to_f32(r[u].e[k]);
        part = fma(d, d, part);
      }
      sum += i + u * 256 < vectors ? part : 0.0;
    }
  }
  if (blockIdx.x == 0 && (int64_t)threadIdx.x < size - vectors * V) {
    const double d = (double)to_f32(x[vectors * V + threadIdx.x]);
    sum += d * d;
  }
#pragma unroll
  for (int s = 1; s < kWave; s <<= 1) sum += __shfl_xor(sum, s);
  if (threadIdx.x % kWave == 0) sums[threadIdx.x / kWave] = sum;
  __syncthreads();
  if (threadIdx.x == 0)
    parts[(int64_t)blockIdx.y * gridDim.x + blockIdx.x] = sums[0] + sums[1] + sums[2] + sums[3];
}

// What a matrix is multiplied by, from the sum of its squares: an infinite norm
// divides by nothing, and the matrix becomes NaN.
__device__ __forceinline__ double factor_of(double squares, double scale) {
  const double norm = sqrt(squares);
  return norm < __builtin_inf() ? scale / (norm + kNormFloor) : __builtin_nan("");
}

struct SplitParams {
  const void* g;
  const double* parts;
  int n_parts;
  int N, K;
  double scale;          // 2^s
  char* same;            // fp16 [N][K padded], ld_same elements apart
  char* turned;          // fp16 [K][N padded], ld_turned apart
  char* lo;              // and what fp16 leaves of the one that holds X^T
  bool lo_turned;
  int64_t ld_same, ld_turned, same_batch, turned_batch;  // elements
};

// X = hi + lo / kLoScale: hi is X in fp16, lo what that leaves, scaled so that it has
// hi's exponents.
constexpr float kLoScale = 2048.f;
__device__ __forceinline__ f16 lo_of(float x, f16 hi) {
  return from_f32<f16>((x - to_f32(hi)) * kLoScale);
}
__device__ __forceinline__ float whole_of(f16 hi, f16 lo) {
  return fmaf(to_f32(lo), 1.f / kLoScale, to_f32(hi));
}

// A matrix divided by its norm, in fp16, as it is and turned around, and lo: 64 x 64
// tiles through LDS. Columns are padded with zeros to whole 16 bytes.
template <typename T>
__global__ __launch_bounds__(256) void ortho_split_kernel(SplitParams p) {
  __shared__ f16 tile[64][64 + 2], low[64][64 + 2];
  __shared__ double factor;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int e = blockIdx.z;
  if (wave == 0) {
    double sum = 0.0;
    for (int i = lane; i < p.n_parts; i += kWave) sum += p.parts[(int64_t)e * p.n_parts + i];
#pragma unroll
    for (int s = 1; s < kWave; s <<= 1) sum += __shfl_xor(sum, s);
    if (lane == 0) factor = factor_of(sum, p.scale);
  }
  __syncthreads();
  const double f = factor;
  const int r0 = blockIdx.y * 64, c0 = blockIdx.x * 64;
  const int Kp = (p.K + 7) & ~7, Np = (p.N + 7) & ~7;
  const T* g = static_cast<const T*>(p.g) + (int64_t)e * p.N * p.K;
  f16* same = reinterpret_cast<f16*>(p.same) + e * p.same_batch;
  f16* turned = reinterpret_cast<f16*>(p.turned) + e * p.turned_batch;
  f16* lo = reinterpret_cast<f16*>(p.lo) + e * (p.lo_turned ? p.turned_batch : p.same_batch);
  const int part = tid >> 4, four = (tid & 15) * 4;
  float v[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = r0 + part + 16 * i, col = c0 + four;
    const T* at = g + (int64_t)row * p.K + col;
    T x[4] = {};
    if (row < p.N && col + 4 <= p.K) {
      __builtin_memcpy(x, at, sizeof x);
    } else if (row < p.N) {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (col + k < p.K) x[k] = at[k];
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) v[i][k] = to_f32(x[k]);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = part + 16 * i, row = r0 + r, col = c0 + four;
    f16x4 h, l;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      // elements past the last are 0, not a NaN factor's product with it
      const bool in = (row < p.N) & (col + k < p.K);
      const float x = in ? (float)((double)v[i][k] * f) : 0.f;
      h[k] = from_f32<f16>(x);
      l[k] = lo_of(x, h[k]);
      tile[r][four + k] = h[k];
      low[r][four + k] = l[k];
    }
    if (row < p.N && col < Kp) {  // whole fours
      *reinterpret_cast<f16x4*>(same + row * p.ld_same + col) = h;
      if (!p.lo_turned) *reinterpret_cast<f16x4*>(lo + row * p.ld_same + col) = l;
    }
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int c = part + 16 * i;
    f16x4 h, l;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      h[k] = tile[four + k][c];
      l[k] = low[four + k][c];
    }
    if (c0 + c < p.K && r0 + four < Np) {
      *reinterpret_cast<f16x4*>(turned + (c0 + c) * p.ld_turned + r0 + four) = h;
      if (p.lo_turned)
        *reinterpret_cast<f16x4*>(lo + (c0 + c) * p.ld_turned + r0 + four) = l;
    }
  }
}

enum OrthoMode {
  kGram,       // A: scaled
  kPoly,       // P from A
  kApply,      // X^T, its lo, and X
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
  // stored: alpha sum + beta A + diag I, or alpha (sum + keep X^T)
  float alpha, beta, diag, keep;
  char* lo;         // of X^T, laid out as act; kApply replaces it by that of out
  bool vec;         // the last product's rows are 16-byte aligned
};

template <int BN, int BM, int kMode>
struct OrthoJob {
  struct Tile {
    int e, m0, n0;
  };
  static constexpr bool kSymmetric = kMode == kGram || kMode == kPoly;
  static constexpr bool kLast = kMode == kLastTall || kMode == kLastWide;
  static constexpr int kStaging = 8192;  // bytes of LDS a wavefront
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

  // Rows m0 .. of a matrix that is stored to: those past `rows` and columns past
  // `cols` are dropped.
  struct Target {
    __amdgpu_buffer_rsrc_t buffer;
    uint16_t* at;
    uint32_t ld;  // bytes
    int rows, cols;
  };
  __device__ __forceinline__ Target target(char* base, int64_t batch, int64_t ld, int m0, int most,
                                           int rows, int cols) const {
    Target t;
    t.at = reinterpret_cast<uint16_t*>(base) + batch + m0 * ld;
    t.ld = (uint32_t)ld * 2;
    t.rows = rows - m0 < most ? rows - m0 : most;
    t.cols = cols;
    t.buffer = __builtin_amdgcn_make_buffer_rsrc(
        (void*)t.at, 0, (int)((uint32_t)(t.rows - 1) * t.ld + (uint32_t)cols * 2), kRsrcWord3);
    return t;
  }
  // 64 rows x 64 columns of 16 bits from LDS (chunk q of row r at q ^ r % 8) to
  // row r0 of the target and column c0: all are read before the first is stored.
  __device__ __forceinline__ void put(const char* stg, const Target& t, int r0, int c0,
                                      int lane) const {
    const int rrow = lane >> 3, rchunk = lane & 7, col = c0 + rchunk * 8;
    u32x4 v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = i * 8 + rrow;
      v[i] = *reinterpret_cast<const u32x4*>(stg + r * 128 + ((rchunk ^ (r & 7)) * 16));
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = i * 8 + rrow;
      if (!kLast || p.vec) {
        const uint32_t off = (uint32_t)(r0 + r) * t.ld + (uint32_t)col * 2;
        __builtin_amdgcn_raw_buffer_store_b128(v[i], t.buffer,
                                               (int)(col < t.cols ? off : kOutOfRange), 0,
                                               kNonTemporal);
      } else if (r0 + r < t.rows) {
        uint16_t* at = t.at + (int64_t)(r0 + r) * (t.ld / 2) + col;
        if (col + 8 <= t.cols) {
          __builtin_memcpy(at, &v[i], 16);
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if (col + k < t.cols) at[k] = (uint16_t)(v[i][k / 2] >> (16 * (k & 1)));
        }
      }
    }
  }

  // And 64 x 64 values of rows lda bytes apart into LDS, from byte `at` of row r0 on:
  // whole row pieces of 128 bytes, where lanes that read their own 8 bytes of 32 rows
  // took 19 us a round of tiles for hi and lo.
  __device__ __forceinline__ void get(char* stg, __amdgpu_buffer_rsrc_t from, int r0, int at,
                                      int lane) const {
    const int rrow = lane >> 3, rchunk = lane & 7;
    u32x4 v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      v[i] = __builtin_bit_cast(
          u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                     from, (r0 + i * 8 + rrow) * (int)p.lda + at + rchunk * 16, 0, 0));
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = i * 8 + rrow;
      *reinterpret_cast<u32x4*>(stg + r * 128 + ((rchunk ^ (r & 7)) * 16)) = v[i];
    }
  }

  // Sums in 64 x 64 blocks: every lane (row l32 of a block of 32, columns 8 q + 4
  // half + 0..3) rounds its 64 values in pairs of columns, which go out by rows and
  // by columns, 8 KiB of LDS at a time. For the columns, neighbouring lanes exchange
  // one value of each pair, so that a lane holds two rows of one column. (A block's lo
  // is read before it is replaced, by the same wavefront.)
  template <int WI, int WJ>
  __device__ __forceinline__ void store(const Tile& T, const f32x16 (&acc)[WI][WJ], char* stg,
                                        int wn, int wm, int lane) const {
    static_assert(WI % 2 == 0 && WJ % 2 == 0, "blocks of 64 x 64");
    typedef f16 f16x2 __attribute__((ext_vector_type(2)));
    constexpr bool kHasLo = kMode == kApply;
    const int half = lane >> 5, l32 = lane & 31;
    const Target out = target(p.out, T.e * p.out_batch, p.ldo, T.m0, BM, p.rows, p.out_cols);
    const Target turned = target(p.turned, T.e * p.turned_batch, p.ldt, T.n0, BN, p.B,
                                 p.turned_cols);
    const bool mirror = !kSymmetric || T.m0 != T.n0;
    // A's or X^T's values where this tile's lie, and lo; what lies past the last row
    // or column is not stored
    const int mr = p.rows - T.m0 < BM ? p.rows - T.m0 : BM;
    const int64_t first = T.e * p.act_batch + T.m0 * p.lda;
    const __amdgpu_buffer_rsrc_t values = __builtin_amdgcn_make_buffer_rsrc(
        (void*)(p.act + first), 0, (int)((uint32_t)mr * (uint32_t)p.lda), kRsrcWord3);
    const __amdgpu_buffer_rsrc_t lows = __builtin_amdgcn_make_buffer_rsrc(
        (void*)(p.lo + first), 0, (int)((uint32_t)mr * (uint32_t)p.lda), kRsrcWord3);
    // halves of (own pair, neighbour's): an even lane takes the first column of
    // both, an odd one the second of both, the neighbour's row before its own
    const uint32_t pick = lane & 1 ? 0x07060302u : 0x01000504u;
    typedef uint32_t block_t[2][2][8];  // of block (j, i): pairs of columns
    auto own8 = [&](int j, int i, int q) {  // this lane's 8 bytes of a block in LDS
      return reinterpret_cast<u32x2*>(stg + (j * 32 + l32) * 128 +
                                      (((i * 4 + q) ^ (l32 & 7)) * 16) + half * 8);
    };
    auto get_rows = [&](block_t& v, __amdgpu_buffer_rsrc_t from, int row0, int col0) {
      get(stg, from, row0, (T.n0 + col0) * 2, lane);
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const u32x2 w = *own8(j, i, q);
            v[j][i][2 * q] = w[0];
            v[j][i][2 * q + 1] = w[1];
          }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    };
    auto put_rows = [&](const block_t& v, const Target& t, int row0, int col0) {
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int q = 0; q < 4; ++q)
            *own8(j, i, q) = u32x2{v[j][i][2 * q], v[j][i][2 * q + 1]};
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      put(stg, t, row0, T.n0 + col0, lane);
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    };
#pragma unroll
    for (int jp = 0; jp < WJ / 2; ++jp)
#pragma unroll
      for (int ip = 0; ip < WI / 2; ++ip) {
        const int row0 = wm * (BM / 2) + jp * 64, col0 = wn * (BN / 2) + ip * 64;
        block_t v, low;  // what is read, then what is stored
        if constexpr (kMode != kGram) get_rows(v, values, row0, col0);
        if constexpr (!kSymmetric) get_rows(low, lows, row0, col0);
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const int row = row0 + j * 32 + l32, col = col0 + i * 32 + 8 * q + 4 * half;
              f16x4 add = {}, rest = {};
              if constexpr (kMode != kGram)
                add = __builtin_bit_cast(f16x4, u32x2{v[j][i][2 * q], v[j][i][2 * q + 1]});
              if constexpr (!kSymmetric)
                rest = __builtin_bit_cast(f16x4, u32x2{low[j][i][2 * q], low[j][i][2 * q + 1]});
              float s[4];
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                s[k] = acc_read(acc[2 * ip + i][2 * jp + j][4 * q + k]);
                if constexpr (!kSymmetric)
                  s[k] = fmaf(p.keep, whole_of(add[k], rest[k]), s[k]);
                if constexpr (kMode != kApply) s[k] *= p.alpha;
                if constexpr (kMode == kPoly) {
                  s[k] = fmaf(p.beta, to_f32(add[k]), s[k]);
                  s[k] += T.m0 + row == T.n0 + col + k ? p.diag : 0.f;
                }
              }
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                v[j][i][2 * q + k] = pack(s[2 * k], s[2 * k + 1]);
                if constexpr (kHasLo) {
                  const f16x2 h = __builtin_bit_cast(f16x2, v[j][i][2 * q + k]);
                  const f16x2 l = {lo_of(s[2 * k], h[0]), lo_of(s[2 * k + 1], h[1])};
                  low[j][i][2 * q + k] = __builtin_bit_cast(uint32_t, l);
                }
              }
            }
        if constexpr (kMode != kLastWide) put_rows(v, out, row0, col0);
        if constexpr (kHasLo)
          put_rows(low, target(p.lo, T.e * p.out_batch, p.ldo, T.m0, BM, p.rows, p.out_cols),
                   row0, col0);
        if constexpr (kMode != kLastTall)
          if (mirror) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
              for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int x = 0; x < 8; ++x) {
                  const uint32_t own = v[j][i][x];
                  const uint32_t next =
                      (uint32_t)__builtin_amdgcn_mov_dpp((int)own, 0xb1, 0xf, 0xf, true);
                  const int r = i * 32 + 8 * (x >> 1) + 4 * half + 2 * (x & 1) + (lane & 1);
                  *reinterpret_cast<uint32_t*>(
                      stg + r * 128 + (((j * 4 + (l32 >> 3)) ^ (r & 7)) * 16) + (l32 & 6) * 2) =
                      __builtin_amdgcn_perm(own, next, pick);
                }
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            put(stg, turned, col0, T.m0 + row0, lane);
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
          }
      }
  }
  __device__ __forceinline__ static uint32_t pack(float a, float b) {
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    typedef f16 f16x2 __attribute__((ext_vector_type(2)));
    typedef bf16 bf16x2 __attribute__((ext_vector_type(2)));
    const f32x2 s = {a, b};
    if constexpr (kLast) return __builtin_bit_cast(uint32_t, __builtin_convertvector(s, bf16x2));
    else return __builtin_bit_cast(uint32_t, __builtin_convertvector(s, f16x2));
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
// CUs times a tile's area over its relative speed. All products of an update, with
// 256 and with 128: 32 of 2048 x 2048 6.6 and 8.9 ms, 4 of them 1.12 and 1.33, one 0.88
// and 0.42; 32 of 512 x 512 445 and 364 us, 16 of 1024 x 1024 715 and 807; 8 of 1024 x
// 2048 817 and 761, by product (as here) 676.
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

// ---------------------------------------------------------------- small matrices
// A matrix whose X and A fit in LDS together is one workgroup's: one launch
// instead of three a step. NB blocks of 32 rows hold m; rows are 16 bytes longer
// than their values, so that 32 of them, read 16 bytes each, cover all banks.
//
// A wavefront's results wait in registers while A is read, then P replaces A. X stays
// in fp32 in the registers of the wavefronts, in strips of 32 columns, and in LDS in
// fp16 as the products' operand: X'[:, strip] = d X[:, strip] + P X[:, strip], so a
// wavefront that holds its strip's fragments may overwrite it. The MFMA's row operand
// is the index that lies along a stored row (a lane ends with fours of it).
//
// Latency: a step of 3 matrices of 201 x 77 takes 2.8 us of its own, reading, the norm
// and writing 8 (22 us in all; 103 with three launches a step); 32 of 128 x 256 40 (135),
// 256 of 128 x 128 33 (148), 512 of 192 x 192 127-144 (600).
constexpr int kSmallBlocks = 6;
constexpr int kSmallWaves = 8;
// LDS of X and A: so that two matrices share a CU where they can, or all of it.
constexpr int kSmallBytes = 65536 - 256, kLargeBytes = 163840 - 256;
// Bytes of a row of n values.
__host__ __device__ constexpr int small_row(int n) { return 2 * n + 16; }

struct SmallParams {
  const void* g;
  bf16* y;
  ElemType type;
  int N, K, steps;
  float up, scale;
  float c[3 * kOrthoMaxSteps], kept[kOrthoMaxSteps];
};

constexpr int kSmallThreads = kSmallWaves * kWave;

// Where an element of G [N][K] or y lies in X [m][n]: a walk along G's rows.
struct Place {
  int c, at;           // column of G, byte of X
  int K, next, turn;   // steps to the next column, and to the next row's first
  __device__ __forceinline__ Place(int e, int N, int K_, int ldx) : K(K_) {
    const bool wide = N <= K;
    // e below 2^24: the quotient is off by one at most
    int r = (int)((float)e * (1.f / (float)K));
    r -= r * K > e;
    r += (r + 1) * K <= e;
    c = e - r * K;
    at = wide ? r * ldx + c * 2 : c * ldx + r * 2;
    next = wide ? 2 : ldx;
    turn = wide ? ldx - K * 2 : 2 - K * ldx;
  }
  __device__ __forceinline__ void step() {
    ++c;
    at += next;
    const bool over = c == K;
    at += over ? turn : 0;
    c = over ? 0 : c;
  }
};

// Strips of X that a wavefront holds at most, where a matrix of NB blocks of rows and
// its A take up to `bytes`.
constexpr int small_strips(int NB, int bytes) {
  const int np = (bytes / (32 * NB) - small_row(32 * NB) - small_row(0)) / 2;
  return (np / 32 + kSmallWaves - 1) / kSmallWaves;
}

// x: G's elements where the strips of this wavefront hold X, zeros past its last row
// and column. Lane: row 32 b + l32 of X, columns 32 s + 8 q + 4 half + 0..3.
template <typename T, int NB, int S>
__device__ __forceinline__ void small_load(const T* g, int N, int K, int wave,
                                           f32x16 (&x)[S][NB]) {
  const int lane = threadIdx.x & (kWave - 1), half = lane >> 5, l32 = lane & 31;
  const bool wide = N <= K;
  const int m = wide ? N : K, n = wide ? K : N, strips = (n + 31) / 32;
  const int down = wide ? K : 1, right = wide ? 1 : K;  // steps in G of a row of X, a column
  const bool fours = wide && n % 4 == 0;
#pragma unroll
  for (int t = 0; t < S; ++t) {
    const int s = wave + t * kSmallWaves;
#pragma unroll
    for (int b = 0; b < NB; ++b) x[t][b] = f32x16{};
    if (s >= strips) continue;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const int row = 32 * b + l32;
      T e[4][4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int col = 32 * s + 8 * q + 4 * half;
        if (fours) {  // from an element's address
          __builtin_memcpy(e[q], g + (row < m && col < n ? row * down + col : 0), sizeof e[q]);
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            e[q][k] = g[row < m && col + k < n ? row * down + (col + k) * right : 0];
        }
      }
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int k = 0; k < 4; ++k)
          x[t][b][4 * q + k] =
              row < m && 32 * s + 8 * q + 4 * half + k < n ? to_f32(e[q][k]) : 0.f;
    }
  }
}

template <int NB, int kBytes>
__global__ __launch_bounds__(kSmallThreads, 1) void ortho_small_kernel(SmallParams p) {
  constexpr int mp = 32 * NB, lda = small_row(mp);
  constexpr int kBlocks = NB * (NB + 1) / 2, kOwn = (kBlocks + kSmallWaves - 1) / kSmallWaves;
  constexpr int S = small_strips(NB, kBytes);
  __shared__ __attribute__((aligned(16))) char lds[kBytes];
  __shared__ double sums[kSmallWaves];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int half = lane >> 5, l32 = lane & 31;
  const bool wide = p.N <= p.K;
  const int n = wide ? p.K : p.N;
  const int np = (n + 31) & ~31, ldx = small_row(np), strips = np / 32;
  char* a = lds;
  char* x = lds + mp * lda;
  const int64_t origin = (int64_t)blockIdx.x * p.N * p.K;
  f32x16 own[S][NB];
  if (p.type == ElemType::kF32)
    small_load(static_cast<const float*>(p.g) + origin, p.N, p.K, wave, own);
  else if (p.type == ElemType::kBF16)
    small_load(static_cast<const bf16*>(p.g) + origin, p.N, p.K, wave, own);
  else
    small_load(static_cast<const f16*>(p.g) + origin, p.N, p.K, wave, own);
  auto store4 = [&](char* at, float v0, float v1, float v2, float v3) {
    const f16x4 h = {from_f32<f16>(v0), from_f32<f16>(v1), from_f32<f16>(v2), from_f32<f16>(v3)};
    *reinterpret_cast<f16x4*>(at) = h;
  };
  // strip t's block b to LDS
  auto store_own = [&](int t, int b) {
    char* at = x + (32 * b + l32) * ldx + 64 * (wave + t * kSmallWaves) + 8 * half;
#pragma unroll
    for (int q = 0; q < 4; ++q)
      store4(at + 16 * q, own[t][b][4 * q], own[t][b][4 * q + 1], own[t][b][4 * q + 2],
             own[t][b][4 * q + 3]);
  };
  {
    // squares in fp64: no fp32 square overflows it
    double sum = 0.0;
#pragma unroll
    for (int t = 0; t < S; ++t)
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int v = 0; v < 16; ++v) {
          const double d = (double)own[t][b][v];
          sum = fma(d, d, sum);
        }
#pragma unroll
    for (int s = 1; s < kWave; s <<= 1) sum += __shfl_xor(sum, s);
    if (lane == 0) sums[wave] = sum;
    __syncthreads();
    sum = 0.0;
#pragma unroll
    for (int w = 0; w < kSmallWaves; ++w) sum += sums[w];
    // in fp32 as two factors, the first a power of two, where f itself could leave
    // its normal numbers
    const double f = factor_of(sum, (double)p.up);
    const float f0 = f < 0x1p-64 ? 0x1p-64f : 1.f, f1 = (float)(f / (double)f0);
#pragma unroll
    for (int t = 0; t < S; ++t)
      if (wave + t * kSmallWaves < strips)
#pragma unroll
        for (int b = 0; b < NB; ++b) {
#pragma unroll
          for (int v = 0; v < 16; ++v) own[t][b][v] = own[t][b][v] * f0 * f1;
          store_own(t, b);
        }
  }
  __syncthreads();

  // rows 32 b .. of a matrix in LDS, 16 of their values from k on: an operand
  auto rows_of = [&](const char* t, int ld, int b, int k) -> f16x8 {
    return *reinterpret_cast<const f16x8*>(t + (32 * b + l32) * ld + (k + 8 * half) * 2);
  };
  // columns 32 s .. of X, its rows 16 k ..: gfx950's transposing LDS read gives lane
  // i of 16 element i % 4 of the 8 bytes that lanes 4 j + i / 4 address, j = 0..3
  const int grp = lane >> 4, tr_row = 8 * (grp >> 1) + ((lane >> 2) & 3);
  const int tr_col = 16 * (grp & 1) + 4 * (lane & 3);
  auto columns_of = [&](int s, int k) -> f16x8 {
    const char* at = x + (16 * k + tr_row) * ldx + (32 * s + tr_col) * 2;
    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(lds_char*)at);
    const s16x4 hi =
        __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(lds_char*)(at + 4 * ldx));
    return __builtin_bit_cast(f16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
  };
  const float down = 1.f / (p.up * p.up);

  // this wavefront's blocks of a symmetric matrix, on and below the diagonal; one
  // past the last repeats it and is not stored
  int bi[kOwn], bj[kOwn];
#pragma unroll
  for (int o = 0; o < kOwn; ++o) {
    const int t = wave + o * kSmallWaves < kBlocks ? wave + o * kSmallWaves : kBlocks - 1;
    int i = 0;
    while ((i + 1) * (i + 2) / 2 <= t) ++i;
    bi[o] = i;
    bj[o] = t - i * (i + 1) / 2;
  }
  // sum over k of rows bi and bj of t, both fragments of the next 32 values in flight
  f32x16 acc[kOwn];
  auto multiply = [&](const char* t, int ld, int count) {
    f16x8 u[kOwn][2], w[kOwn][2];
    auto load = [&](int k) {
#pragma unroll
      for (int o = 0; o < kOwn; ++o)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          u[o][h] = rows_of(t, ld, bi[o], k + 16 * h);
          w[o][h] = rows_of(t, ld, bj[o], k + 16 * h);
        }
    };
#pragma unroll
    for (int o = 0; o < kOwn; ++o) acc[o] = f32x16{};
    load(0);
    for (int k = 0; k < count; k += 32) {
      f16x8 u0[kOwn][2], w0[kOwn][2];
#pragma unroll
      for (int o = 0; o < kOwn; ++o)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          u0[o][h] = u[o][h];
          w0[o][h] = w[o][h];
        }
      load(k + 32 < count ? k + 32 : 0);
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int o = 0; o < kOwn; ++o)
          acc[o] = __builtin_amdgcn_mfma_f32_32x32x16_f16(u0[o][h], w0[o][h], acc[o], 0, 0, 0);
    }
  };
  // a block to its place and, turned around, to the one across the diagonal
  auto store_blocks = [&]() {
#pragma unroll
    for (int o = 0; o < kOwn; ++o)
      if (wave + o * kSmallWaves < kBlocks) {
        char* at = a + (32 * bj[o] + l32) * lda + 64 * bi[o] + 8 * half;
#pragma unroll
        for (int q = 0; q < 4; ++q)
          store4(at + 16 * q, acc[o][4 * q], acc[o][4 * q + 1], acc[o][4 * q + 2],
                 acc[o][4 * q + 3]);
        if (bi[o] != bj[o]) {
          char* across = a + (32 * bi[o] + 4 * half) * lda + (32 * bj[o] + l32) * 2;
#pragma unroll
          for (int v = 0; v < 16; ++v)
            *reinterpret_cast<f16*>(across + (8 * (v >> 2) + (v & 3)) * lda) =
                from_f32<f16>(acc[o][v]);
        }
      }
  };

  for (int step = 0; step < p.steps; ++step) {
    const float kept = p.kept[step];
    const float ca = p.c[3 * step] - kept, cb = p.c[3 * step + 1], cc = p.c[3 * step + 2];
    // A = X X^T
    multiply(x, ldx, np);
#pragma unroll
    for (int o = 0; o < kOwn; ++o)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[o][v] *= down;
    store_blocks();
    __syncthreads();
    // P = (a - d) I + b A + c A A
    multiply(a, lda, mp);
#pragma unroll
    for (int o = 0; o < kOwn; ++o) {
      const char* at = a + (32 * bj[o] + l32) * lda + 64 * bi[o] + 8 * half;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const f16x4 h = *reinterpret_cast<const f16x4*>(at + 16 * q);
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const float r = fmaf(cb, to_f32(h[v]), cc * acc[o][4 * q + v]);
          acc[o][4 * q + v] = bi[o] == bj[o] && l32 == 8 * q + 4 * half + v ? r + ca : r;
        }
      }
    }
    __syncthreads();
    store_blocks();
    __syncthreads();
    // X' = d X + P X
    const bool last = step + 1 == p.steps;
    const float out = p.scale / p.up;
#pragma unroll
    for (int t = 0; t < S; ++t) {
      const int s = wave + t * kSmallWaves;
      if (s >= strips) continue;
      f16x8 col[2 * NB];
#pragma unroll
      for (int k = 0; k < 2 * NB; ++k) col[k] = columns_of(s, k);
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int v = 0; v < 16; ++v) own[t][b][v] *= kept;
#pragma unroll
      for (int k = 0; k < 2 * NB; ++k)
#pragma unroll
        for (int b = 0; b < NB; ++b)
          own[t][b] = __builtin_amdgcn_mfma_f32_32x32x16_f16(col[k], rows_of(a, lda, b, 16 * k),
                                                             own[t][b], 0, 0, 0);
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        if (!last) {
          store_own(t, b);
        } else {  // y, in X's place
          char* at = x + (32 * b + l32) * ldx + 64 * s + 8 * half;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const bf16x4 h = {from_f32<bf16>(own[t][b][4 * q] * out),
                              from_f32<bf16>(own[t][b][4 * q + 1] * out),
                              from_f32<bf16>(own[t][b][4 * q + 2] * out),
                              from_f32<bf16>(own[t][b][4 * q + 3] * out)};
            *reinterpret_cast<bf16x4*>(at + 16 * q) = h;
          }
        }
      }
    }
    __syncthreads();
  }
  // y, 16 bytes a lane
  constexpr int V = 8;
  bf16* y = p.y + origin;
  const int size = p.N * p.K;
  for (int i = tid * V; i < size; i += kSmallThreads * V) {
    bf16 h[V];
    Place at(i, p.N, p.K, ldx);
#pragma unroll
    for (int k = 0; k < V; ++k) {
      h[k] = *reinterpret_cast<const bf16*>(x + (i + k < size ? at.at : 0));
      at.step();
    }
    if (i + V <= size) {
      __builtin_memcpy(y + i, h, 16);
    } else {
#pragma unroll
      for (int k = 0; k < V; ++k)
        if (i + k < size) y[i + k] = h[k];
    }
  }
}

// d of each step. X's rounding in its null spaces still grows by the product of the |a|
// from a step on; while that is above kGrowth d is a (16: the usual coefficients' last
// two steps are below it).
constexpr float kGrowth = 16.f;
void kept_of(int steps, const float* coefficients, float* kept) {
  float growth = 1.f;
  for (int i = steps - 1; i >= 0; --i) {
    const float* c = coefficients + 3 * i;
    const float middle = c[0] + 0.5f * (c[1] + c[2]);
    growth *= fabsf(c[0]);
    kept[i] = growth <= kGrowth && fabsf(middle) < fabsf(c[0]) ? middle : c[0];
  }
}

constexpr int small_bytes(int m, int n) {
  const int mp = (m + 31) / 32 * 32, np = (n + 31) / 32 * 32;
  return mp * (small_row(mp) + small_row(np));
}
bool small_takes(int m, int n) {
  return m <= 32 * kSmallBlocks && n <= 16384 && small_bytes(m, n) <= kLargeBytes;
}

template <int NB>
void launch_blocks(const SmallParams& p, int E, int bytes, hipStream_t st) {
  if constexpr (small_bytes(32 * NB, 32 * NB) <= kSmallBytes)
    if (bytes <= kSmallBytes) {
      hipLaunchKernelGGL((ortho_small_kernel<NB, kSmallBytes>), dim3(E), dim3(kSmallThreads), 0, st,
                         p);
      return;
    }
  hipLaunchKernelGGL((ortho_small_kernel<NB, kLargeBytes>), dim3(E), dim3(kSmallThreads), 0, st,
                     p);
}

hipError_t launch_small(ElemType t, int E, int N, int K, const void* g, void* y, int steps,
                        const float* coefficients, float scale, float up, hipStream_t st) {
  SmallParams p{};
  p.g = g;
  p.y = static_cast<bf16*>(y);
  p.type = t;
  p.N = N;
  p.K = K;
  p.steps = steps;
  p.up = up;
  p.scale = scale;
  for (int i = 0; i < 3 * steps; ++i) p.c[i] = coefficients[i];
  kept_of(steps, coefficients, p.kept);
  const int m = N < K ? N : K, n = N < K ? K : N, bytes = small_bytes(m, n);
  switch ((m + 31) / 32) {
    case 1: launch_blocks<1>(p, E, bytes, st); break;
    case 2: launch_blocks<2>(p, E, bytes, st); break;
    case 3: launch_blocks<3>(p, E, bytes, st); break;
    case 4: launch_blocks<4>(p, E, bytes, st); break;
    case 5: launch_blocks<5>(p, E, bytes, st); break;
    default: launch_blocks<6>(p, E, bytes, st);
  }
  return hipGetLastError();
}

int64_t up64(int64_t v) { return (v + 63) / 64 * 64; }

// The workspace: sums of squares, X, X^T twice and its lo, A and P.
struct Layout {
  int64_t m, n, ldm, ldn;                   // ldm, ldn: row strides of m and n values
  int64_t x_size, t_size, a_size;           // elements of one matrix
  size_t parts, x, t[2], lo, a, q, total;   // bytes
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
    lo = take(E * t_size * 2);
    a = take(E * a_size * 2);
    q = take(E * a_size * 2);
    total = at;
  }
};

template <typename T>
hipError_t split(int E, int N, int K, const void* g, double scale, const Layout& L, char* ws,
                 hipStream_t st) {
  const int64_t size = (int64_t)N * K;
  int parts = (int)((size + 256 * 32 - 1) / (256 * 32));
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
  p.lo = ws + L.lo;
  p.lo_turned = wide;
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
  if (small_takes((int)L.m, (int)L.n))
    return launch_small(t, E, N, K, g, y, steps, coefficients, scale, up, st);
  hipError_t e = t == ElemType::kF32    ? split<float>(E, N, K, g, up, L, ws, st)
                 : t == ElemType::kBF16 ? split<bf16>(E, N, K, g, up, L, ws, st)
                                        : split<f16>(E, N, K, g, up, L, ws, st);
  const int m = (int)L.m, n = (int)L.n, m8 = (m + 7) & ~7, n8 = (n + 7) & ~7;
  float kept[kOrthoMaxSteps];
  kept_of(steps, coefficients, kept);
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
    // P = (a - d) I + b A + c A A
    p.act = p.w = ws + L.a;
    p.lda = p.ldw = L.ldm * 2;
    p.act_batch = p.w_batch = L.a_size * 2;
    p.cbytes = m8 * 2;
    p.out = p.turned = ws + L.q;
    p.alpha = c[2];
    p.beta = c[1];
    p.diag = c[0] - kept[i];
    if ((e = product<kPoly>(p, num_cus, st)) != hipSuccess) break;
    // X'^T = d X^T + X^T P
    p.act = ws + L.t[cur];
    p.act_batch = L.t_size * 2;
    p.w = ws + L.q;
    p.rows = n;
    p.keep = kept[i];
    p.lo = ws + L.lo;
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
