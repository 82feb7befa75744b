// Products over rows sorted by expert, and their gradients, for any sizes
// and strides (gfx950 matrix cores).
//
//   forward         y[i][n]  = sum_k x[i][k] w[e][n][k]
//   input gradient  dx[i][k] = sum_n dy[i][n] w[e][n][k]
//   weight gradient dw[e][n][k] = sum_i dy[i][n] x[i][k]
//
// for the rows i of expert e, offsets[e] <= i < offsets[e + 1]. All three
// are out[a][b] = sum_c P(c, a) Q(c, b): an operand either holds its
// contracted index c along its rows (x and w of the forward, dy of the input
// gradient) or down its columns (the others).
#include "ragged_device.hpp"
#include "ragged_operand.hpp"
#include "ragged_ring.hpp"

namespace moe {
namespace {

enum RaggedMode { kForward = 0, kInputGrad = 1, kWeightGrad = 2 };

struct RaggedParams {
  const void* p;  // rows a (forward: x; input gradient: dy; weight gradient: dy)
  const void* q;  // rows b (forward, input gradient: w; weight gradient: x)
  void* out;      // y, dx, or dw
  float* slots;   // weight gradient: partial sums of the chunks past the first
  const int32_t* offsets;
  int64_t ldp, ldq, ldo;  // elements
  int rows, E;
  int A, B, C;   // extents of a (weight gradient), b and c (forward, input gradient)
  int chunk;     // weight gradient: rows of a chunk
  int n_slots;   // weight gradient: slots of the workspace
  int accumulate;
  int tiles_b;   // tiles along b
  int tiles_a;   // weight gradient: tiles along a
};

// One step of a type over 32 bytes of c: 32 x 32 outputs, lane l supplies row
// l % 32 and 16 bytes of c, the first half of the step's for l < 32.
template <typename T>
struct Mma;
constexpr int kStepBytes = 32;
template <>
struct Mma<bf16> {
  typedef bf16x8 frag_t;
  __device__ static __forceinline__ f32x16 mma(frag_t a, frag_t b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
  }
};
template <>
struct Mma<f16> {
  typedef f16x8 frag_t;
  __device__ static __forceinline__ f32x16 mma(frag_t a, frag_t b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
  }
};
template <>
struct Mma<float> {
  typedef f32x4 frag_t;
  // instruction i takes c = i and 4 + i: a lane's values then are 16 adjacent
  // bytes, one LDS read where c lies along the row
  __device__ static __forceinline__ f32x16 mma(frag_t a, frag_t b, f32x16 c) {
#pragma unroll
    for (int i = 0; i < 4; ++i) c = __builtin_amdgcn_mfma_f32_32x32x2f32(a[i], b[i], c, 0, 0, 0);
    return c;
  }
};

typedef __attribute__((address_space(3))) char lds_char;
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

constexpr int kAhead = 2;    // stages of loads in flight

// One operand's share of a stage in LDS. Along: one LDS row per row, 16 bytes of
// padding. Down: one LDS row per c, kExt elements and 16 bytes of padding.
template <typename T, bool kAlong, int kExt, int kStage>
struct Operand : OperandLoads<T, kAlong, kExt, kStage> {
  typedef OperandLoads<T, kAlong, kExt, kStage> Loads;
  using Loads::kChunks;
  using Loads::kCk;
  using Loads::kEs;
  using Loads::kPieces;
  using typename Loads::regs_t;
  static constexpr int kPitch = (kAlong ? kStage : kExt * kEs) + 16;
  static constexpr int kBytes = kAlong ? kExt * kPitch : kCk * kPitch;

  __device__ static __forceinline__ void store(const regs_t& reg, char* lds) {
#pragma unroll
    for (int u = 0; u < kPieces; ++u) {
      const int id = (int)threadIdx.x + 256 * u;
      int off;
      if constexpr (kAlong) {
        off = (id / kChunks) * kPitch + (id % kChunks) * 16;
      } else {
        constexpr int kPer = kExt * kEs / 16;
        off = (id / kPer) * kPitch + (id % kPer) * 16;
      }
      *reinterpret_cast<u32x4*>(lds + off) = reg[u];
    }
  }
  // this lane's fragment of MFMA step s, rows row0 .. row0 + 31
  __device__ static __forceinline__ typename Mma<T>::frag_t frag(const char* lds, int row0,
                                                                 int s) {
    const int lane = threadIdx.x & 63, l32 = lane & 31, half = lane >> 5;
    typedef typename Mma<T>::frag_t frag_t;
    if constexpr (kAlong) {
      return *reinterpret_cast<const frag_t*>(lds + (row0 + l32) * kPitch + s * kStepBytes +
                                              half * 16);
    } else if constexpr (kEs == 4) {
      frag_t f;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        f[i] = *reinterpret_cast<const float*>(lds + (8 * s + 4 * half + i) * kPitch +
                                               (row0 + l32) * 4);
      return f;
    } else {
      // transposing LDS read: in each group of 16 lanes, lane i receives
      // 16-bit element i % 4 of the 8 bytes addressed by lanes 4 j + i / 4,
      // j = 0..3, so lane i gets row i of the group at four consecutive c
      const int grp = lane >> 4, gj = (lane >> 2) & 3, gq = lane & 3;
      const int c = 16 * s + 8 * (grp >> 1) + gj;
      const char* at = lds + c * kPitch + (row0 + 16 * (grp & 1) + 4 * gq) * 2;
      const s16x4 lo =
          __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(lds_char*)at);
      const s16x4 hi =
          __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(lds_char*)(at + 4 * kPitch));
      return __builtin_bit_cast(frag_t, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    }
  }
};

// General kernel: one workgroup per output tile, of 128 x 128 or 64 x 64 with 2
// x 2 wavefronts of W x W blocks of 32 x 32. Stages of 128 bytes of c go through
// registers into two LDS buffers, the loads of the next two stages in flight
// while one is multiplied. Takes every size, stride and element alignment.
// Whole stages run without a bounds check; the partial one (split_stages) goes
// first and shifts what it loads at the ends of rows. 32768 rows, N = K = 2049, 8
// experts, fp16: 490-532 us, 515-560 TFLOP/s (with 64-byte stages or one stage
// ahead 10-20% more); what bounds it is LDS, which the 64 x 64 wavefront tiles read 1
// KiB of per 32 x 32 x 16 product, and the barrier of each stage. 5002 rows, N
// = 777, K = 1111, fp16: 31-33 us by how unevenly the rows fall (with the
// partial stage last and its ends loaded an element at a time 35.5, where this
// takes 31.1); K = 1104 in aligned rows, on the ring, takes 27. fp32, 20480 rows,
// 5 experts, N = 192, K = 2240: 161 us, 109 TFLOP/s; 8192 rows of 4 of 2048 x
// 2048: 527 us, 130 TFLOP/s.
//
// Where there are few outputs a tile is 32 x 32, so that more CUs have one, and
// its four wavefronts share c: each takes every fourth step of a stage (of
// 512 bytes), and their sums are joined in LDS, in wavefront order.
template <typename T, int kMode, int kTile>
__global__ __launch_bounds__(256, kTile == 64 ? 4 : 2) void ragged_general_kernel(RaggedParams p) {
  constexpr bool kSplit = kTile == 32;
  constexpr int W = kSplit ? 1 : kTile / 64;
  constexpr int kStage = kSplit ? 512 : 128;  // bytes of c
  constexpr bool kPAlong = kMode != kWeightGrad;
  constexpr bool kQAlong = kMode == kForward;
  typedef Operand<T, kPAlong, kTile, kStage> P_t;
  typedef Operand<T, kQAlong, kTile, kStage> Q_t;
  constexpr int kCk = P_t::kCk;
  __shared__ __attribute__((aligned(16))) char lds[2][P_t::kBytes + Q_t::kBytes];

  const int per = kMode == kWeightGrad ? p.tiles_a * p.tiles_b : p.tiles_b;
  auto units = [&](int rows) {
    if constexpr (kMode == kWeightGrad) {
      // an expert without rows still stores its zeros
      const int n = (int)(((int64_t)rows + p.chunk - 1) / p.chunk);
      return (n == 0 && !p.accumulate ? 1 : n) * per;
    } else {
      return (int)(((int64_t)rows + kTile - 1) / kTile) * per;
    }
  };
  // Each XCD (workgroups b % 8) takes a contiguous eighth of the tiles: it
  // then reads an eighth of the rows, and the weights of few experts.
  ExpertUnit u;
  int t = 0;
  if (!find_xcd_unit(p.offsets, p.E, p.rows, units, &t, &u)) return;
  const int local = t - u.first, tid = threadIdx.x;

  P_t P;
  Q_t Q;
  int c_begin = 0, c_end, a0, b0, a_ext, part = 0;
  if constexpr (kMode == kWeightGrad) {
    part = local / per;
    a0 = (local % per) / p.tiles_b * kTile;
    b0 = (local % per) % p.tiles_b * kTile;
    c_begin = part * p.chunk;
    c_end = u.rows - c_begin < p.chunk ? u.rows : c_begin + p.chunk;
    a_ext = p.A - a0;
    P.set(static_cast<const T*>(p.p) + (int64_t)u.start * p.ldp + a0, p.ldp, a_ext, a0, tid);
    Q.set(static_cast<const T*>(p.q) + (int64_t)u.start * p.ldq + b0, p.ldq, p.B - b0, b0, tid);
  } else {
    a0 = local / p.tiles_b * kTile;
    b0 = local % p.tiles_b * kTile;
    c_end = p.C;
    a_ext = u.rows - a0;
    P.set(static_cast<const T*>(p.p) + ((int64_t)u.start + a0) * p.ldp, p.ldp, a_ext, a0,
          tid);
    Q.set(static_cast<const T*>(p.q) + (int64_t)u.e * p.B * p.C +
              (kMode == kForward ? (int64_t)b0 * p.ldq : (int64_t)b0),
          p.ldq, p.B - b0, b0, tid);
  }

  // weight gradient: the slot of this chunk (past the last one only if the
  // offsets overlap: then it is not stored)
  int slot = 0;
  if (kMode == kWeightGrad && part > 0) {
    slot = slots_before(p.offsets, u.e, p.rows, p.chunk) + part - 1;
    if ((uint32_t)slot >= (uint32_t)p.n_slots) return;
  }
  const int wave = threadIdx.x >> 6;
  const int wa = kSplit ? 0 : (wave >> 1) * 32 * W, wb = kSplit ? 0 : (wave & 1) * 32 * W;
  f32x16 acc[W][W];
#pragma unroll
  for (int i = 0; i < W; ++i)
#pragma unroll
    for (int j = 0; j < W; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.f;

  auto step = [&](const char* buf, int s) {
    typename Mma<T>::frag_t fa[W], fb[W];
#pragma unroll
    for (int i = 0; i < W; ++i) fa[i] = P_t::frag(buf, wa + 32 * i, s);
#pragma unroll
    for (int j = 0; j < W; ++j) fb[j] = Q_t::frag(buf + P_t::kBytes, wb + 32 * j, s);
#pragma unroll
    for (int i = 0; i < W; ++i)
#pragma unroll
      for (int j = 0; j < W; ++j) acc[i][j] = Mma<T>::mma(fa[i], fb[j], acc[i][j]);
  };
  constexpr int kSteps = kStage / kStepBytes;
  auto multiply = [&](const char* buf) {
    if constexpr (kSplit) {
#pragma unroll
      for (int s = 0; s < kSteps; s += 4) step(buf, s + wave);
    } else {
#pragma unroll
      for (int s = 0; s < kSteps; ++s) step(buf, s);
    }
  };
  // the stages that are checked go first, so that their loads are as far ahead
  // as the others'
  const StageSplit split = split_stages(c_end - c_begin, kCk, P.keep > Q.keep ? P.keep : Q.keep);
  const int rest = split.checked, stages = split.whole + rest;
  static_assert(kAhead == 2, "the checked stages' loads are the first two");
  typename P_t::regs_t p0, p1;
  typename Q_t::regs_t q0, q1;
  auto load = [&](int i, typename P_t::regs_t& rp, typename Q_t::regs_t& rq) {
    P.load(rp, c_begin + (i - rest) * kCk);
    Q.load(rq, c_begin + (i - rest) * kCk);
  };
  auto load_some = [&](int i, typename P_t::regs_t& rp, typename Q_t::regs_t& rq) {
    P.load_some(rp, c_begin + (split.whole + i) * kCk, c_end, tid);
    Q.load_some(rq, c_begin + (split.whole + i) * kCk, c_end, tid);
  };
  // stage i from its registers into LDS buffer i % 2, the loads of stage i +
  // kAhead into them, and its products. The buffer's last readers passed the
  // barrier of the stage between.
  auto stage = [&](int i, int buf, typename P_t::regs_t& rp, typename Q_t::regs_t& rq) {
    P_t::store(rp, lds[buf]);
    Q_t::store(rq, lds[buf] + P_t::kBytes);
    __syncthreads();
    if (i + kAhead < stages) load(i + kAhead, rp, rq);
    multiply(lds[buf]);
  };
  if (rest > 0)
    load_some(0, p0, q0);
  else if (stages > 0)
    load(0, p0, q0);
  if (rest > 1)
    load_some(1, p1, q1);
  else if (stages > 1)
    load(1, p1, q1);
  for (int i = 0; i < stages; i += 2) {
    stage(i, 0, p0, q0);
    if (i + 1 < stages) stage(i + 1, 1, p1, q1);
  }

  // lane: column b = l % 32 of a block, rows a = 8 (v / 4) + 4 (l / 32) + v % 4
  const int lane = threadIdx.x & 63, l32 = lane & 31, half = lane >> 5;
  auto put = [&](int da, int b, float r) {
    if (da >= a_ext) return;
    if constexpr (kMode == kWeightGrad) {
      if (part == 0) {
        float* o = static_cast<float*>(p.out) + ((int64_t)u.e * p.A + a0 + da) * p.B + b;
        *o = p.accumulate ? *o + r : r;
      } else {
        p.slots[((int64_t)slot * p.A + a0 + da) * p.B + b] = r;
      }
    } else {
      static_cast<T*>(p.out)[((int64_t)u.start + a0 + da) * p.ldo + b] = from_f32<T>(r);
    }
  };
  if constexpr (kSplit) {
    // wavefront w joins and stores rows 8 w .. 8 w + 7: values 4 w .. 4 w + 3
    float(*joined)[16][64] = reinterpret_cast<float(*)[16][64]>(&lds[0][0]);
    static_assert(sizeof(lds) >= 4 * 16 * 64 * 4, "");
    __syncthreads();
#pragma unroll
    for (int v = 0; v < 16; ++v) joined[wave][v][lane] = acc[0][0][v];
    __syncthreads();
    if (b0 + l32 >= p.B) return;
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      float r = 0.f;
#pragma unroll
      for (int w = 0; w < 4; ++w) r += joined[w][4 * wave + v][lane];
      put(8 * wave + 4 * half + v, b0 + l32, r);
    }
  } else {
#pragma unroll
    for (int i = 0; i < W; ++i) {
#pragma unroll
      for (int j = 0; j < W; ++j) {
        const int b = b0 + wb + 32 * j + l32;
        if (b >= p.B) continue;
#pragma unroll
        for (int v = 0; v < 16; ++v)
          put(wa + 32 * i + 8 * (v >> 2) + 4 * half + (v & 3), b, acc[i][j][v]);
      }
    }
  }
}

// Adds the slots of every expert that has any to dw, in chunk order. The
// workgroups share [N][K] of each such expert (found 64 experts at a time).
// V: floats per lane and step.
template <int V>
__global__ __launch_bounds__(256) void ragged_add_slots_kernel(RaggedParams p) {
  typedef float vec_t __attribute__((ext_vector_type(V)));
  const int64_t n = (int64_t)p.A * p.B / V;
  const int lane = threadIdx.x & 63;
  int before = 0;  // slots of the experts below
  uint32_t turn = 0;  // experts with slots so far
  for (int base = 0; base < p.E; base += kWave) {
    int start, rows = 0, own = 0;
    if (base + lane < p.E) {
      expert_rows(p.offsets, base + lane, p.rows, &start, &rows);
      own = rows > 0 ? (int)(((int64_t)rows + p.chunk - 1) / p.chunk) - 1 : 0;
    }
    const int incl = wave_inclusive_scan(own) + before;
    before = __builtin_amdgcn_readlane(incl, kWave - 1);
    if ((uint32_t)before > (uint32_t)p.n_slots) return;  // overlapping offsets
    uint64_t todo = __builtin_amdgcn_ballot_w64(own > 0);
    while (todo) {
      const int l = __builtin_ctzll(todo);
      todo &= todo - 1;
      if (turn++ % gridDim.y != blockIdx.y) continue;
      const int last = __builtin_amdgcn_readlane(incl, l);
      const int first = last - __builtin_amdgcn_readlane(own, l);
      const int count = last - first;
      vec_t* o = static_cast<vec_t*>(p.out) + (base + l) * n;
      const vec_t* s = reinterpret_cast<const vec_t*>(p.slots) + first * n;
      for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n;
           i += (int64_t)gridDim.x * 256) {
        vec_t r = o[i];
#pragma unroll 4
        for (int k = 0; k < count; ++k) r += s[k * n + i];
        o[i] = r;
      }
    }
  }
}

int ceil_div(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }

// Tile of the general kernel: 128 x 128 unless the outputs are too few to
// give every CU two; 32 x 32 where all tiles run at once (two fit a CU).
// 32 x 32 against 64 x 64: fp32, 1024 rows of 4 experts, N = 256, K = 2047
// (288 tiles of 32 x 32) 30 and 48 us, 846 rows of one expert, N = 128, K =
// 2496 (108) 21 and 54; fp16, 300 rows of 4, N = 2001, K = 1500 (819) 20 and
// 16, 64 rows of 4, N = 512, K = 511 (96) 7 and 7.
constexpr int kLargeJobs = 2, kSmallJobs = 2;

// Tiles of the forward or the input gradient at most, over B outputs a row:
// every expert's last one may be partial.
int64_t product_tiles(int64_t rows, int64_t E, int B, int tile) {
  return (rows / tile + (rows < E ? rows : E)) * ceil_div(B, tile);
}

template <typename T, int kMode>
hipError_t launch_general(RaggedParams p, int num_cus, hipStream_t st) {
  auto jobs = [&](int tile) -> int64_t {
    p.tiles_b = ceil_div(p.B, tile);
    p.tiles_a = ceil_div(p.A, tile);
    // the most units that offsets can make
    if (kMode == kWeightGrad)
      return ((int64_t)p.rows / p.chunk + p.E) * p.tiles_a * p.tiles_b;
    return product_tiles(p.rows, p.E, p.B, tile);
  };
  // (rounded up to whole turns over the XCDs)
  const int64_t large = (jobs(128) + 7) / 8 * 8;
  if (large >= kLargeJobs * (int64_t)num_cus) {
    hipLaunchKernelGGL((ragged_general_kernel<T, kMode, 128>), dim3((unsigned)large), dim3(256),
                       0, st, p);
    return hipGetLastError();
  }
  const int64_t small = (jobs(32) + 7) / 8 * 8;
  if (small <= kSmallJobs * (int64_t)num_cus) {
    hipLaunchKernelGGL((ragged_general_kernel<T, kMode, 32>), dim3((unsigned)small), dim3(256),
                       0, st, p);
    return hipGetLastError();
  }
  const int64_t medium = (jobs(64) + 7) / 8 * 8;
  hipLaunchKernelGGL((ragged_general_kernel<T, kMode, 64>), dim3((unsigned)medium), dim3(256), 0,
                     st, p);
  return hipGetLastError();
}

template <int kMode>
hipError_t dispatch(ElemType t, const RaggedParams& p, int num_cus, hipStream_t st) {
  switch (t) {
    case ElemType::kF32: return launch_general<float, kMode>(p, num_cus, st);
    case ElemType::kBF16: return launch_general<bf16, kMode>(p, num_cus, st);
    default: return launch_general<f16, kMode>(p, num_cus, st);
  }
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// The ring kernel takes 16-bit rows of whole 16-byte chunks; the output may
// have any alignment.
bool ring_takes(const RaggedShape& s, const void* act, int64_t ld, const void* w, int c) {
  return s.type != ElemType::kF32 && c % 8 == 0 && s.K % 8 == 0 && ld % 8 == 0 &&
         aligned16(act) && aligned16(w);
}

RingParams ring_params(const RaggedShape& s, const int32_t* offsets, const void* act, int64_t ld,
                       const void* w, void* out, int64_t ldo, int c, int b) {
  RingParams r{};
  r.act = static_cast<const char*>(act);
  r.w = static_cast<const char*>(w);
  r.out = static_cast<char*>(out);
  r.offsets = offsets;
  r.lda = ld * 2;
  r.ldw = (int64_t)s.K * 2;
  r.ldo = ldo * 2;
  r.wbytes = (int64_t)s.N * s.K * 2;
  r.rows = (int)s.rows;
  r.E = s.E;
  r.B = b;
  r.C = c;
  r.cbytes = c * 2;
  r.out_vec = b % 8 == 0 && ldo % 8 == 0 && aligned16(out);
  return r;
}

RaggedParams base_params(const RaggedShape& s, const int32_t* offsets) {
  RaggedParams p{};
  p.offsets = offsets;
  p.rows = (int)s.rows;
  p.E = s.E;
  return p;
}

}  // namespace

// Chunks: an expert's tiles run at once, so a chunk may hold half of the rows
// that a CU sums in all (rows * tiles / 256), or an expert with many rows
// holds up the launch. A chunk past the first costs a write and a read of
// [N][K] in fp32 against 2 N K flops a row: 512 rows at least (8192 rows of 8
// experts with N = K = 512: 46 us with chunks of 512, 59 with 128; 65536 rows of
// 64 with N = K = 256: 36 and 63). Few rows in fp32, whose products take eight
// times as long, may go down to 128 where [N][K] is one tile: 2048 rows of 16
// uneven experts with N = K = 256 take 22 us with 512 and 13 with 128, 4096 of 64
// 32 and 25, 4096 of 8 even ones 17 and 18; but 16384 of 64 even ones 27 and 40,
// and bf16 at 2048 of 16 uneven ones 10.3 and 9.6, at 2048 of 4 even ones 7.1 and
// 10.1. A function of the shape alone: it fixes the order of the sums.
DwSplit dw_split(const RaggedShape& s) {
  const int64_t tiles = (int64_t)ceil_div(s.N, 256) * ceil_div(s.K, 256);
  const bool few = s.type == ElemType::kF32 && tiles == 1 && s.rows <= 4096;
  const int64_t least = few ? 128 : 512;
  int64_t chunk = (s.rows * tiles + 511) / 512;
  chunk = chunk < least ? least : (chunk + 63) / 64 * 64;
  // a chunk's rows are addressed with 32-bit byte offsets
  const int64_t ld = (s.ld_x > s.ld_y ? s.ld_x : s.ld_y) * elem_bytes(s.type);
  const int64_t most = (((int64_t)1 << 31) - 1) / ld / 64 * 64;
  if (chunk > most) chunk = most;
  return DwSplit{chunk, s.rows / chunk};
}

hipError_t launch_ragged_gemm(const RaggedShape& s, const int32_t* offsets, const void* x,
                              const void* w, void* y, int num_cus, hipStream_t st) {
  if (s.rows == 0) return hipSuccess;
  if (ring_takes(s, x, s.ld_x, w, s.K))
    return launch_ring(
        s.type == ElemType::kBF16 ? RingKind::kForwardBF16 : RingKind::kForwardF16,
        ring_params(s, offsets, x, s.ld_x, w, y, s.ld_y, s.K, s.N), num_cus, st);
  RaggedParams p = base_params(s, offsets);
  p.p = x;
  p.q = w;
  p.out = y;
  p.ldp = s.ld_x;
  p.ldq = s.K;
  p.ldo = s.ld_y;
  p.B = s.N;
  p.C = s.K;
  return dispatch<kForward>(s.type, p, num_cus, st);
}

hipError_t launch_ragged_dx(const RaggedShape& s, const int32_t* offsets, const void* dy,
                            const void* w, void* dx, int num_cus, hipStream_t st) {
  if (s.rows == 0) return hipSuccess;
  // few outputs: the general kernel's 32 x 32 tiles. bf16, ring against them: 8
  // rows, E 4, N = K = 2048 17 and 9 us, 1024 rows of one expert, N = 4096, K =
  // 256 (264 tiles) 23 and 13; 512 rows, E 64, N = K = 512 (1280) 7.8 and 8.0.
  if (ring_takes(s, dy, s.ld_y, w, s.N) &&
      product_tiles(s.rows, s.E, s.K, 32) > kSmallJobs * (int64_t)num_cus)
    return launch_ring(
        s.type == ElemType::kBF16 ? RingKind::kInputGradBF16 : RingKind::kInputGradF16,
        ring_params(s, offsets, dy, s.ld_y, w, dx, s.ld_x, s.N, s.K), num_cus, st);
  RaggedParams p = base_params(s, offsets);
  p.p = dy;
  p.q = w;
  p.out = dx;
  p.ldp = s.ld_y;
  p.ldq = s.K;
  p.ldo = s.ld_x;
  p.B = s.K;
  p.C = s.N;
  return dispatch<kInputGrad>(s.type, p, num_cus, st);
}

hipError_t launch_ragged_dw(const RaggedShape& s, const int32_t* offsets, const void* x,
                            const void* dy, float* dw, float* slots, bool accumulate,
                            int num_cus, hipStream_t st) {
  const DwSplit split = dw_split(s);
  RaggedParams p = base_params(s, offsets);
  p.p = dy;
  p.q = x;
  p.out = dw;
  p.slots = slots;
  p.ldp = s.ld_y;
  p.ldq = s.ld_x;
  p.A = s.N;
  p.B = s.K;
  p.chunk = (int)split.chunk;
  p.n_slots = (int)split.slots;
  p.accumulate = accumulate ? 1 : 0;
  hipError_t e;
  // The ring where it has a 256 x 256 tile for every CU (at the mean rows of an
  // expert); fewer go to the general kernel's smaller ones. bf16, ring against
  // general: 16384 rows, E 64, N = K = 512 (256 tiles) 27 and 32 us, E 4 (128)
  // 45 and 34, 4096 rows, E 8, N = K = 1024 (128) 32 and 26, 2792 rows, E 4,
  // N = 448, K = 128 (10) 23 and 11.
  const int64_t chunks = s.rows / split.chunk;
  const int64_t tiles = (chunks > s.E ? chunks : s.E) * ceil_div(s.N, 256) * ceil_div(s.K, 256);
  if (s.type != ElemType::kF32 && s.rows > 0 && tiles >= num_cus && s.ld_x % 8 == 0 &&
      s.ld_y % 8 == 0 && aligned16(x) && aligned16(dy)) {
    const WgradRingParams r{static_cast<const char*>(dy), static_cast<const char*>(x), dw, slots,
                            offsets, s.ld_y * 2, s.ld_x * 2, (int)s.rows, s.E, s.N, s.K,
                            p.chunk, p.n_slots, p.accumulate, 1};
    e = launch_wgrad_ring(s.type == ElemType::kBF16, r, num_cus, st);
  } else {
    e = dispatch<kWeightGrad>(s.type, p, num_cus, st);
  }
  if (e != hipSuccess || split.slots == 0) return e;
  const bool vec = (int64_t)s.N * s.K % 4 == 0 && aligned16(dw);
  const int most = num_cus * 8, blocks = ceil_div((int64_t)s.N * s.K, vec ? 1024 : 256);
  // and y over the experts with slots, where [N][K] is small
  const int gx = blocks < most ? blocks : most;
  const dim3 grid(gx, gx < num_cus ? (s.E < 8 ? s.E : 8) : 1);
  if (vec)
    hipLaunchKernelGGL((ragged_add_slots_kernel<4>), grid, dim3(256), 0, st, p);
  else
    hipLaunchKernelGGL((ragged_add_slots_kernel<1>), grid, dim3(256), 0, st, p);
  return hipGetLastError();
}

}  // namespace moe
