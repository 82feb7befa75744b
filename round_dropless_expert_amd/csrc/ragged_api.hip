// C ABI of the ragged expert operators: argument checks and launches. No
// call allocates, waits or keeps state, so every one of them can be captured
// into a graph.
#include "api_common.hpp"
#include "ragged.hpp"

namespace {

using moe::api_fail;
using moe::ElemType;

constexpr int64_t k2G = int64_t(1) << 31;
// Output tiles of one launch (of 128 x 128): its grid's threads stay below 2^32.
constexpr int64_t kMaxTiles = int64_t(1) << 23;

int64_t div_up(int64_t a, int64_t b) { return (a + b - 1) / b; }

moe_status_t check_dtype(int32_t dtype, ElemType* out) {
  switch (dtype) {
    case MOE_F32: *out = ElemType::kF32; return MOE_OK;
    case MOE_BF16: *out = ElemType::kBF16; return MOE_OK;
    case MOE_F16: *out = ElemType::kF16; return MOE_OK;
  }
  return api_fail(MOE_ERR_INVALID_ARGUMENT, "unknown dtype");
}

moe_status_t check_ptr(const void* p, const char* name, size_t align) {
  if (!p) return api_fail(MOE_ERR_INVALID_ARGUMENT, "is NULL", name);
  if (reinterpret_cast<uintptr_t>(p) % align)
    return api_fail(MOE_ERR_INVALID_ARGUMENT,
                    align == 16 ? "must be 16-byte aligned" : "must be aligned to its element",
                    name);
  return MOE_OK;
}

// A leading dimension (0: the width) of rows of `width` elements.
moe_status_t check_ld(int64_t ld, int64_t width, const char* name, int64_t* out) {
  *out = ld == 0 ? width : ld;
  if (*out < width)
    return api_fail(MOE_ERR_INVALID_ARGUMENT, "is below the row's width (0 means the width)",
                    name);
  if (*out > moe::kRaggedMaxWidth)
    return api_fail(MOE_ERR_UNSUPPORTED, "is above 2^20 elements", name);
  return MOE_OK;
}

moe_status_t check_grouped(const moe_grouped_t* g, moe::RaggedShape* s) {
  if (!g) return api_fail(MOE_ERR_INVALID_ARGUMENT, "config is NULL");
  if (g->rows < 0) return api_fail(MOE_ERR_INVALID_ARGUMENT, "rows must be >= 0");
  if (g->E < 1) return api_fail(MOE_ERR_INVALID_ARGUMENT, "E must be >= 1");
  if (g->N < 1 || g->K < 1) return api_fail(MOE_ERR_INVALID_ARGUMENT, "N and K must be >= 1");
  moe_status_t st = check_dtype(g->dtype, &s->type);
  if (st != MOE_OK) return st;
  if (g->E > moe::kRaggedMaxExperts)
    return api_fail(MOE_ERR_UNSUPPORTED, "E > 1024 is not supported");
  if (g->rows >= k2G) return api_fail(MOE_ERR_UNSUPPORTED, "rows must be < 2^31");
  if ((st = check_ld(g->ld_x, g->K, "ld_x", &s->ld_x)) != MOE_OK) return st;
  if ((st = check_ld(g->ld_y, g->N, "ld_y", &s->ld_y)) != MOE_OK) return st;
  // fp32 for every type: the weight gradient's matrices are fp32
  if ((int64_t)g->N * g->K * 4 >= k2G)
    return api_fail(MOE_ERR_UNSUPPORTED, "N*K must be < 2^29");
  const int64_t tn = div_up(g->N, 128), tk = div_up(g->K, 128);
  s->rows = g->rows;
  s->E = g->E;
  s->N = g->N;
  s->K = g->K;
  if ((g->rows / 128 + g->E) * (tn > tk ? tn : tk) >= kMaxTiles ||
      (moe::dw_split(*s).slots + g->E) * tn * tk >= kMaxTiles)
    return api_fail(MOE_ERR_UNSUPPORTED, "more than 2^23 output tiles of 128 x 128");
  return MOE_OK;
}

size_t dw_bytes(const moe::RaggedShape& s) {
  return (size_t)moe::dw_split(s).slots * (size_t)s.N * (size_t)s.K * 4;
}

moe_status_t check_rows(int64_t rows, int64_t width) {
  if (rows < 0) return api_fail(MOE_ERR_INVALID_ARGUMENT, "rows must be >= 0");
  if (width < 1) return api_fail(MOE_ERR_INVALID_ARGUMENT, "the row's width must be >= 1");
  if (rows >= k2G) return api_fail(MOE_ERR_UNSUPPORTED, "rows must be < 2^31");
  if (width > moe::kRaggedMaxWidth)
    return api_fail(MOE_ERR_UNSUPPORTED, "the row's width is above 2^20 elements");
  return MOE_OK;
}

moe_status_t check_mx_width(int64_t K) {
  if (K % MOE_MXFP4_BLOCK)
    return api_fail(MOE_ERR_INVALID_ARGUMENT, "K must be a multiple of 32");
  return MOE_OK;
}

#define MOE_TRY(call)                    \
  do {                                   \
    const moe_status_t _s = (call);      \
    if (_s != MOE_OK) return _s;         \
  } while (0)

#define MOE_LAUNCH(call, where)                                      \
  do {                                                               \
    const hipError_t _e = (call);                                    \
    return _e == hipSuccess ? MOE_OK : moe::api_hip_fail(_e, where); \
  } while (0)

}  // namespace

extern "C" {

moe_status_t moe_grouped_gemm(const moe_grouped_t* g, const int32_t* offsets, const void* x,
                              const void* w, void* y, void* stream) {
  moe::RaggedShape s;
  MOE_TRY(check_grouped(g, &s));
  if (s.rows == 0) return MOE_OK;
  const size_t es = (size_t)moe::elem_bytes(s.type);
  MOE_TRY(check_ptr(offsets, "offsets", 4));
  MOE_TRY(check_ptr(x, "x", es));
  MOE_TRY(check_ptr(w, "w", es));
  MOE_TRY(check_ptr(y, "y", es));
  int cus = 0;
  MOE_TRY(moe::api_num_cus(&cus));
  MOE_LAUNCH(moe::launch_ragged_gemm(s, offsets, x, w, y, cus, static_cast<hipStream_t>(stream)),
             "grouped product launch");
}

moe_status_t moe_grouped_gemm_dx(const moe_grouped_t* g, const int32_t* offsets, const void* dy,
                                 const void* w, void* dx, void* stream) {
  moe::RaggedShape s;
  MOE_TRY(check_grouped(g, &s));
  if (s.rows == 0) return MOE_OK;
  const size_t es = (size_t)moe::elem_bytes(s.type);
  MOE_TRY(check_ptr(offsets, "offsets", 4));
  MOE_TRY(check_ptr(dy, "dy", es));
  MOE_TRY(check_ptr(w, "w", es));
  MOE_TRY(check_ptr(dx, "dx", es));
  int cus = 0;
  MOE_TRY(moe::api_num_cus(&cus));
  MOE_LAUNCH(moe::launch_ragged_dx(s, offsets, dy, w, dx, cus, static_cast<hipStream_t>(stream)),
             "grouped input gradient launch");
}

moe_status_t moe_grouped_dw_workspace_size(const moe_grouped_t* g, size_t* bytes) {
  moe::RaggedShape s;
  MOE_TRY(check_grouped(g, &s));
  if (!bytes) return api_fail(MOE_ERR_INVALID_ARGUMENT, "bytes is NULL");
  *bytes = dw_bytes(s);
  return MOE_OK;
}

moe_status_t moe_grouped_gemm_dw(const moe_grouped_t* g, const int32_t* offsets, const void* x,
                                 const void* dy, float* dw, int32_t accumulate, void* ws,
                                 size_t ws_bytes, void* stream) {
  moe::RaggedShape s;
  MOE_TRY(check_grouped(g, &s));
  if (accumulate != 0 && accumulate != 1)
    return api_fail(MOE_ERR_INVALID_ARGUMENT, "accumulate must be 0 or 1");
  const size_t es = (size_t)moe::elem_bytes(s.type);
  MOE_TRY(check_ptr(offsets, "offsets", 4));
  if (s.rows > 0) {
    MOE_TRY(check_ptr(x, "x", es));
    MOE_TRY(check_ptr(dy, "dy", es));
  }
  MOE_TRY(check_ptr(dw, "dw", 4));
  const size_t need = dw_bytes(s);
  if (need > 0) {
    MOE_TRY(check_ptr(ws, "workspace", 16));
    if (ws_bytes < need) return api_fail(MOE_ERR_WORKSPACE_TOO_SMALL, "workspace too small");
  }
  int cus = 0;
  MOE_TRY(moe::api_num_cus(&cus));
  MOE_LAUNCH(moe::launch_ragged_dw(s, offsets, x, dy, dw, static_cast<float*>(ws),
                                   accumulate != 0, cus, static_cast<hipStream_t>(stream)),
             "grouped weight gradient launch");
}

moe_status_t moe_swiglu(int32_t dtype, int64_t rows, int64_t f, const void* gu, int64_t ld_gu,
                        void* h, int64_t ld_h, const int32_t* n_rows, void* stream) {
  ElemType t;
  MOE_TRY(check_dtype(dtype, &t));
  MOE_TRY(check_rows(rows, f));
  MOE_TRY(check_ld(ld_gu, 2 * f, "ld_gu", &ld_gu));
  MOE_TRY(check_ld(ld_h, f, "ld_h", &ld_h));
  if (rows == 0) return MOE_OK;
  const size_t es = (size_t)moe::elem_bytes(t);
  MOE_TRY(check_ptr(gu, "gu", es));
  MOE_TRY(check_ptr(h, "h", es));
  if (n_rows) MOE_TRY(check_ptr(n_rows, "n_rows", 4));
  int cus = 0;
  MOE_TRY(moe::api_num_cus(&cus));
  MOE_LAUNCH(moe::launch_swiglu(t, rows, f, gu, ld_gu, h, ld_h, n_rows, cus,
                                static_cast<hipStream_t>(stream)),
             "SwiGLU launch");
}

moe_status_t moe_swiglu_backward(int32_t dtype, int64_t rows, int64_t f, const void* gu,
                                 int64_t ld_gu, const void* dh, int64_t ld_dh, void* dgu,
                                 int64_t ld_dgu, const int32_t* n_rows, void* stream) {
  ElemType t;
  MOE_TRY(check_dtype(dtype, &t));
  MOE_TRY(check_rows(rows, f));
  MOE_TRY(check_ld(ld_gu, 2 * f, "ld_gu", &ld_gu));
  MOE_TRY(check_ld(ld_dh, f, "ld_dh", &ld_dh));
  MOE_TRY(check_ld(ld_dgu, 2 * f, "ld_dgu", &ld_dgu));
  if (rows == 0) return MOE_OK;
  const size_t es = (size_t)moe::elem_bytes(t);
  MOE_TRY(check_ptr(gu, "gu", es));
  MOE_TRY(check_ptr(dh, "dh", es));
  MOE_TRY(check_ptr(dgu, "dgu", es));
  if (n_rows) MOE_TRY(check_ptr(n_rows, "n_rows", 4));
  int cus = 0;
  MOE_TRY(moe::api_num_cus(&cus));
  MOE_LAUNCH(moe::launch_swiglu_backward(t, rows, f, gu, ld_gu, dh, ld_dh, dgu, ld_dgu, n_rows,
                                         cus, static_cast<hipStream_t>(stream)),
             "SwiGLU gradient launch");
}

int64_t moe_mxfp4_scale_stride(int64_t K) {
  return K < MOE_MXFP4_BLOCK || K % MOE_MXFP4_BLOCK ? -1 : moe::mx_scale_stride(K);
}

moe_status_t moe_mxfp4_quantize(int32_t dtype, int64_t rows, int64_t K, const void* x,
                                int64_t ld_x, int64_t src_rows, const int32_t* index,
                                int32_t index_div, const int32_t* n_rows, uint8_t* codes,
                                uint8_t* scales, void* stream) {
  ElemType t;
  MOE_TRY(check_dtype(dtype, &t));
  MOE_TRY(check_rows(rows, K));
  MOE_TRY(check_mx_width(K));
  MOE_TRY(check_ld(ld_x, K, "ld_x", &ld_x));
  if (index) {
    if (src_rows < 0) return api_fail(MOE_ERR_INVALID_ARGUMENT, "src_rows must be >= 0");
    if (index_div < 1) return api_fail(MOE_ERR_INVALID_ARGUMENT, "index_div must be >= 1");
    MOE_TRY(check_ptr(index, "index", 4));
  }
  if (rows == 0) return MOE_OK;
  const size_t es = (size_t)moe::elem_bytes(t);
  if (!index || src_rows > 0) MOE_TRY(check_ptr(x, "x", es));
  if (n_rows) MOE_TRY(check_ptr(n_rows, "n_rows", 4));
  MOE_TRY(check_ptr(codes, "codes", 16));
  MOE_TRY(check_ptr(scales, "scales", 16));
  int cus = 0;
  MOE_TRY(moe::api_num_cus(&cus));
  MOE_LAUNCH(moe::launch_mx_quantize(t, rows, K, x, ld_x, src_rows, index, index_div, n_rows,
                                     codes, scales, cus, static_cast<hipStream_t>(stream)),
             "4-bit quantisation launch");
}

moe_status_t moe_mxfp4_dequantize(int32_t dtype, int64_t rows, int64_t K, const uint8_t* codes,
                                  const uint8_t* scales, void* y, int64_t ld_y,
                                  const int32_t* n_rows, void* stream) {
  ElemType t;
  MOE_TRY(check_dtype(dtype, &t));
  MOE_TRY(check_rows(rows, K));
  MOE_TRY(check_mx_width(K));
  MOE_TRY(check_ld(ld_y, K, "ld_y", &ld_y));
  if (rows == 0) return MOE_OK;
  MOE_TRY(check_ptr(codes, "codes", 16));
  MOE_TRY(check_ptr(scales, "scales", 16));
  MOE_TRY(check_ptr(y, "y", (size_t)moe::elem_bytes(t)));
  if (n_rows) MOE_TRY(check_ptr(n_rows, "n_rows", 4));
  int cus = 0;
  MOE_TRY(moe::api_num_cus(&cus));
  MOE_LAUNCH(moe::launch_mx_dequantize(t, rows, K, codes, scales, y, ld_y, n_rows, cus,
                                       static_cast<hipStream_t>(stream)),
             "4-bit dequantisation launch");
}

moe_status_t moe_mxfp4_grouped_gemm(const moe_grouped_t* g, const int32_t* offsets,
                                    const uint8_t* x_codes, const uint8_t* x_scales,
                                    const uint8_t* w_codes, const uint8_t* w_scales, void* y,
                                    void* stream) {
  moe::RaggedShape s;
  MOE_TRY(check_grouped(g, &s));
  MOE_TRY(check_mx_width(g->K));
  if (g->ld_x != 0 && g->ld_x != g->K)
    return api_fail(MOE_ERR_INVALID_ARGUMENT, "ld_x must be K (or 0): 4-bit rows are contiguous");
  if (s.rows == 0) return MOE_OK;
  MOE_TRY(check_ptr(offsets, "offsets", 4));
  MOE_TRY(check_ptr(x_codes, "x_codes", 16));
  MOE_TRY(check_ptr(x_scales, "x_scales", 16));
  MOE_TRY(check_ptr(w_codes, "w_codes", 16));
  MOE_TRY(check_ptr(w_scales, "w_scales", 16));
  MOE_TRY(check_ptr(y, "y", (size_t)moe::elem_bytes(s.type)));
  int cus = 0;
  MOE_TRY(moe::api_num_cus(&cus));
  MOE_LAUNCH(moe::launch_mx_gemm(s, offsets, x_codes, x_scales, w_codes, w_scales, y, cus,
                                 static_cast<hipStream_t>(stream)),
             "4-bit grouped product launch");
}

}  // extern "C"
