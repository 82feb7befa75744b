// C ABI of the ragged expert operators: argument checks and launches. No
// call allocates, waits or keeps state, so every one of them can be captured
// into a graph.
#include "ragged_checks.hpp"

namespace {

using namespace moe;

size_t dw_bytes(const moe::RaggedShape& s) {
  return (size_t)moe::dw_split(s).slots * (size_t)s.N * (size_t)s.K * 4;
}

moe_status_t check_mx_width(int64_t K) {
  if (K % MOE_MXFP4_BLOCK)
    return api_fail(MOE_ERR_INVALID_ARGUMENT, "K must be a multiple of 32");
  return MOE_OK;
}

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
