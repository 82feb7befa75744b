// C ABI of the operators around the experts' products: argument checks and
// launches. No call allocates, waits or keeps state, so every one of them can
// be captured into a graph.
#include <cmath>

#include "ragged_checks.hpp"
#include "router.hpp"

namespace {

using namespace moe;

struct Router {
  ElemType type;
  int64_t ld;
  int groups, per_group, top_groups, group_top;
};

moe_status_t check_router(const moe_router_t* r, Router* out) {
  if (!r) return api_fail(MOE_ERR_INVALID_ARGUMENT, "router is NULL");
  if (r->T < 0) return api_fail(MOE_ERR_INVALID_ARGUMENT, "T must be >= 0");
  if (r->E < 1) return api_fail(MOE_ERR_INVALID_ARGUMENT, "E must be >= 1");
  if (r->k < 1 || r->k > r->E)
    return api_fail(MOE_ERR_INVALID_ARGUMENT, "k must lie in [1, E]");
  MOE_TRY(check_dtype(r->dtype, &out->type));
  if (r->score != MOE_SCORE_SOFTMAX && r->score != MOE_SCORE_SIGMOID)
    return api_fail(MOE_ERR_INVALID_ARGUMENT, "unknown score");
  if (r->renormalize != 0 && r->renormalize != 1)
    return api_fail(MOE_ERR_INVALID_ARGUMENT, "renormalize must be 0 or 1");
  if (!std::isfinite(r->scale)) return api_fail(MOE_ERR_INVALID_ARGUMENT, "scale must be finite");
  if (r->groups < 0 || r->top_groups < 0 || r->group_top < 0 || r->group_top > 2)
    return api_fail(MOE_ERR_INVALID_ARGUMENT,
                    "groups and top_groups must be >= 0, group_top 0, 1 or 2");
  out->groups = r->groups ? r->groups : 1;
  out->top_groups = r->top_groups ? r->top_groups : out->groups;
  out->group_top = r->group_top ? r->group_top : 2;
  if (r->E % out->groups)
    return api_fail(MOE_ERR_INVALID_ARGUMENT, "groups must divide E");
  if (out->top_groups > out->groups)
    return api_fail(MOE_ERR_INVALID_ARGUMENT, "top_groups is above groups");
  out->per_group = r->E / out->groups;
  if ((int64_t)r->k > (int64_t)out->top_groups * out->per_group)
    return api_fail(MOE_ERR_INVALID_ARGUMENT, "the top_groups hold fewer than k experts");
  // a choice from all groups needs no scores of theirs
  if (out->top_groups == out->groups) {
    out->groups = out->top_groups = 1;
    out->per_group = r->E;
  }
  if (r->E > kRaggedMaxExperts) return api_fail(MOE_ERR_UNSUPPORTED, "E > 1024 is not supported");
  if (r->k > kRouterMaxTopK) return api_fail(MOE_ERR_UNSUPPORTED, "k > 64 is not supported");
  if (out->groups > kRouterMaxGroups)
    return api_fail(MOE_ERR_UNSUPPORTED, "more than 64 groups are not supported");
  MOE_TRY(check_ld(r->ld, r->E, "ld", &out->ld));
  if (r->T >= k2G || r->T * r->k >= k2G)
    return api_fail(MOE_ERR_UNSUPPORTED, "T*k must be < 2^31");
  return MOE_OK;
}

bool rows_aligned(const void* p, int64_t ld, ElemType t) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld * elem_bytes(t) % 16 == 0;
}

moe_status_t check_sort(int64_t n, int32_t E) {
  if (n < 0) return api_fail(MOE_ERR_INVALID_ARGUMENT, "n must be >= 0");
  if (E < 1) return api_fail(MOE_ERR_INVALID_ARGUMENT, "E must be >= 1");
  if (n >= k2G) return api_fail(MOE_ERR_UNSUPPORTED, "n must be < 2^31");
  if (E > kRaggedMaxExperts) return api_fail(MOE_ERR_UNSUPPORTED, "E > 1024 is not supported");
  return MOE_OK;
}

moe_status_t check_collect(int32_t dtype, int64_t T, int32_t k, int64_t rows, int64_t d,
                           ElemType* t) {
  MOE_TRY(check_dtype(dtype, t));
  MOE_TRY(check_rows(rows, d));
  if (T < 0) return api_fail(MOE_ERR_INVALID_ARGUMENT, "T must be >= 0");
  if (k < 1) return api_fail(MOE_ERR_INVALID_ARGUMENT, "k must be >= 1");
  if (T >= k2G || T * k >= k2G) return api_fail(MOE_ERR_UNSUPPORTED, "T*k must be < 2^31");
  return MOE_OK;
}

moe_status_t check_orthogonalize(int32_t E, int32_t N, int32_t K) {
  if (E < 1 || N < 1 || K < 1)
    return api_fail(MOE_ERR_INVALID_ARGUMENT, "E, N and K must be >= 1");
  if (E > kRaggedMaxExperts) return api_fail(MOE_ERR_UNSUPPORTED, "E > 1024 is not supported");
  if (N > kOrthoMaxSide || K > kOrthoMaxSide)
    return api_fail(MOE_ERR_UNSUPPORTED, "N and K must be <= 16384");
  return MOE_OK;
}

}  // namespace

extern "C" {

moe_status_t moe_route(const moe_router_t* r, const void* logits, const float* bias, int32_t* idx,
                       float* weight, void* stream) {
  Router c;
  MOE_TRY(check_router(r, &c));
  if (r->T == 0) return MOE_OK;
  MOE_TRY(check_ptr(logits, "logits", (size_t)elem_bytes(c.type)));
  if (bias) MOE_TRY(check_ptr(bias, "bias", 4));
  MOE_TRY(check_ptr(idx, "idx", 4));
  MOE_TRY(check_ptr(weight, "weight", 4));
  RouterParams p{};
  p.logits = logits;
  p.bias = bias;
  p.idx = idx;
  p.weight = weight;
  p.T = r->T;
  p.ld = c.ld;
  p.type = c.type;
  p.E = r->E;
  p.k = r->k;
  p.groups = c.groups;
  p.per_group = c.per_group;
  p.top_groups = c.top_groups;
  p.group_top = c.group_top;
  p.scale = r->scale;
  p.sigmoid = r->score == MOE_SCORE_SIGMOID;
  p.renormalize = r->renormalize != 0;
  p.vec = rows_aligned(logits, c.ld, c.type) && r->E * elem_bytes(c.type) % 16 == 0;
  p.bias_vec = rows_aligned(bias, r->E, ElemType::kF32);
  MOE_LAUNCH(launch_router(p, static_cast<hipStream_t>(stream)), "routing launch");
}

moe_status_t moe_route_backward(const moe_router_t* r, const void* logits, const int32_t* idx,
                                const float* dweight, void* dlogits, void* stream) {
  Router c;
  MOE_TRY(check_router(r, &c));
  if (r->T == 0) return MOE_OK;
  const size_t es = (size_t)elem_bytes(c.type);
  MOE_TRY(check_ptr(logits, "logits", es));
  MOE_TRY(check_ptr(idx, "idx", 4));
  MOE_TRY(check_ptr(dweight, "dweight", 4));
  MOE_TRY(check_ptr(dlogits, "dlogits", es));
  int cus = 0;
  MOE_TRY(api_num_cus(&cus));
  RouterGradParams p{};
  p.logits = logits;
  p.idx = idx;
  p.dweight = dweight;
  p.dlogits = dlogits;
  p.T = r->T;
  p.ld = c.ld;
  p.E = r->E;
  p.k = r->k;
  p.scale = r->scale;
  p.sigmoid = r->score == MOE_SCORE_SIGMOID;
  p.renormalize = r->renormalize != 0;
  p.vec = rows_aligned(logits, c.ld, c.type) && rows_aligned(dlogits, c.ld, c.type);
  MOE_LAUNCH(launch_router_backward(c.type, p, cus, static_cast<hipStream_t>(stream)),
             "routing gradient launch");
}

moe_status_t moe_sort_workspace_size(int64_t n, int32_t E, size_t* bytes) {
  MOE_TRY(check_sort(n, E));
  if (!bytes) return api_fail(MOE_ERR_INVALID_ARGUMENT, "bytes is NULL");
  *bytes = sort_bytes(n, E);
  return MOE_OK;
}

moe_status_t moe_sort(int64_t n, int32_t E, const int32_t* idx, int32_t* perm, int32_t* pos,
                      int32_t* offsets, void* ws, size_t ws_bytes, void* stream) {
  MOE_TRY(check_sort(n, E));
  if (n > 0) {
    MOE_TRY(check_ptr(idx, "idx", 4));
    MOE_TRY(check_ptr(perm, "perm", 4));
    MOE_TRY(check_ptr(pos, "pos", 4));
  }
  MOE_TRY(check_ptr(offsets, "offsets", 4));
  const size_t need = sort_bytes(n, E);
  if (need > 0) {
    MOE_TRY(check_ptr(ws, "workspace", 16));
    if (ws_bytes < need) return api_fail(MOE_ERR_WORKSPACE_TOO_SMALL, "workspace too small");
  }
  MOE_LAUNCH(launch_sort(n, E, idx, perm, pos, offsets, static_cast<int32_t*>(ws),
                         static_cast<hipStream_t>(stream)),
             "sort launch");
}

moe_status_t moe_collect(int32_t dtype, int64_t T, int32_t k, int64_t rows, int64_t d,
                         const void* z, int64_t ld_z, const int32_t* pos, const float* weight,
                         void* y, int64_t ld_y, void* stream) {
  ElemType t;
  MOE_TRY(check_collect(dtype, T, k, rows, d, &t));
  MOE_TRY(check_ld(ld_z, d, "ld_z", &ld_z));
  MOE_TRY(check_ld(ld_y, d, "ld_y", &ld_y));
  if (T == 0) return MOE_OK;
  const size_t es = (size_t)elem_bytes(t);
  if (rows > 0) MOE_TRY(check_ptr(z, "z", es));
  MOE_TRY(check_ptr(pos, "pos", 4));
  if (weight) MOE_TRY(check_ptr(weight, "weight", 4));
  MOE_TRY(check_ptr(y, "y", es));
  int cus = 0;
  MOE_TRY(api_num_cus(&cus));
  CollectParams p{};
  p.z = z;
  p.pos = pos;
  p.weight = weight;
  p.y = y;
  p.T = T;
  p.rows = rows;
  p.d = d;
  p.ld_z = ld_z;
  p.ld_y = ld_y;
  p.k = k;
  MOE_LAUNCH(launch_collect(t, p, cus, static_cast<hipStream_t>(stream)), "collect launch");
}

moe_status_t moe_collect_backward(int32_t dtype, int64_t T, int32_t k, int64_t rows, int64_t d,
                                  const void* dy, int64_t ld_dy, const void* z, int64_t ld_z,
                                  const int32_t* pos, const float* weight, void* dz,
                                  int64_t ld_dz, float* dweight, void* stream) {
  ElemType t;
  MOE_TRY(check_collect(dtype, T, k, rows, d, &t));
  MOE_TRY(check_ld(ld_dy, d, "ld_dy", &ld_dy));
  MOE_TRY(check_ld(ld_z, d, "ld_z", &ld_z));
  MOE_TRY(check_ld(ld_dz, d, "ld_dz", &ld_dz));
  if (!dz && !dweight)
    return api_fail(MOE_ERR_INVALID_ARGUMENT, "dz and dweight are both NULL");
  if (T == 0) return MOE_OK;
  const size_t es = (size_t)elem_bytes(t);
  MOE_TRY(check_ptr(dy, "dy", es));
  MOE_TRY(check_ptr(pos, "pos", 4));
  if (weight) MOE_TRY(check_ptr(weight, "weight", 4));
  if (dz) MOE_TRY(check_ptr(dz, "dz", es));
  if (dweight) {
    if (rows > 0) MOE_TRY(check_ptr(z, "z", es));
    MOE_TRY(check_ptr(dweight, "dweight", 4));
  }
  int cus = 0;
  MOE_TRY(api_num_cus(&cus));
  CollectParams p{};
  p.z = z;
  p.dy = dy;
  p.pos = pos;
  p.weight = weight;
  p.dz = dz;
  p.dweight = dweight;
  p.T = T;
  p.rows = rows;
  p.d = d;
  p.ld_z = ld_z;
  p.ld_y = ld_dy;
  p.ld_dz = ld_dz;
  p.k = k;
  MOE_LAUNCH(launch_collect_backward(t, p, cus, static_cast<hipStream_t>(stream)),
             "collect gradient launch");
}

int64_t moe_int8_stride(int64_t K) { return K < 1 || K > kRaggedMaxWidth ? -1 : int8_stride(K); }

moe_status_t moe_int8_quantize(int32_t dtype, int64_t rows, int64_t K, const void* x, int64_t ld_x,
                               int64_t src_rows, const int32_t* index, int32_t index_div,
                               const int32_t* n_rows, int8_t* codes, float* scales,
                               void* stream) {
  ElemType t;
  MOE_TRY(check_dtype(dtype, &t));
  MOE_TRY(check_rows(rows, K));
  MOE_TRY(check_ld(ld_x, K, "ld_x", &ld_x));
  if (index) {
    if (src_rows < 0) return api_fail(MOE_ERR_INVALID_ARGUMENT, "src_rows must be >= 0");
    if (index_div < 1) return api_fail(MOE_ERR_INVALID_ARGUMENT, "index_div must be >= 1");
    MOE_TRY(check_ptr(index, "index", 4));
  }
  if (rows == 0) return MOE_OK;
  if (!index || src_rows > 0) MOE_TRY(check_ptr(x, "x", (size_t)elem_bytes(t)));
  if (n_rows) MOE_TRY(check_ptr(n_rows, "n_rows", 4));
  MOE_TRY(check_ptr(codes, "codes", 16));
  MOE_TRY(check_ptr(scales, "scales", 4));
  int cus = 0;
  MOE_TRY(api_num_cus(&cus));
  MOE_LAUNCH(launch_int8_quantize(t, rows, K, x, ld_x, src_rows, index, index_div, n_rows, codes,
                                  scales, cus, static_cast<hipStream_t>(stream)),
             "8-bit quantisation launch");
}

moe_status_t moe_int8_dequantize(int32_t dtype, int64_t rows, int64_t K, const int8_t* codes,
                                 const float* scales, void* y, int64_t ld_y,
                                 const int32_t* n_rows, void* stream) {
  ElemType t;
  MOE_TRY(check_dtype(dtype, &t));
  MOE_TRY(check_rows(rows, K));
  MOE_TRY(check_ld(ld_y, K, "ld_y", &ld_y));
  if (rows == 0) return MOE_OK;
  MOE_TRY(check_ptr(codes, "codes", 16));
  MOE_TRY(check_ptr(scales, "scales", 4));
  MOE_TRY(check_ptr(y, "y", (size_t)elem_bytes(t)));
  if (n_rows) MOE_TRY(check_ptr(n_rows, "n_rows", 4));
  int cus = 0;
  MOE_TRY(api_num_cus(&cus));
  MOE_LAUNCH(launch_int8_dequantize(t, rows, K, codes, scales, y, ld_y, n_rows, cus,
                                    static_cast<hipStream_t>(stream)),
             "8-bit dequantisation launch");
}

moe_status_t moe_int8_grouped_gemm(const moe_grouped_t* g, const int32_t* offsets,
                                   const int8_t* x_codes, const float* x_scales,
                                   const int8_t* w_codes, const float* w_scales, void* y,
                                   void* stream) {
  RaggedShape s;
  MOE_TRY(check_grouped(g, &s));
  if (g->ld_x != 0 && g->ld_x != g->K)
    return api_fail(MOE_ERR_INVALID_ARGUMENT, "ld_x must be K (or 0): 8-bit rows are contiguous");
  if (g->K > kInt8MaxWidth)
    return api_fail(MOE_ERR_UNSUPPORTED, "K must be < 2^17: the sums are 32-bit integers");
  if (s.rows == 0) return MOE_OK;
  MOE_TRY(check_ptr(offsets, "offsets", 4));
  MOE_TRY(check_ptr(x_codes, "x_codes", 16));
  MOE_TRY(check_ptr(x_scales, "x_scales", 4));
  MOE_TRY(check_ptr(w_codes, "w_codes", 16));
  MOE_TRY(check_ptr(w_scales, "w_scales", 4));
  MOE_TRY(check_ptr(y, "y", (size_t)elem_bytes(s.type)));
  int cus = 0;
  MOE_TRY(api_num_cus(&cus));
  MOE_LAUNCH(launch_int8_gemm(s, offsets, x_codes, x_scales, w_codes, w_scales, y, cus,
                              static_cast<hipStream_t>(stream)),
             "8-bit grouped product launch");
}

moe_status_t moe_orthogonalize_workspace_size(int32_t E, int32_t N, int32_t K, size_t* bytes) {
  MOE_TRY(check_orthogonalize(E, N, K));
  if (!bytes) return api_fail(MOE_ERR_INVALID_ARGUMENT, "bytes is NULL");
  *bytes = orthogonalize_bytes(E, N, K);
  return MOE_OK;
}

moe_status_t moe_orthogonalize(int32_t dtype, int32_t E, int32_t N, int32_t K, const void* g,
                               void* y, int32_t steps, const float* coefficients, float scale,
                               void* ws, size_t ws_bytes, void* stream) {
  ElemType t;
  MOE_TRY(check_dtype(dtype, &t));
  MOE_TRY(check_orthogonalize(E, N, K));
  if (steps < 1) return api_fail(MOE_ERR_INVALID_ARGUMENT, "steps must be >= 1");
  if (steps > kOrthoMaxSteps) return api_fail(MOE_ERR_UNSUPPORTED, "steps must be <= 32");
  if (!std::isfinite(scale)) return api_fail(MOE_ERR_INVALID_ARGUMENT, "scale must be finite");
  float c[3 * kOrthoMaxSteps];
  for (int i = 0; i < 3 * steps; ++i) {
    const float usual[3] = {3.4445f, -4.7750f, 2.0315f};
    c[i] = coefficients ? coefficients[i] : usual[i % 3];
    if (!std::isfinite(c[i]))
      return api_fail(MOE_ERR_INVALID_ARGUMENT, "coefficients must be finite");
  }
  MOE_TRY(check_ptr(g, "g", (size_t)elem_bytes(t)));
  MOE_TRY(check_ptr(y, "y", 2));
  MOE_TRY(check_ptr(ws, "workspace", 16));
  if (ws_bytes < orthogonalize_bytes(E, N, K))
    return api_fail(MOE_ERR_WORKSPACE_TOO_SMALL, "workspace too small");
  int cus = 0;
  MOE_TRY(api_num_cus(&cus));
  MOE_LAUNCH(launch_orthogonalize(t, E, N, K, g, y, steps, c, scale, static_cast<char*>(ws), cus,
                                  static_cast<hipStream_t>(stream)),
             "orthogonalisation launch");
}

}  // extern "C"
