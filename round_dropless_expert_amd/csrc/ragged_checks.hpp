// Argument checks that the operators' C ABI units share.
#pragma once

#include "api_common.hpp"
#include "ragged.hpp"

namespace moe {

constexpr int64_t k2G = int64_t(1) << 31;
// Output tiles of one launch (of 128 x 128): its grid's threads stay below 2^32.
constexpr int64_t kMaxTiles = int64_t(1) << 23;

inline int64_t div_up(int64_t a, int64_t b) { return (a + b - 1) / b; }

inline moe_status_t check_dtype(int32_t dtype, ElemType* out) {
  switch (dtype) {
    case MOE_F32: *out = ElemType::kF32; return MOE_OK;
    case MOE_BF16: *out = ElemType::kBF16; return MOE_OK;
    case MOE_F16: *out = ElemType::kF16; return MOE_OK;
  }
  return api_fail(MOE_ERR_INVALID_ARGUMENT, "unknown dtype");
}

inline moe_status_t check_ptr(const void* p, const char* name, size_t align) {
  if (!p) return api_fail(MOE_ERR_INVALID_ARGUMENT, "is NULL", name);
  if (reinterpret_cast<uintptr_t>(p) % align)
    return api_fail(MOE_ERR_INVALID_ARGUMENT,
                    align == 16 ? "must be 16-byte aligned" : "must be aligned to its element",
                    name);
  return MOE_OK;
}

// A leading dimension (0: the width) of rows of `width` elements.
inline moe_status_t check_ld(int64_t ld, int64_t width, const char* name, int64_t* out) {
  *out = ld == 0 ? width : ld;
  if (*out < width)
    return api_fail(MOE_ERR_INVALID_ARGUMENT, "is below the row's width (0 means the width)",
                    name);
  if (*out > kRaggedMaxWidth)
    return api_fail(MOE_ERR_UNSUPPORTED, "is above 2^20 elements", name);
  return MOE_OK;
}

inline moe_status_t check_grouped(const moe_grouped_t* g, RaggedShape* s) {
  if (!g) return api_fail(MOE_ERR_INVALID_ARGUMENT, "config is NULL");
  if (g->rows < 0) return api_fail(MOE_ERR_INVALID_ARGUMENT, "rows must be >= 0");
  if (g->E < 1) return api_fail(MOE_ERR_INVALID_ARGUMENT, "E must be >= 1");
  if (g->N < 1 || g->K < 1) return api_fail(MOE_ERR_INVALID_ARGUMENT, "N and K must be >= 1");
  moe_status_t st = check_dtype(g->dtype, &s->type);
  if (st != MOE_OK) return st;
  if (g->E > kRaggedMaxExperts)
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
      (dw_split(*s).slots + g->E) * tn * tk >= kMaxTiles)
    return api_fail(MOE_ERR_UNSUPPORTED, "more than 2^23 output tiles of 128 x 128");
  return MOE_OK;
}

inline moe_status_t check_rows(int64_t rows, int64_t width) {
  if (rows < 0) return api_fail(MOE_ERR_INVALID_ARGUMENT, "rows must be >= 0");
  if (width < 1) return api_fail(MOE_ERR_INVALID_ARGUMENT, "the row's width must be >= 1");
  if (rows >= k2G) return api_fail(MOE_ERR_UNSUPPORTED, "rows must be < 2^31");
  if (width > kRaggedMaxWidth)
    return api_fail(MOE_ERR_UNSUPPORTED, "the row's width is above 2^20 elements");
  return MOE_OK;
}

}  // namespace moe

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
