// Argument checks and the saved block's layout, shared by the entry points.
#pragma once

#include <cmath>

#include "internal.h"

namespace hstu {

// ---------------------------------------------------------------------------
// Argument checks
// ---------------------------------------------------------------------------
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline hstu_status check_cfg(const hstu_config* c) {
  if (!c) return HSTU_ERR_INVALID;
  if (c->dtype != HSTU_F32 && c->dtype != HSTU_BF16) return HSTU_ERR_INVALID;
  if (c->io_dtype != HSTU_F32 && c->io_dtype != HSTU_BF16) return HSTU_ERR_INVALID;
  if (c->io_dtype != c->dtype && !(c->dtype == HSTU_BF16 && c->io_dtype == HSTU_F32))
    return HSTU_ERR_UNSUPPORTED;
  if (c->d_model <= 0 || c->num_heads <= 0 || c->head_dim <= 0) return HSTU_ERR_INVALID;
  if (c->num_heads * c->head_dim != c->d_model) return HSTU_ERR_INVALID;
  if (!(c->norm_N > 0.f) || !std::isfinite(c->norm_N)) return HSTU_ERR_INVALID;
  if (!(c->ln_eps >= 0.f) || !std::isfinite(c->ln_eps)) return HSTU_ERR_INVALID;
  if (c->max_seq_len <= 0) return HSTU_ERR_INVALID;
  if (c->head_dim != 32 && c->head_dim != 64 && c->head_dim != 128) return HSTU_ERR_UNSUPPORTED;
  if (c->d_model % 16 != 0 || c->d_model > 2048) return HSTU_ERR_UNSUPPORTED;
  if (c->num_pos_buckets < 1 || c->num_pos_buckets > 32) return HSTU_ERR_UNSUPPORTED;
  if (c->num_time_buckets < 1 || c->num_time_buckets > 32) return HSTU_ERR_UNSUPPORTED;
  if (c->max_seq_len > 65536) return HSTU_ERR_UNSUPPORTED;
  return HSTU_OK;
}

// Required pointer: non-null and 16-byte aligned when count > 0.
inline hstu_status need(const void* p, int64_t count) {
  if (count <= 0) return HSTU_OK;
  if (!p) return HSTU_ERR_INVALID;
  return aligned16(p) ? HSTU_OK : HSTU_ERR_UNSUPPORTED;
}
// Optional pointer: may be null; aligned when present.
inline hstu_status opt(const void* p) { return (!p || aligned16(p)) ? HSTU_OK : HSTU_ERR_UNSUPPORTED; }
// Metadata pointers (int64/int32 arrays) need natural alignment only.
inline hstu_status meta(const void* p, int64_t count, size_t align) {
  if (count <= 0) return HSTU_OK;
  if (!p) return HSTU_ERR_INVALID;
  return (reinterpret_cast<uintptr_t>(p) % align) == 0 ? HSTU_OK : HSTU_ERR_UNSUPPORTED;
}

#define HSTU_TRY(x)                         \
  do {                                      \
    hstu_status _s = (x);                   \
    if (_s != HSTU_OK) return _s;           \
  } while (0)
#define HSTU_CUDA(x)                        \
  do {                                      \
    cudaError_t _e = (x);                   \
    if (_e != cudaSuccess) return HSTU_ERR_CUDA; \
  } while (0)

// ---------------------------------------------------------------------------
// Layouts
// ---------------------------------------------------------------------------
inline void saved_offsets(const hstu_config* c, int64_t T, size_t off[HSTU_SAVED_COUNT + 1]) {
  const size_t es = (size_t)dtype_size(c->dtype);
  const size_t d = (size_t)c->d_model;
  const size_t t = (size_t)T;
  const size_t xlow = c->io_dtype != c->dtype ? t * d * es : 0;
  const size_t sizes[HSTU_SAVED_COUNT] = {t * 4 * d * es, t * 4 * d * es, t * d * 4,
                                          t * d * es,     t * 4,          t * 4, xlow};
  size_t o = 0;
  for (int i = 0; i < HSTU_SAVED_COUNT; ++i) {
    off[i] = o;
    o = align_up(o + sizes[i], 256);
  }
  off[HSTU_SAVED_COUNT] = o;
}

}  // namespace hstu
