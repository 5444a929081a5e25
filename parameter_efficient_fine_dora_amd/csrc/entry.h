// Internal entry points and argument checks shared by the C ABI's source files.
#pragma once
#include <stddef.h>
#include <stdint.h>

#include "../../include/dora.h"

namespace dora {

// dora_forward's body.  allow_side_stream = false keeps every launch on the
// caller's stream (no side stream or events are created).
int forward_impl(const dora_shape* shape, const void* x, const void* W0, const void* A,
                 const void* B, const void* m, void* y, float* norm_out, void* xs_out, void* ws,
                 size_t ws_bytes, void* hip_stream, bool allow_side_stream);

// A tensor that needs the alignment of its element only (4, 2 or 1 bytes);
// `optional`: may be NULL (not wanted, or empty).
inline int check_elem(const void* p, size_t elem_bytes, bool optional) {
  if (!p) return optional ? DORA_OK : DORA_ERR_NULL;
  return reinterpret_cast<uintptr_t>(p) % elem_bytes ? DORA_ERR_ALIGN : DORA_OK;
}

// A workspace of at least `need` bytes.
inline int check_ws(const void* ws, size_t ws_bytes, size_t need) {
  if (need > 0 && !ws) return DORA_ERR_NULL;
  if (reinterpret_cast<uintptr_t>(ws) % 16) return DORA_ERR_ALIGN;
  return ws_bytes < need ? DORA_ERR_WORKSPACE : DORA_OK;
}

}  // namespace dora

#define DORA_CHECK(expr)            \
  do {                              \
    const int rc_ = (expr);         \
    if (rc_ != DORA_OK) return rc_; \
  } while (0)

#define HIP_TRY(expr)                              \
  do {                                             \
    if ((expr) != hipSuccess) return DORA_ERR_HIP; \
  } while (0)
