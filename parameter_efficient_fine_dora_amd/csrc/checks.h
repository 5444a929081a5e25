// Argument checks of the entry points in include/dora_finetune.h.
#pragma once
#include <stddef.h>
#include <stdint.h>

#include "../../include/dora_finetune.h"

namespace dora {

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
