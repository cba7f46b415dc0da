// The 8-bit block-scaled cache: argument checks shared by its entry points.
#pragma once

#include "internal.h"

namespace mtkv {

constexpr int kMaxF8KvHeads = 256;

// Shape, pointers and alignment of a cache descriptor. `where` names the call.
mt_status check_f8_cache(const mt_f8_cache *c, const char *where);

// MT_F32, MT_F16 or MT_BF16; element bytes, or 0 for an unknown type.
inline int dtype_bytes(mt_dtype t) {
  switch (t) {
    case MT_F32: return 4;
    case MT_F16:
    case MT_BF16: return 2;
  }
  return 0;
}

}  // namespace mtkv
