// Host-side argument checks of the attention-layer entry points.
#pragma once

#include <stdio.h>

#include "gdn_launch.h"

#define GDN_TRY(x)                      \
  do {                                  \
    const gdn_status _s = (x);          \
    if (_s != GDN_OK) return _s;        \
  } while (0)

namespace gdn {

// GDN_OK, or GDN_ERR_ARG when `p` (named `name` in the message) is NULL or not aligned.
inline gdn_status check_ptr(const void *p, const char *name, size_t align = 16) {
  char buf[96];
  if (!p) {
    snprintf(buf, sizeof buf, "%s is NULL", name);
    return fail(GDN_ERR_ARG, buf);
  }
  if (reinterpret_cast<uintptr_t>(p) % align != 0) {
    snprintf(buf, sizeof buf, "%s is not %zu-byte aligned", name, align);
    return fail(GDN_ERR_ARG, buf);
  }
  return GDN_OK;
}

}  // namespace gdn
