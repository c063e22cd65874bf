// kv4_host.h -- argument checks shared by the calls on the 4-bit cache.
#pragma once

#include "hb_cache.h"

namespace hb {

// HB_OK or HB_EINVAL.
int kv4_check_pool(const hb_kv4_pool *p);
// A bf16 row operand of n rows of `width` values: aligned to 16 bytes, rows
// apart by a multiple of 8 values that is at least the width.
int kv4_check_rows(const void *p, long long stride, int n, int width);

}  // namespace hb
