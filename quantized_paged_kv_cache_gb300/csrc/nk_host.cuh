// nk_host.cuh -- host helpers shared by the entry points.
#pragma once

#include <stdint.h>

#include "nk.h"

namespace nk {

// NK_OK, or why the pool struct is refused.
int check_pool(const nk_kv_pool* pool);

// SMs of the current device (0 when it cannot be asked).
int device_sms();

inline bool aligned_to(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

}  // namespace nk
