// nk_host.cuh -- host helpers shared by the entry points.
#pragma once

#include <stdint.h>

#include "nk.h"

namespace nk {

// NK_OK, or why the pool struct is refused.
int check_pool(const nk_kv_pool* pool);

// SMs of the current device (0 when it cannot be asked).
int device_sms();

// Limit of a bounded wait, and the number of the first copy withheld (-1: none) --
// nk_test_inject_copy_stall.
struct WaitLimits {
  unsigned long long cycles;
  int withhold;
};
WaitLimits wait_limits();

inline bool aligned_to(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Bytes that a call reads or writes: rows of as many, `stride` apart (at least as many).
struct Range {
  const void* at;
  uint64_t bytes;
  uint64_t rows = 1, stride = 0;
};
// Whether a (of one row) shares a byte with b.
inline bool overlap(const Range& a, const Range& b) {
  if (a.bytes == 0 || b.bytes == 0) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.at), y = reinterpret_cast<uintptr_t>(b.at);
  if (x < y + b.bytes) return y < x + a.bytes;
  // the first row behind the one in front that ends past x
  const uint64_t row = b.stride > 0 ? (x - y - b.bytes) / b.stride + 1 : b.rows;
  return row < b.rows && y + row * b.stride < x + a.bytes;
}

}  // namespace nk
