// Limits that host code without HIP needs too.
#pragma once

#include <stdint.h>

namespace moe {

// Buffer resources address their range with 32-bit byte offsets, and a
// load at an offset at or past the range returns zero (tile masking).
// kOob is the offset the kernels give a masked load; every resource range
// is at most kOob bytes, so a masked load never reads memory.
constexpr uint32_t kOob = 0xffffff00u;
constexpr int64_t kMaxResourceBytes = kOob;

}  // namespace moe
