// wait_limit.h -- how long the kernels' bounded waits for work may take.
#pragma once

#include <cstdlib>

namespace kda {

// 2 s, or KDA_WAIT_LIMIT_NS (a positive integer, read at each call) for tests that make those waits run out.
inline unsigned long long wait_limit_ns() {
  const char* e = std::getenv("KDA_WAIT_LIMIT_NS");
  if (e) {
    char* end = nullptr;
    const unsigned long long v = std::strtoull(e, &end, 10);
    if (end != e && v > 0) return v;
  }
  return 2000000000ull;
}

}  // namespace kda
