// wait_bound.h -- how long a wait inside a kernel lasts at most (host and device).
#pragma once

#include <stdint.h>

namespace rd {

// Longest a single try_wait may suspend the thread before returning false;
// without an explicit hint the suspension window is system-defined and can be
// long enough to hide the bound of the waits.
constexpr uint32_t kSuspendHintNs = 1000;

// A bound, and the window of its tries, which the host works out: the tries are on every K block's way.
struct WaitBound {
  uint64_t ns;
  uint32_t try_ns;
};

constexpr WaitBound wait_bound(uint64_t ns) {
  return {ns, ns < kSuspendHintNs ? static_cast<uint32_t>(ns) : kSuspendHintNs};
}

}  // namespace rd
