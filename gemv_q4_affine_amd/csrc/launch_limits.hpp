// launch_limits.hpp -- what a launch can hold.
#pragma once

#include <cstdint>

namespace q4 {

// A launch has less than 2^32 threads along a dimension; one with more runs,
// without an error, on what is left of them modulo 2^32.
inline bool launchable(int64_t blocks, int threads) { return blocks * threads < int64_t(1) << 32; }

}  // namespace q4
