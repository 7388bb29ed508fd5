// wave_exchange.hpp -- sums over the waves of a workgroup.  Plain C++ around the
// barrier that the caller passes: tests/test_wave_exchange.py compiles it for
// the host and runs it with one thread a wave.
#pragma once

namespace q4 {

constexpr int kMaxWaves = 16;

// Sums of two values over the waves, in wave order, the same in every wave.
// `writes`: this lane hands over its wave's pair.  One barrier a call: the calls
// of a workgroup take the two buffers of `red` in turn (`turn`, the same in all
// its waves), so that between the reads of a buffer in one call and its next
// write, two calls later, lies the barrier of the call between them.  With one
// buffer a fast wave would write its next pair under a slow wave's reads.
template <class Barrier>
__device__ __forceinline__ void wave_sums(float& a, float& b, int wave, int waves, bool writes, float (*red)[kMaxWaves][2],
                                          int& turn, Barrier barrier) {
    float (*mine)[2] = red[turn];
    turn ^= 1;
    if (writes) {
        mine[wave][0] = a;
        mine[wave][1] = b;
    }
    barrier();
    a = b = 0.0f;
    for (int w = 0; w < waves; w++) {
        a += mine[w][0];
        b += mine[w][1];
    }
}

}  // namespace q4
