// capi_checks.hpp -- the argument checks that the C ABIs of the feed-forward
// operators (block_capi.cpp) and of the microscaled ones (mx_capi.cpp) share.
#pragma once

#include <cmath>
#include <cstdint>
#include <initializer_list>

#include <hip/hip_runtime.h>

#include "q4_block.h"

namespace q4 {
namespace checks {

constexpr int64_t kMaxDim = int64_t(1) << 30;
// N and K: a panel of 32 rows of an operand image stays below 2^32 bytes
constexpr int64_t kMaxSum = int64_t(1) << 25;

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline int need(std::initializer_list<const void*> ps) {
    for (const void* p : ps)
        if (!p) return Q4_ERR_NULL;
    for (const void* p : ps)
        if (!aligned16(p)) return Q4_ERR_ALIGN;
    return Q4_OK;
}
inline int optional(std::initializer_list<const void*> ps) {
    for (const void* p : ps)
        if (!aligned16(p)) return Q4_ERR_ALIGN;
    return Q4_OK;
}

inline bool act_ok(int act) { return act >= Q4_ACT_NONE && act <= Q4_ACT_RELU; }
inline bool norm_ok(int norm) { return norm >= Q4_NORM_NONE && norm <= Q4_NORM_LAYER; }

inline int check_workspace(const void* ws, int64_t have, int64_t want) {
    if (want <= 0) return Q4_OK;
    if (!ws || have < want) return Q4_ERR_WORKSPACE;
    return aligned16(ws) ? Q4_OK : Q4_ERR_ALIGN;
}

inline int hip_status(hipError_t e) { return e == hipSuccess ? Q4_OK : Q4_ERR_HIP; }
inline hipStream_t as_stream(void* s) { return reinterpret_cast<hipStream_t>(s); }

inline int check_norm(int dtype, int r_dtype, int64_t M, int64_t D, int64_t gate_rows, float scale, int post_norm,
                      int pre_norm) {
    if (dtype != Q4_BF16 && dtype != Q4_F16 && dtype != Q4_F32) return Q4_ERR_DTYPE;
    if (r_dtype != dtype && r_dtype != Q4_F32) return Q4_ERR_DTYPE;
    if (M < 0 || D < 0 || M > kMaxDim || D > Q4_NORM_MAX_D) return Q4_ERR_SHAPE;
    if (!norm_ok(post_norm) || !norm_ok(pre_norm) || !std::isfinite(scale)) return Q4_ERR_ARG;
    if (gate_rows < 1 && M > 0) return Q4_ERR_ARG;
    return Q4_OK;
}

}  // namespace checks
}  // namespace q4
