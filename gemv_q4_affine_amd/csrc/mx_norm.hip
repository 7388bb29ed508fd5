// mx_norm.hip -- block_norm_mx: the residual add and the norms of block_norm
// (norm.hip), with n rounded to MX codes where it is computed.
//
// A code is a rounding to 2 or 4 bits: a value next to a border between two
// codes goes to either side by an error of its last bit, and a flipped code is
// 6 to 50 percent off.  So everything between the inputs and the codes is
// binary64 (error about 1e-15, flips one value in 1e13): the codes are those
// of the exact n.  n passes to binary32 on the way to the code by rounding to
// odd (cut, with the last bit set where anything was cut off), after which the
// second rounding gives what one rounding of n would.
//
// A workgroup holds a row in registers as it lies in memory, V pieces of eight
// values a thread, and the next row is requested before this row's sums; four
// lanes share a block of 32.
//
// Bounds.  One read and one write of a row; at 2048 x 4096 bfloat16 with two norms and
// 8-bit codes 59 MB in 17.4 us a call among others (3.4 TB/s), where binary64 sums
// and their joins across the waves lie between a row's loads and its stores
// (two barriers a row; two workgroups of 512 threads are resident on a CU, and each
// has its next row's loads in flight meanwhile).
// Binary32 throughout would be nearer to memory but flips codes; binary32 with binary64 only for
// values near a border is not tried.  One row: 3.9 us.
#include "mx_common.hpp"
#include "tile_image.hpp"
#include "wave_exchange.hpp"

namespace q4 {

namespace {

// Sum over a wave, the same in every lane: DPP inside rows of 16 lanes (swap
// neighbours, pairs, halves of eight, eights), then the lane swaps between them.
template <int CTRL>
__device__ __forceinline__ double dpp_add(double v) {
    const u32x2_t b = __builtin_bit_cast(u32x2_t, v);
    const u32x2_t t = {(uint32_t)__builtin_amdgcn_mov_dpp((int)b[0], CTRL, 0xF, 0xF, false),
                       (uint32_t)__builtin_amdgcn_mov_dpp((int)b[1], CTRL, 0xF, 0xF, false)};
    return v + __builtin_bit_cast(double, t);
}
__device__ __forceinline__ double lanes_sum(double v) {
    v = dpp_add<0xB1>(v);
    v = dpp_add<0x4E>(v);
    v = dpp_add<0x141>(v);
    v = dpp_add<0x140>(v);
    u32x2_t b = __builtin_bit_cast(u32x2_t, v);
    auto lo = __builtin_amdgcn_permlane16_swap(b[0], b[0], false, false);
    auto hi = __builtin_amdgcn_permlane16_swap(b[1], b[1], false, false);
    v = __builtin_bit_cast(double, u32x2_t{lo[0], hi[0]}) + __builtin_bit_cast(double, u32x2_t{lo[1], hi[1]});
    b = __builtin_bit_cast(u32x2_t, v);
    lo = __builtin_amdgcn_permlane32_swap(b[0], b[0], false, false);
    hi = __builtin_amdgcn_permlane32_swap(b[1], b[1], false, false);
    return __builtin_bit_cast(double, u32x2_t{lo[0], hi[0]}) + __builtin_bit_cast(double, u32x2_t{lo[1], hi[1]});
}

// Eight values of a row as they lie in memory.
template <int DT>
struct Raw {
    u32x4_t v[DT == DT_F32 ? 2 : 1];
};
template <int DT>
__device__ __forceinline__ Raw<DT> get8(const void* p, int64_t i) {
    Raw<DT> r;
    const u32x4_t* q = reinterpret_cast<const u32x4_t*>(static_cast<const char*>(p) + i * (DT == DT_F32 ? 4 : 2));
    r.v[0] = q[0];
    if constexpr (DT == DT_F32) r.v[1] = q[1];
    return r;
}
template <int DT>
__device__ __forceinline__ float value(const Raw<DT>& r, int e) {
    if constexpr (DT == DT_F32) return __uint_as_float(r.v[e >> 2][e & 3]);
    else if constexpr (DT == DT_BF16) return __uint_as_float(e & 1 ? r.v[0][e >> 1] & 0xFFFF0000u : r.v[0][e >> 1] << 16);
    else return f16_to_f32((r.v[0][e >> 1] >> (16 * (e & 1))) & 0xFFFFu);
}
template <int DT>
__device__ __forceinline__ void put8(void* p, int64_t i, const float (&f)[8]) {
    if constexpr (DT == DT_F32) {
        floatx4_t* q = reinterpret_cast<floatx4_t*>(static_cast<float*>(p) + i);
        q[0] = floatx4_t{f[0], f[1], f[2], f[3]};
        q[1] = floatx4_t{f[4], f[5], f[6], f[7]};
    } else {
        *reinterpret_cast<u32x4_t*>(static_cast<uint16_t*>(p) + i) = pack8(DT, f);
    }
}

// d rounded to odd: toward zero, the last bit set if that was not exact.
__device__ __forceinline__ float round_to_odd(double d) {
    const float f = (float)d;
    const double back = (double)f;
    if (back == d || d != d) return f;
    uint32_t b = __float_as_uint(f);
    if (fabs(back) > fabs(d)) b--;             // (an f that overflowed steps back to the largest number)
    return __uint_as_float(b | 1u);
}

}  // namespace

template <int DT, int RT, int V, int TYPE>
__global__ __launch_bounds__(1024) void k_block_norm_mx(const MxNormArgs args) {
    const NormArgs& a = args.norm;
    __shared__ double red[2][kMaxWaves];
    int turn = 0;
    const int tid = threadIdx.x, T = blockDim.x, waves = T >> 6;
    const int64_t D = a.D;
    const double inv = 1.0 / (double)D;
    auto row_sum = [&](double s) __attribute__((always_inline)) {
        s = lanes_sum(s);
        if (waves == 1) return s;
        // the two buffers in turn: between the reads of one and its next write lies a barrier
        double* mine = red[turn];
        turn ^= 1;
        if ((tid & 63) == 0) mine[tid >> 6] = s;
        __syncthreads();
        s = 0.0;
        for (int w = 0; w < waves; w++) s += mine[w];
        return s;
    };
    // pieces past the row's end read its last one and count for nothing
    int at[V];
    bool in[V];
#pragma unroll
    for (int v = 0; v < V; v++) {
        at[v] = (v * T + tid) * 8;
        in[v] = at[v] < (int)D;
        if (!in[v]) at[v] = (int)D - 8;
    }
    // mean and 1 / sqrt(variance + eps) of x(v, e), by the norm's kind
    auto stats = [&](auto x, int kind, double& mean, double& rstd) __attribute__((always_inline)) {
        mean = 0.0;
        rstd = 1.0;
        if (kind == NORM_NONE) return;
        double s = 0.0;
        if (kind == NORM_LAYER) {
#pragma unroll
            for (int v = 0; v < V; v++)
                if (in[v])
#pragma unroll
                    for (int e = 0; e < 8; e++) s += x(v, e);
            mean = row_sum(s) * inv;
            s = 0.0;
#pragma unroll
            for (int v = 0; v < V; v++)
                if (in[v])
#pragma unroll
                    for (int e = 0; e < 8; e++) {
                        const double d = x(v, e) - mean;
                        s = fma(d, d, s);
                    }
        } else {
#pragma unroll
            for (int v = 0; v < V; v++)
                if (in[v])
#pragma unroll
                    for (int e = 0; e < 8; e++) s = fma(x(v, e), x(v, e), s);
        }
        rstd = 1.0 / sqrt(fma(row_sum(s), inv, (double)a.eps));
    };
    // one piece a thread: the weights stay in registers; more of them are read again
    Raw<DT> pre_w = {}, post_w = {};
    if constexpr (V == 1) {
        if (a.pre_w) pre_w = get8<DT>(a.pre_w, at[0]);
        if (a.post_w) post_w = get8<DT>(a.post_w, at[0]);
    }
    Raw<RT> nr[V];
    Raw<DT> ny[V];
    auto request = [&](int64_t m) __attribute__((always_inline)) {
#pragma unroll
        for (int v = 0; v < V; v++) {
            nr[v] = get8<RT>(a.r, m * D + at[v]);
            if (a.y) ny[v] = get8<DT>(a.y, m * D + at[v]);
        }
    };
    if (blockIdx.x < a.M) request(blockIdx.x);
    for (int64_t m = blockIdx.x; m < a.M; m += gridDim.x) {
        const int64_t o = m * D;
        double r[V][8], m0 = 0.0, i0 = 1.0, m1, i1;
        Raw<DT> y[V];
#pragma unroll
        for (int v = 0; v < V; v++) {
            y[v] = ny[v];
#pragma unroll
            for (int e = 0; e < 8; e++) r[v][e] = (double)value<RT>(nr[v], e);
        }
        if (m + gridDim.x < a.M) request(m + gridDim.x);
        if (a.y) {
            const int64_t gr = a.gate_rows >= a.M ? 0 : (uint32_t)m / (uint32_t)a.gate_rows;
            Raw<DT> gate = {};
            if (V == 1 && a.gate) gate = get8<DT>(a.gate, gr * D + at[0]);
            stats([&](int v, int e) __attribute__((always_inline)) { return (double)value<DT>(y[v], e); }, a.post, m0, i0);
            const double scale = (double)a.scale;
#pragma unroll
            for (int v = 0; v < V; v++) {
                // scale gate ((y - mean) rstd w + b)
                double p[8];
#pragma unroll
                for (int e = 0; e < 8; e++) p[e] = (double)value<DT>(y[v], e);
                if (a.post == NORM_LAYER) {
#pragma unroll
                    for (int e = 0; e < 8; e++) p[e] -= m0;
                }
                if (a.post != NORM_NONE) {
#pragma unroll
                    for (int e = 0; e < 8; e++) p[e] *= i0;
                }
                if (a.post_w) {
                    const Raw<DT> w = V == 1 ? post_w : get8<DT>(a.post_w, at[v]);
#pragma unroll
                    for (int e = 0; e < 8; e++) p[e] *= (double)value<DT>(w, e);
                }
                if (a.post_b) {
                    const Raw<DT> b = get8<DT>(a.post_b, at[v]);
#pragma unroll
                    for (int e = 0; e < 8; e++) p[e] += (double)value<DT>(b, e);
                }
                if (a.gate) {
                    const Raw<DT> g = V == 1 ? gate : get8<DT>(a.gate, gr * D + at[v]);
#pragma unroll
                    for (int e = 0; e < 8; e++) p[e] *= (double)value<DT>(g, e);
                }
                float out[8];
#pragma unroll
                for (int e = 0; e < 8; e++) {
                    r[v][e] = fma(scale, p[e], r[v][e]);
                    out[e] = (float)r[v][e];
                }
                if (in[v]) put8<RT>(a.r_out, o + at[v], out);
            }
        }
        stats([&](int v, int e) __attribute__((always_inline)) { return r[v][e]; }, a.pre, m1, i1);
#pragma unroll
        for (int v = 0; v < V; v++) {
            double t[8];
#pragma unroll
            for (int e = 0; e < 8; e++) t[e] = r[v][e];
            if (a.pre == NORM_LAYER) {
#pragma unroll
                for (int e = 0; e < 8; e++) t[e] -= m1;
            }
#pragma unroll
            for (int e = 0; e < 8; e++) t[e] *= i1;
            if (a.pre_w) {
                const Raw<DT> w = V == 1 ? pre_w : get8<DT>(a.pre_w, at[v]);
#pragma unroll
                for (int e = 0; e < 8; e++) t[e] *= (double)value<DT>(w, e);
            }
            if (a.pre_b) {
                const Raw<DT> b = get8<DT>(a.pre_b, at[v]);
#pragma unroll
                for (int e = 0; e < 8; e++) t[e] += (double)value<DT>(b, e);
            }
            // Two roundings differ from one only where the first gives a border between
            // two codes or a power of two.  A normal number that is one ends in 19 zeros;
            // below 2^-126, where steps are even, borders may end in 12, but only under
            // scales below 2^-120 and so among values below 2^-112.
            float n[8], most = 0.0f;
            uint32_t low = ~0u;
#pragma unroll
            for (int e = 0; e < 8; e++) {
                n[e] = (float)t[e];
                const uint32_t b = __float_as_uint(n[e]) << 13;
                low = b < low ? b : low;
                most = fmaxf(most, fabsf(n[e]));
            }
            if (low == 0u || most < 0x1p-112f) {
#pragma unroll
                for (int e = 0; e < 8; e++) n[e] = round_to_odd(t[e]);
            }
            uint32_t top = 0u;
#pragma unroll
            for (int e = 0; e < 8; e++) {
                const uint32_t bits = abs_bits(n[e]);
                top = bits > top ? bits : top;
            }
            const uint32_t s = mx_scale_byte<TYPE>(quad_max(top));      // D % 32 == 0: a quad lies in the row or past it
            const u32x2_t q = mx_codes8<TYPE>(n, s);
            const int64_t piece = (o + at[v]) >> 3;
            if (in[v]) {
                if constexpr (TYPE == XT_MXFP4) reinterpret_cast<uint32_t*>(args.codes)[piece] = q[0];
                else reinterpret_cast<u32x2_t*>(args.codes)[piece] = q;
                if ((tid & 3) == 0) args.scales[piece >> 2] = (uint8_t)s;
            }
        }
        if (a.stats && tid < 4) a.stats[m * 4 + tid] = (float)(tid == 0 ? m0 : tid == 1 ? i0 : tid == 2 ? m1 : i1);
    }
}

// 1280 threads a CU, a workgroup's rows in turn: 2048 x 4096 17.9 us, with 2560 threads 18.7, a
// workgroup a row 20.0 (2907 x 672: 9.1, 9.0, 9.0; 3000 x 2048: 16.1, 15.3, 15.4).
template <int DT, int RT, int V>
static void norm_v(const MxNormArgs& a, hipStream_t s) {
    const int64_t D = a.norm.D, M = a.norm.M;
    const unsigned threads = (unsigned)((D / 8 + 64 * V - 1) / (64 * V) * 64);
    const int64_t fit = (int64_t)current_cu_count() * (1280 / threads > 0 ? 1280 / threads : 1);
    auto k = a.n_type == XT_MXFP4 ? k_block_norm_mx<DT, RT, V, XT_MXFP4> : k_block_norm_mx<DT, RT, V, XT_MXFP8>;
    hipLaunchKernelGGL(k, dim3((unsigned)(M < fit ? M : fit)), dim3(threads), 0, s, a);
}
template <int DT, int RT>
static void norm_t(const MxNormArgs& a, hipStream_t s) {
    if (a.norm.D <= 8192) norm_v<DT, RT, 1>(a, s);
    else if (a.norm.D <= 16384) norm_v<DT, RT, 2>(a, s);
    else norm_v<DT, RT, 4>(a, s);
}

hipError_t launch_block_norm_mx(const MxNormArgs& a, hipStream_t s) {
    if (a.norm.dtype == DT_F32) norm_t<DT_F32, DT_F32>(a, s);
    else if (a.norm.dtype == DT_BF16 && a.norm.r_dtype == DT_BF16) norm_t<DT_BF16, DT_BF16>(a, s);
    else if (a.norm.dtype == DT_BF16) norm_t<DT_BF16, DT_F32>(a, s);
    else if (a.norm.r_dtype == DT_F16) norm_t<DT_F16, DT_F16>(a, s);
    else norm_t<DT_F16, DT_F32>(a, s);
    return hipGetLastError();
}

}  // namespace q4
