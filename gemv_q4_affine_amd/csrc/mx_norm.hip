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
// A workgroup holds a row in registers, V pieces of eight values a thread; four
// lanes share a block of 32.
#include "mx_common.hpp"
#include "tile_image.hpp"
#include "wave_exchange.hpp"

namespace q4 {

namespace {

__device__ __forceinline__ double lanes_sum(double v) {
#pragma unroll
    for (int d = 1; d < 64; d *= 2) v += __shfl_xor(v, d, 64);
    return v;
}

template <int DT>
__device__ __forceinline__ void get8(const void* p, int64_t i, float (&f)[8]) {
    if constexpr (DT == DT_F32) {
        const floatx4_t* q = reinterpret_cast<const floatx4_t*>(static_cast<const float*>(p) + i);
        const floatx4_t lo = q[0], hi = q[1];
#pragma unroll
        for (int e = 0; e < 4; e++) {
            f[e] = lo[e];
            f[4 + e] = hi[e];
        }
    } else {
        unpack8(DT, load8_raw<true>(p, i, 8), f);
    }
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
    bool in[V];
#pragma unroll
    for (int v = 0; v < V; v++) in[v] = (int64_t)(v * T + tid) * 8 < D;
    auto stats = [&](const double (&x)[V][8], int kind, double& mean, double& rstd) __attribute__((always_inline)) {
        mean = 0.0;
        rstd = 1.0;
        if (kind == NORM_NONE) return;
        double s = 0.0;
        if (kind == NORM_LAYER) {
#pragma unroll
            for (int v = 0; v < V; v++)
#pragma unroll
                for (int e = 0; e < 8; e++) s += x[v][e];          // zeros past the row's end
            mean = row_sum(s) * inv;
            s = 0.0;
        }
#pragma unroll
        for (int v = 0; v < V; v++)
#pragma unroll
            for (int e = 0; e < 8; e++) {
                const double d = in[v] ? x[v][e] - mean : 0.0;
                s = fma(d, d, s);
            }
        rstd = 1.0 / sqrt(fma(row_sum(s), inv, (double)a.eps));
    };
    // (v - mean) * rstd * w + b of one value
    for (int64_t m = blockIdx.x; m < a.M; m += gridDim.x) {
        const int64_t o = m * D;
        double r[V][8], m0 = 0.0, i0 = 1.0, m1, i1;
#pragma unroll
        for (int v = 0; v < V; v++) {
            float f[8] = {0, 0, 0, 0, 0, 0, 0, 0};
            if (in[v]) get8<RT>(a.r, o + (v * T + tid) * 8, f);
#pragma unroll
            for (int e = 0; e < 8; e++) r[v][e] = (double)f[e];
        }
        if (a.y) {
            const int64_t gr = a.gate_rows >= a.M ? 0 : (uint32_t)m / (uint32_t)a.gate_rows;
            double y[V][8];
#pragma unroll
            for (int v = 0; v < V; v++) {
                float f[8] = {0, 0, 0, 0, 0, 0, 0, 0};
                if (in[v]) get8<DT>(a.y, o + (v * T + tid) * 8, f);
#pragma unroll
                for (int e = 0; e < 8; e++) y[v][e] = (double)f[e];
            }
            stats(y, a.post, m0, i0);
#pragma unroll
            for (int v = 0; v < V; v++) {
                if (!in[v]) continue;
                const int c = (v * T + tid) * 8;
                float w[8], b[8], g[8], out[8];
                if (a.post_w) get8<DT>(a.post_w, c, w);
                if (a.post_b) get8<DT>(a.post_b, c, b);
                if (a.gate) get8<DT>(a.gate, gr * D + c, g);
#pragma unroll
                for (int e = 0; e < 8; e++) {
                    double p = (y[v][e] - m0) * i0;
                    if (a.post_w) p *= (double)w[e];
                    if (a.post_b) p += (double)b[e];
                    if (a.gate) p *= (double)g[e];
                    r[v][e] = fma((double)a.scale, p, r[v][e]);
                    out[e] = (float)r[v][e];
                }
                put8<RT>(a.r_out, o + c, out);
            }
        }
        stats(r, a.pre, m1, i1);
#pragma unroll
        for (int v = 0; v < V; v++) {
            const int c = (v * T + tid) * 8;
            float w[8], b[8], n[8];
            uint32_t top = 0u;
            if (a.pre_w && in[v]) get8<DT>(a.pre_w, c, w);
            if (a.pre_b && in[v]) get8<DT>(a.pre_b, c, b);
#pragma unroll
            for (int e = 0; e < 8; e++) {
                double t = (r[v][e] - m1) * i1;
                if (a.pre_w) t *= (double)w[e];
                if (a.pre_b) t += (double)b[e];
                n[e] = round_to_odd(t);
                const uint32_t bits = abs_bits(n[e]);
                top = bits > top ? bits : top;
            }
            const uint32_t s = mx_scale_byte<TYPE>(quad_max(top));      // D % 32 == 0: a quad lies in the row or past it
            if (!in[v]) continue;
            const u32x2_t q = mx_codes8<TYPE>(n, s);
            const int64_t piece = (o + c) >> 3;
            if constexpr (TYPE == XT_MXFP4) reinterpret_cast<uint32_t*>(args.codes)[piece] = q[0];
            else reinterpret_cast<u32x2_t*>(args.codes)[piece] = q;
            if ((tid & 3) == 0) args.scales[piece >> 2] = (uint8_t)s;
        }
        if (a.stats && tid < 4) a.stats[m * 4 + tid] = (float)(tid == 0 ? m0 : tid == 1 ? i0 : tid == 2 ? m1 : i1);
    }
}

template <int DT, int RT, int V>
static void norm_v(const MxNormArgs& a, hipStream_t s) {
    const int64_t D = a.norm.D, M = a.norm.M;
    const unsigned threads = (unsigned)((D / 8 + 64 * V - 1) / (64 * V) * 64);
    const int64_t fit = (int64_t)current_cu_count() * ((V == 1 ? 2048 : 1024) / threads);
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
