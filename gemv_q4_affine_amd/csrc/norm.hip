// norm.hip -- block_norm and its gradients: the residual add with the norms
// before and after a block, one pass over the data.
//
// A workgroup holds a row in registers, V pieces of eight values a thread, so
// every tensor is read once and written once: that traffic is the bound.  Sums
// run over a wave by lane permutes and over the waves through LDS, in an order
// that depends on D only.  A workgroup takes several rows: weights and biases
// stay in its registers, and the gradients' sums over the rows with them.
//
// Measured, D = 4096 bfloat16, RMS norms before and after, a gate: forward 17 us
// at 2048 rows, 53 us at 8192 (5.1 TB/s, a large copy's rate); gradients 102 us
// at 8192 rows (4.0 TB/s) and 7 us for the sums' join.  With one RMS norm and no gate
// 49 and 88 us at 8192 rows, the gradients with their join.  What
// cost most on the way: registers.  With the weights held in binary32 and the
// absent tensors' cases compiled in, the gradients took 205 registers, one
// workgroup a CU and 118 us, and bounded to 128 they spilled 108 (258 us); rows
// that are not a multiple of eight values, read element by element, took 21 us
// for 1000 x 1537 against 7 with loads aligned to elements only.
#include "tile_image.hpp"
#include "wave_exchange.hpp"

namespace q4 {

namespace {

// Sum over a wave, the same in every lane: DPP inside rows of 16 lanes (swap
// neighbours, pairs, halves of eight, eights), then the lane swaps between them.
template <int CTRL>
__device__ __forceinline__ float dpp_add(float v) {
    return v + __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), CTRL, 0xF, 0xF, false));
}
__device__ __forceinline__ float lanes_sum(float v) {
    v = dpp_add<0xB1>(v);
    v = dpp_add<0x4E>(v);
    v = dpp_add<0x141>(v);
    v = dpp_add<0x140>(v);
    const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(a[0]) + __uint_as_float(a[1]);
    const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

// Sums of two values over the workgroup (wave_sums: `red` and `turn`).
__device__ __forceinline__ void row_sums(float& a, float& b, float (*red)[kMaxWaves][2], int& turn) {
    a = lanes_sum(a);
    b = lanes_sum(b);
    if (blockDim.x > 64)
        wave_sums(a, b, (int)(threadIdx.x >> 6), (int)(blockDim.x >> 6), (threadIdx.x & 63) == 0, red, turn,
                  []() __attribute__((always_inline)) { __syncthreads(); });
}

// Element o of a tensor: o is the same in all lanes, so that an access is a
// scalar address and a 32-bit column.
template <int DT>
__device__ __forceinline__ const void* from(const void* p, int64_t o) {
    return static_cast<const char*>(p) + o * (DT == DT_F32 ? 4 : 2);
}
template <int DT>
__device__ __forceinline__ void* from(void* p, int64_t o) {
    return static_cast<char*>(p) + o * (DT == DT_F32 ? 4 : 2);
}
// The gate row of row m (both below 2^31: a short division).
template <class Args>
__device__ __forceinline__ int64_t gate_row(const Args& a, int64_t m) {
    return a.gate_rows >= a.M ? 0 : (uint32_t)m / (uint32_t)a.gate_rows;
}
// Whether value e of a piece lies in the row.
template <bool VEC>
__device__ __forceinline__ bool inside(int e, int left) { return VEC ? left > 0 : e < left; }

// Eight values of a row as they lie in memory.
template <int DT>
struct Raw8 {
    u32x4_t v[DT == DT_F32 ? 2 : 1];
};
typedef u32x4_t f32x4_any_t __attribute__((aligned(4)));
template <int DT, bool VEC>
__device__ __forceinline__ Raw8<DT> get8(const void* p, uint32_t i, int left) {
    Raw8<DT> r;
    if constexpr (DT == DT_F32) {
        const float* q = static_cast<const float*>(p) + i;
        const u32x4_t z = {0u, 0u, 0u, 0u};
        if (left >= 8 || VEC) {
            r.v[0] = left > 0 ? reinterpret_cast<const f32x4_any_t*>(q)[0] : z;
            r.v[1] = left > 0 ? reinterpret_cast<const f32x4_any_t*>(q)[1] : z;
        } else {
#pragma unroll
            for (int e = 0; e < 8; e++) r.v[e >> 2][e & 3] = e < left ? __float_as_uint(q[e]) : 0u;
        }
    } else {
        r.v[0] = load8_raw<VEC>(p, i, left);
    }
    return r;
}
template <int DT>
__device__ __forceinline__ void values(const Raw8<DT>& r, float (&f)[8]) {
    if constexpr (DT == DT_F32) {
#pragma unroll
        for (int e = 0; e < 8; e++) f[e] = __uint_as_float(r.v[e >> 2][e & 3]);
    } else {
        unpack8(DT, r.v[0], f);
    }
}
template <int DT, bool VEC>
__device__ __forceinline__ void put8(void* p, uint32_t i, int left, const float (&f)[8]) {
    if constexpr (DT == DT_F32) {
        float* q = static_cast<float*>(p) + i;
        if (left >= 8) {
            const floatx4_t lo = {f[0], f[1], f[2], f[3]}, hi = {f[4], f[5], f[6], f[7]};
            reinterpret_cast<f32x4_any_t*>(q)[0] = __builtin_bit_cast(u32x4_t, lo);
            reinterpret_cast<f32x4_any_t*>(q)[1] = __builtin_bit_cast(u32x4_t, hi);
        } else {
#pragma unroll
            for (int e = 0; e < 8; e++)
                if (e < left) q[e] = f[e];
        }
    } else {
        store8<VEC>(p, i, left, pack8(DT, f));
    }
}
// Keeps a piece as it lies in memory: without it the compiler converts the
// weights once, before the rows, and holds twice the registers.
template <int DT>
__device__ __forceinline__ void keep_raw(Raw8<DT>& r) {
#pragma unroll
    for (auto& v : r.v) asm volatile("" : "+v"(v));
}
// A weight, bias or gate piece, or ones or zeros where there is none.
template <int DT, bool VEC>
__device__ __forceinline__ Raw8<DT> vector8(const void* p, uint32_t i, int left, bool ones) {
    if (p) return get8<DT, VEC>(p, i, left);
    Raw8<DT> r;
    const uint32_t one = DT == DT_F32 ? 0x3F800000u : DT == DT_BF16 ? 0x3F803F80u : 0x3C003C00u;
#pragma unroll
    for (auto& v : r.v)
#pragma unroll
        for (int e = 0; e < 4; e++) v[e] = ones ? one : 0u;
    return r;
}

}  // namespace

// Rows m = blockIdx, blockIdx + gridDim, ..: the next row's y and r are
// requested before this row's sums.
template <int DT, int RT, int V, bool VEC>
__global__ __launch_bounds__(1024, V == 1 ? 5 : 4) void k_block_norm(const NormArgs a) {
    __shared__ float red[2][kMaxWaves][2];
    int turn = 0;
    const int tid = threadIdx.x, T = blockDim.x;
    const int64_t D = a.D;
    const float inv = 1.0f / (float)D;
    int left[V];
    Raw8<DT> pw[V], pb[V], qw[V], qb[V];
#pragma unroll
    for (int v = 0; v < V; v++) {
        const uint32_t c = (uint32_t)(v * T + tid) * 8;
        left[v] = (int)D - (int)c < 8 ? (int)D - (int)c : 8;
        pw[v] = vector8<DT, VEC>(a.pre_w, c, left[v], true);
        pb[v] = vector8<DT, VEC>(a.pre_b, c, left[v], false);
        qw[v] = vector8<DT, VEC>(a.post_w, c, left[v], true);
        qb[v] = vector8<DT, VEC>(a.post_b, c, left[v], false);
    }
    Raw8<DT> ny[V];
    Raw8<RT> nr[V];
    auto request = [&](int64_t m) __attribute__((always_inline)) {
#pragma unroll
        for (int v = 0; v < V; v++) {
            const uint32_t c = (uint32_t)(v * T + tid) * 8;
            nr[v] = get8<RT, VEC>(from<RT>(a.r, m * D), c, left[v]);
            if (a.y) ny[v] = get8<DT, VEC>(from<DT>(a.y, m * D), c, left[v]);
        }
    };
    // mean and 1 / sqrt(variance + eps) of x, by the norm's kind
    auto stats = [&](const float (&x)[V][8], int kind, float& mean, float& rstd) __attribute__((always_inline)) {
        float s = 0.0f, unused = 0.0f;
        mean = 0.0f;
        rstd = 1.0f;
        if (kind == NORM_NONE) return;
        if (kind == NORM_LAYER) {
#pragma unroll
            for (int v = 0; v < V; v++)
#pragma unroll
                for (int e = 0; e < 8; e++) s += x[v][e];          // zeros past the row's end
            row_sums(s, unused, red, turn);
            mean = s * inv;
            s = 0.0f;
        }
#pragma unroll
        for (int v = 0; v < V; v++)
#pragma unroll
            for (int e = 0; e < 8; e++) {
                const float d = inside<VEC>(e, left[v]) ? x[v][e] - mean : 0.0f;
                s = fmaf(d, d, s);
            }
        row_sums(s, unused, red, turn);
        rstd = 1.0f / sqrtf(fmaf(s, inv, a.eps));
    };
    int64_t m = blockIdx.x;
    if (m < a.M) request(m);
    for (; m < a.M; m += gridDim.x) {
        float y[V][8], r[V][8];
#pragma unroll
        for (int v = 0; v < V; v++) {
            keep_raw(pw[v]);
            keep_raw(pb[v]);
            keep_raw(qw[v]);
            keep_raw(qb[v]);
            values<RT>(nr[v], r[v]);
            if (a.y) values<DT>(ny[v], y[v]);
        }
        if (m + gridDim.x < a.M) request(m + gridDim.x);
        float m0 = 0.0f, i0 = 1.0f, m1, i1;
        const int64_t o = m * D;
        if (a.y) {
            const int64_t gr = gate_row(a, m);
            Raw8<DT> gate[V];
#pragma unroll
            for (int v = 0; v < V; v++)
                gate[v] = vector8<DT, VEC>(a.gate ? from<DT>(a.gate, gr * D) : nullptr, (uint32_t)(v * T + tid) * 8, left[v], true);
            stats(y, a.post, m0, i0);
#pragma unroll
            for (int v = 0; v < V; v++) {
                float w[8], b[8], g[8];
                values<DT>(qw[v], w);
                values<DT>(qb[v], b);
                values<DT>(gate[v], g);
#pragma unroll
                for (int e = 0; e < 8; e++) {
                    const float p = a.post != NORM_NONE ? fmaf((y[v][e] - m0) * i0, w[e], b[e]) : y[v][e];
                    r[v][e] = inside<VEC>(e, left[v]) ? fmaf(a.scale * g[e], p, r[v][e]) : 0.0f;
                }
                put8<RT, VEC>(from<RT>(a.r_out, o), (uint32_t)(v * T + tid) * 8, left[v], r[v]);
            }
        }
        stats(r, a.pre, m1, i1);
        if (a.n) {
#pragma unroll
            for (int v = 0; v < V; v++) {
                float w[8], b[8];
                values<DT>(pw[v], w);
                values<DT>(pb[v], b);
#pragma unroll
                for (int e = 0; e < 8; e++) r[v][e] = fmaf((r[v][e] - m1) * i1, w[e], b[e]);
                put8<DT, VEC>(from<DT>(a.n, o), (uint32_t)(v * T + tid) * 8, left[v], r[v]);
            }
        }
        if (a.stats && tid < 4) a.stats[m * 4 + tid] = tid == 0 ? m0 : tid == 1 ? i0 : tid == 2 ? m1 : i1;
    }
}

// ---- gradients -----------------------------------------------------------------------
//
// Workgroup b takes the R rows b R .. of the M (grad_rows) and keeps, per column,
// its sums for the weight and bias gradients and for the current gate row.  The sums go
// to the workspace, [workgroup][pre_dw, pre_db, post_dw, post_db][D], and
// k_norm_join adds them in workgroup order.  A gate row whose rows lie in one
// workgroup is finished there; of the others a workgroup has at most two, its
// first and its last, kept at [workgroup][2][D] for k_norm_join.

// Forms compiled apart, with every tensor there, for registers: the norms after
// and before the block, and the one before it only (1000 x 1537, bfloat16: 9.2 us
// against 22.3 in the general form, which spills).
enum : int { FORM_ANY = 0, FORM_BOTH = 1, FORM_PRE = 2 };

template <int DT, int RT, int V, bool VEC, bool BIAS, int FORM>
__global__ __launch_bounds__(1024) void k_norm_grad(const NormGradArgs a, int64_t R, float* __restrict__ sums,
                                                         float* __restrict__ pieces) {
    __shared__ float red[2][kMaxWaves][2];
    int turn = 0;
    const int tid = threadIdx.x, T = blockDim.x;
    const bool has_dn = FORM || a.dn, has_dr = FORM || a.dr_out, has_y = FORM || a.y;
    const bool has_post = FORM == FORM_BOTH || (FORM == FORM_ANY && a.post != NORM_NONE);
    const int64_t D = a.D, r0 = blockIdx.x * R, r1 = r0 + R < a.M ? r0 + R : a.M;
    const float inv = 1.0f / (float)D;
    int left[V];
    Raw8<DT> pw[V], qw[V], qb[V];
    float spw[V][8], spb[V][8], sqw[V][8], sqb[V][8], sg[V][8];
#pragma unroll
    for (int v = 0; v < V; v++) {
        const uint32_t c = (uint32_t)(v * T + tid) * 8;
        left[v] = (int)D - (int)c < 8 ? (int)D - (int)c : 8;
        pw[v] = vector8<DT, VEC>(a.pre_w, c, left[v], true);
        qw[v] = vector8<DT, VEC>(a.post_w, c, left[v], true);
        qb[v] = vector8<DT, VEC>(a.post_b, c, left[v], false);
#pragma unroll
        for (int e = 0; e < 8; e++) spw[v][e] = spb[v][e] = sqw[v][e] = sqb[v][e] = sg[v][e] = 0.0f;
    }
    Raw8<DT> nn[V], ny[V];
    Raw8<RT> nd[V], nr[V];
    float4 nst = make_float4(0.0f, 1.0f, 0.0f, 1.0f);
    auto request = [&](int64_t m) __attribute__((always_inline)) {
        nst = reinterpret_cast<const float4*>(a.stats)[m];
#pragma unroll
        for (int v = 0; v < V; v++) {
            const uint32_t c = (uint32_t)(v * T + tid) * 8;
            if (has_dn) {
                nn[v] = get8<DT, VEC>(from<DT>(a.dn, m * D), c, left[v]);
                nr[v] = get8<RT, VEC>(from<RT>(a.r_out, m * D), c, left[v]);
            }
            if (has_dr) nd[v] = get8<RT, VEC>(from<RT>(a.dr_out, m * D), c, left[v]);
            if (has_y) ny[v] = get8<DT, VEC>(from<DT>(a.y, m * D), c, left[v]);
        }
    };
    request(r0);
    for (int64_t m = r0; m < r1; m++) {
        const float4 st = nst;
        float G[V][8], hat[V][8], y[V][8];
#pragma unroll
        for (int v = 0; v < V; v++) {
            keep_raw(pw[v]);
            keep_raw(qw[v]);
            keep_raw(qb[v]);
            if (has_dr) {
                values<RT>(nd[v], G[v]);
            } else {
#pragma unroll
                for (int e = 0; e < 8; e++) G[v][e] = 0.0f;
            }
            if (has_y) values<DT>(ny[v], y[v]);
        }
        const int64_t o = m * D, gr = gate_row(a, m);
        Raw8<DT> gate[V];
        if (has_y) {
#pragma unroll
            for (int v = 0; v < V; v++)
                gate[v] = vector8<DT, VEC>(a.gate ? from<DT>(a.gate, gr * D) : nullptr, (uint32_t)(v * T + tid) * 8, left[v], true);
        }
        if (has_dn) {
            // G += (t - mean(t) - hat mean(t hat)) rstd with t = dn w
            float t[V][8], c1 = 0.0f, c2 = 0.0f;
#pragma unroll
            for (int v = 0; v < V; v++) {
                float dn[8], r[8], w[8];
                values<DT>(nn[v], dn);
                values<RT>(nr[v], r);
                values<DT>(pw[v], w);
#pragma unroll
                for (int e = 0; e < 8; e++) {
                    hat[v][e] = (r[e] - st.z) * st.w;       // dn is zero past the row's end
                    t[v][e] = dn[e] * w[e];
                    c1 += t[v][e];
                    c2 = fmaf(t[v][e], hat[v][e], c2);
                    spw[v][e] = fmaf(dn[e], hat[v][e], spw[v][e]);
                    if constexpr (BIAS) spb[v][e] += dn[e];
                }
            }
            if (m + 1 < r1) request(m + 1);
            row_sums(c1, c2, red, turn);
            c1 = a.pre == NORM_LAYER ? c1 * inv : 0.0f;
            c2 *= inv;
#pragma unroll
            for (int v = 0; v < V; v++)
#pragma unroll
                for (int e = 0; e < 8; e++)
                    G[v][e] = fmaf(t[v][e] - c1 - hat[v][e] * c2, st.w, G[v][e]);
        } else if (m + 1 < r1) {
            request(m + 1);
        }
#pragma unroll
        for (int v = 0; v < V; v++) put8<RT, VEC>(from<RT>(a.dr, o), (uint32_t)(v * T + tid) * 8, left[v], G[v]);
        if (!has_y) continue;
        // dp = scale gate G; the gate's gradient takes scale G p
        float c1 = 0.0f, c2 = 0.0f;
#pragma unroll
        for (int v = 0; v < V; v++) {
            float w[8], b[8], gt[8];
            values<DT>(qw[v], w);
            values<DT>(qb[v], b);
            values<DT>(gate[v], gt);
#pragma unroll
            for (int e = 0; e < 8; e++) {
                const float g = inside<VEC>(e, left[v]) ? a.scale * G[v][e] : 0.0f;
                if (has_post) {
                    hat[v][e] = (y[v][e] - st.x) * st.y;
                    sg[v][e] = fmaf(g, fmaf(hat[v][e], w[e], b[e]), sg[v][e]);
                    const float dp = g * gt[e];
                    sqw[v][e] = fmaf(dp, hat[v][e], sqw[v][e]);
                    if constexpr (BIAS) sqb[v][e] += dp;
                    G[v][e] = dp * w[e];
                    c1 += G[v][e];
                    c2 = fmaf(G[v][e], hat[v][e], c2);
                } else {
                    sg[v][e] = fmaf(g, y[v][e], sg[v][e]);
                    G[v][e] = g * gt[e];
                }
            }
        }
        if (has_post) {
            row_sums(c1, c2, red, turn);
            c1 = a.post == NORM_LAYER ? c1 * inv : 0.0f;
            c2 *= inv;
#pragma unroll
            for (int v = 0; v < V; v++)
#pragma unroll
                for (int e = 0; e < 8; e++) G[v][e] = (G[v][e] - c1 - hat[v][e] * c2) * st.y;
        }
#pragma unroll
        for (int v = 0; v < V; v++) put8<DT, VEC>(from<DT>(a.dy, o), (uint32_t)(v * T + tid) * 8, left[v], G[v]);
        // the last row of a gate row, or of this workgroup
        const bool ends = m + 1 == a.M || gate_row(a, m + 1) != gr;
        if (a.dgate && (ends || m + 1 == r1)) {
            const bool whole = ends && gr * a.gate_rows >= r0;
#pragma unroll
            for (int v = 0; v < V; v++) {
                const uint32_t c = (uint32_t)(v * T + tid) * 8;
                const int64_t piece = 2 * (int64_t)blockIdx.x + (gr == gate_row(a, r0) ? 0 : 1);
                if (whole) put8<DT, VEC>(from<DT>(a.dgate, gr * D), c, left[v], sg[v]);
                else put8<DT_F32, VEC>(from<DT_F32>(pieces, piece * D), c, left[v], sg[v]);
#pragma unroll
                for (int e = 0; e < 8; e++) sg[v][e] = 0.0f;
            }
        }
    }
#pragma unroll
    for (int v = 0; v < V; v++) {
        const uint32_t c = (uint32_t)(v * T + tid) * 8;
        const int64_t at = (int64_t)blockIdx.x * 4 * D;
        if (a.pre_dw) put8<DT_F32, VEC>(from<DT_F32>(sums, at), c, left[v], spw[v]);
        if (a.post_dw) put8<DT_F32, VEC>(from<DT_F32>(sums, at + 2 * D), c, left[v], sqw[v]);
        if constexpr (BIAS) {
            if (a.pre_db) put8<DT_F32, VEC>(from<DT_F32>(sums, at + D), c, left[v], spb[v]);
            if (a.post_db) put8<DT_F32, VEC>(from<DT_F32>(sums, at + 3 * D), c, left[v], sqb[v]);
        }
    }
}

// The workgroups' sums in a fixed order, 64 columns a workgroup: sixteen lanes
// take four columns each, the 64 groups of sixteen lanes every 64th term.
// blockIdx.y 0 .. 3: the weight and bias gradients, then the gate rows that
// span workgroups.
__global__ __launch_bounds__(1024) void k_norm_join(const float* __restrict__ sums, const float* __restrict__ pieces,
                                                    int64_t groups, int64_t R, const NormGradArgs a) {
    __shared__ float red[16][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, k = blockIdx.y;
    const int64_t D = a.D, n4 = (int64_t)blockIdx.x * 64 + (lane & 15) * 4, n = (int64_t)blockIdx.x * 64 + lane;
    // the sum over i < count of row(i)[n], in wave 0
    auto joined = [&](int64_t count, auto row) __attribute__((always_inline)) {
        float t[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
        for (int64_t i = wave * 4 + (lane >> 4); i < count; i += 64) {
            const float* p = row(i);
            if (n4 + 4 <= D) {
                const u32x4_t v = *reinterpret_cast<const f32x4_any_t*>(p + n4);
#pragma unroll
                for (int e = 0; e < 4; e++) t[e] += __uint_as_float(v[e]);
            } else {
                for (int e = 0; e < 4; e++)
                    if (n4 + e < D) t[e] += p[n4 + e];
            }
        }
#pragma unroll
        for (int e = 0; e < 4; e++) {
            t[e] += __shfl_xor(t[e], 16, 64);
            t[e] += __shfl_xor(t[e], 32, 64);
            if (lane < 16) red[wave][lane * 4 + e] = t[e];
        }
        __syncthreads();
        float out = 0.0f;
        if (wave == 0)
            for (int w = 0; w < 16; w++) out += red[w][lane];
        __syncthreads();
        return out;
    };
    if (k < 4) {
        float* out = k == 0 ? a.pre_dw : k == 1 ? a.pre_db : k == 2 ? a.post_dw : a.post_db;
        if (!out) return;
        const float t = joined(groups, [&](int64_t b) { return sums + (b * 4 + k) * D; });
        if (wave == 0 && n < D) out[n] = t;
        return;
    }
    const int64_t gates = (a.M + a.gate_rows - 1) / a.gate_rows;
    for (int64_t g = k - 4; g < gates; g += gridDim.y - 4) {
        const int64_t end = (g + 1) * a.gate_rows < a.M ? (g + 1) * a.gate_rows : a.M;
        const int64_t b0 = g * a.gate_rows / R, b1 = (end - 1) / R;
        if (b0 == b1) continue;                        // finished by its workgroup
        const float t = joined(b1 - b0 + 1, [&](int64_t i) {
            const int64_t b = b0 + i;
            return pieces + (2 * b + (b * R / a.gate_rows == g ? 0 : 1)) * D;
        });
        if (wave == 0 && n < D) store_elem(a.dgate, a.dtype, g * D + n, t);
    }
}

// ---- host ------------------------------------------------------------------------------

// Pieces of eight a thread: one up to D = 8192 (1024 threads), then two, then four.
static int pieces_of(int64_t D) { return D <= 8192 ? 1 : D <= 16384 ? 2 : 4; }
static unsigned threads_of(int64_t D, int V) {
    const int64_t chunks = (D + 7) / 8;
    return (unsigned)((chunks + 64 * V - 1) / (64 * V) * 64);
}

template <int DT, int RT, int V>
static void norm_v(const NormArgs& a, hipStream_t s) {
    const unsigned threads = threads_of(a.D, V);
    // as many workgroups as the CUs hold at once (2048 threads; half of them with more pieces)
    const int64_t fit = (int64_t)current_cu_count() * ((V == 1 ? 2048 : 1024) / threads);
    const unsigned grid = (unsigned)(a.M < fit ? a.M : fit);
    auto k = a.D % 8 == 0 ? k_block_norm<DT, RT, V, true> : k_block_norm<DT, RT, V, false>;
    hipLaunchKernelGGL(k, dim3(grid), dim3(threads), 0, s, a);
}
template <int DT, int RT>
static void norm_t(const NormArgs& a, hipStream_t s) {
    const int V = pieces_of(a.D);
    if (V == 1) norm_v<DT, RT, 1>(a, s);
    else if (V == 2) norm_v<DT, RT, 2>(a, s);
    else norm_v<DT, RT, 4>(a, s);
}

hipError_t launch_block_norm(const NormArgs& a, hipStream_t s) {
    if (a.dtype == DT_F32) norm_t<DT_F32, DT_F32>(a, s);
    else if (a.dtype == DT_BF16 && a.r_dtype == DT_BF16) norm_t<DT_BF16, DT_BF16>(a, s);
    else if (a.dtype == DT_BF16) norm_t<DT_BF16, DT_F32>(a, s);
    else if (a.r_dtype == DT_F16) norm_t<DT_F16, DT_F16>(a, s);
    else norm_t<DT_F16, DT_F32>(a, s);
    return hipGetLastError();
}

// Rows of a workgroup: 1024 threads a CU of 256, at most four workgroups, since
// the join reads a row of sums for each (8192 x 512: 7.5 us, with sixteen 23.6).
static int64_t grad_rows(int64_t M, int64_t D) {
    const int64_t fit = 1024 / (int64_t)threads_of(D, pieces_of(D)), groups = 256 * (fit < 4 ? fit : 4);
    const int64_t rows = (M + groups - 1) / groups;
    return rows < 2 ? 2 : rows;              // one row a workgroup writes as much in sums as it reads
}
static int64_t grad_groups(int64_t M, int64_t D) { return (M + grad_rows(M, D) - 1) / grad_rows(M, D); }

// Six binary32 rows a workgroup: four sums and two gate pieces.
int64_t norm_grad_workspace_bytes(int64_t M, int64_t D, int64_t) { return grad_groups(M, D) * 6 * ((D + 3) / 4 * 4) * 4; }

template <int DT, int RT, int V, bool BIAS, int FORM>
static void grad_k(const NormGradArgs& a, float* sums, float* pieces, hipStream_t s) {
    auto k = a.D % 8 == 0 ? k_norm_grad<DT, RT, V, true, BIAS, FORM> : k_norm_grad<DT, RT, V, false, BIAS, FORM>;
    hipLaunchKernelGGL(k, dim3((unsigned)grad_groups(a.M, a.D)), dim3(threads_of(a.D, V)), 0, s, a, grad_rows(a.M, a.D),
                       sums, pieces);
}
template <int DT, int RT, int V>
static void grad_v(const NormGradArgs& a, float* sums, float* pieces, hipStream_t s) {
    const bool bias = a.pre_db || a.post_db;
    if constexpr (V == 1) {
        // the layers' usual forms
        if (a.dn && a.dr_out && a.y) {
            if (a.post == NORM_NONE && bias) grad_k<DT, RT, 1, true, FORM_PRE>(a, sums, pieces, s);
            else if (a.post == NORM_NONE) grad_k<DT, RT, 1, false, FORM_PRE>(a, sums, pieces, s);
            else if (bias) grad_k<DT, RT, 1, true, FORM_BOTH>(a, sums, pieces, s);
            else grad_k<DT, RT, 1, false, FORM_BOTH>(a, sums, pieces, s);
            return;
        }
    }
    grad_k<DT, RT, V, true, FORM_ANY>(a, sums, pieces, s);
}
template <int DT, int RT>
static void grad_t(const NormGradArgs& a, float* sums, float* pieces, hipStream_t s) {
    const int V = pieces_of(a.D);
    if (V == 1) grad_v<DT, RT, 1>(a, sums, pieces, s);
    else if (V == 2) grad_v<DT, RT, 2>(a, sums, pieces, s);
    else grad_v<DT, RT, 4>(a, sums, pieces, s);
}

hipError_t launch_block_norm_grad(const NormGradArgs& a, void* workspace, hipStream_t s) {
    const int64_t groups = grad_groups(a.M, a.D);
    float* sums = static_cast<float*>(workspace);
    float* pieces = sums + groups * 4 * a.D;
    if (a.dtype == DT_F32) grad_t<DT_F32, DT_F32>(a, sums, pieces, s);
    else if (a.dtype == DT_BF16 && a.r_dtype == DT_BF16) grad_t<DT_BF16, DT_BF16>(a, sums, pieces, s);
    else if (a.dtype == DT_BF16) grad_t<DT_BF16, DT_F32>(a, sums, pieces, s);
    else if (a.r_dtype == DT_F16) grad_t<DT_F16, DT_F16>(a, sums, pieces, s);
    else grad_t<DT_F16, DT_F32>(a, sums, pieces, s);
    const bool spans = a.dgate && a.gate_rows > 1 && groups > 1;
    if (spans || a.pre_dw || a.pre_db || a.post_dw || a.post_db) {
        const int64_t gates = spans ? (a.M + a.gate_rows - 1) / a.gate_rows : 0;
        hipLaunchKernelGGL(k_norm_join, dim3((unsigned)((a.D + 63) / 64), 4 + (unsigned)(gates < 1024 ? gates : 1024)),
                           dim3(1024), 0, s, sums, pieces, groups, grad_rows(a.M, a.D), a);
    }
    return hipGetLastError();
}

}  // namespace q4
