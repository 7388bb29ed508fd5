// block_simple.hip -- block_norm and its gradients in their simplest form.
#include "block_common.hpp"

namespace q4 {

// ---- norms: one workgroup per row --------------------------------------------

__device__ __forceinline__ float block_sum(float v, float* red) {
    const int tid = threadIdx.x;
    __syncthreads();
    red[tid] = v;
    __syncthreads();
    for (int o = 128; o >= 1; o >>= 1) {
        if (tid < o) red[tid] += red[tid + o];
        __syncthreads();
    }
    return red[0];
}

__global__ __launch_bounds__(256) void k_norm_simple(const NormArgs a) {
    __shared__ float red[256];
    const int64_t m = blockIdx.x, o = m * a.D, go = (m / a.gate_rows) * a.D;
    float mean[2] = {0.0f, 0.0f}, rstd[2] = {1.0f, 1.0f};
    auto r_of = [&](int64_t i) {
        float r = load_elem(a.r, a.r_dtype, o + i);
        if (!a.y) return r;
        float p = load_elem(a.y, a.dtype, o + i);
        if (a.post != NORM_NONE) {
            p = (p - mean[0]) * rstd[0];
            if (a.post_w) p *= load_elem(a.post_w, a.dtype, i);
            if (a.post_b) p += load_elem(a.post_b, a.dtype, i);
        }
        return r + a.scale * (a.gate ? load_elem(a.gate, a.dtype, go + i) : 1.0f) * p;
    };
    auto norm = [&](int kind, int w, auto value) {
        if (kind == NORM_NONE) return;
        float s = 0.0f;
        if (kind == NORM_LAYER) {
            for (int64_t i = threadIdx.x; i < a.D; i += 256) s += value(i);
            mean[w] = block_sum(s, red) / (float)a.D;
            s = 0.0f;
        }
        for (int64_t i = threadIdx.x; i < a.D; i += 256) {
            const float d = value(i) - mean[w];
            s = fmaf(d, d, s);
        }
        rstd[w] = 1.0f / sqrtf(block_sum(s, red) / (float)a.D + a.eps);
    };
    norm(a.post, 0, [&](int64_t i) { return load_elem(a.y, a.dtype, o + i); });
    norm(a.pre, 1, r_of);
    __syncthreads();
    for (int64_t i = threadIdx.x; i < a.D; i += 256) {
        const float r = r_of(i);
        if (a.n) {
            float v = (r - mean[1]) * rstd[1];
            if (a.pre_w) v *= load_elem(a.pre_w, a.dtype, i);
            if (a.pre_b) v += load_elem(a.pre_b, a.dtype, i);
            store_elem(a.n, a.dtype, o + i, v);
        }
        if (a.r_out) store_elem(a.r_out, a.r_dtype, o + i, r);
    }
    if (a.stats && threadIdx.x < 4)
        a.stats[m * 4 + threadIdx.x] = (threadIdx.x & 1) ? rstd[threadIdx.x >> 1] : mean[threadIdx.x >> 1];
}

// Rows: dr and dy.
__global__ __launch_bounds__(256) void k_norm_grad_simple(const NormGradArgs a) {
    __shared__ float red[256];
    const int64_t m = blockIdx.x, o = m * a.D, go = (m / a.gate_rows) * a.D;
    float st[4] = {0.0f, 1.0f, 0.0f, 1.0f};
    for (int i = 0; i < 4; i++) st[i] = a.stats[m * 4 + i];
    float c1 = 0.0f, c2 = 0.0f;      // mean of t, of t * hat
    auto pre_hat = [&](int64_t i) { return (load_elem(a.r_out, a.r_dtype, o + i) - st[2]) * st[3]; };
    auto pre_t = [&](int64_t i) {
        return load_elem(a.dn, a.dtype, o + i) * (a.pre_w ? load_elem(a.pre_w, a.dtype, i) : 1.0f);
    };
    if (a.pre != NORM_NONE) {
        float s1 = 0.0f, s2 = 0.0f;
        for (int64_t i = threadIdx.x; i < a.D; i += 256) {
            s1 += pre_t(i);
            s2 = fmaf(pre_t(i), pre_hat(i), s2);
        }
        c1 = a.pre == NORM_LAYER ? block_sum(s1, red) / (float)a.D : 0.0f;
        c2 = block_sum(s2, red) / (float)a.D;
    }
    auto G = [&](int64_t i) {
        float g = a.dr_out ? load_elem(a.dr_out, a.r_dtype, o + i) : 0.0f;
        if (a.pre != NORM_NONE) g += (pre_t(i) - c1 - pre_hat(i) * c2) * st[3];
        return g;
    };
    auto dp = [&](int64_t i) { return a.scale * (a.gate ? load_elem(a.gate, a.dtype, go + i) : 1.0f) * G(i); };
    auto post_hat = [&](int64_t i) { return (load_elem(a.y, a.dtype, o + i) - st[0]) * st[1]; };
    auto post_t = [&](int64_t i) { return dp(i) * (a.post_w ? load_elem(a.post_w, a.dtype, i) : 1.0f); };
    float e1 = 0.0f, e2 = 0.0f;
    if (a.post != NORM_NONE) {
        float s1 = 0.0f, s2 = 0.0f;
        for (int64_t i = threadIdx.x; i < a.D; i += 256) {
            s1 += post_t(i);
            s2 = fmaf(post_t(i), post_hat(i), s2);
        }
        e1 = a.post == NORM_LAYER ? block_sum(s1, red) / (float)a.D : 0.0f;
        e2 = block_sum(s2, red) / (float)a.D;
    }
    for (int64_t i = threadIdx.x; i < a.D; i += 256) {
        store_elem(a.dr, a.r_dtype, o + i, G(i));
        if (a.dy) {
            const float v = a.post != NORM_NONE ? (post_t(i) - e1 - post_hat(i) * e2) * st[1] : dp(i);
            store_elem(a.dy, a.dtype, o + i, v);
        }
    }
}

hipError_t launch_block_norm(const NormArgs& a, hipStream_t s) {
    hipLaunchKernelGGL(k_norm_simple, dim3((unsigned)a.M), dim3(256), 0, s, a);
    return hipGetLastError();
}

// Columns: one thread per column; the row constants of G come from the
// workspace (c1, c2 per row).
__global__ __launch_bounds__(256) void k_norm_rows_simple(const NormGradArgs a, float* c) {
    __shared__ float red[256];
    const int64_t m = blockIdx.x, o = m * a.D;
    float s1 = 0.0f, s2 = 0.0f;
    if (a.pre != NORM_NONE)
        for (int64_t i = threadIdx.x; i < a.D; i += 256) {
            const float t = load_elem(a.dn, a.dtype, o + i) * (a.pre_w ? load_elem(a.pre_w, a.dtype, i) : 1.0f);
            s1 += t;
            s2 = fmaf(t, (load_elem(a.r_out, a.r_dtype, o + i) - a.stats[m * 4 + 2]) * a.stats[m * 4 + 3], s2);
        }
    s1 = block_sum(s1, red);
    s2 = block_sum(s2, red);
    if (threadIdx.x == 0) {
        c[2 * m] = a.pre == NORM_LAYER ? s1 / (float)a.D : 0.0f;
        c[2 * m + 1] = s2 / (float)a.D;
    }
}
__global__ void k_norm_cols_simple(const NormGradArgs a, const float* c) {
    const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= a.D) return;
    float pw = 0.0f, pb = 0.0f, qw = 0.0f, qb = 0.0f, dg = 0.0f;
    const float prew = a.pre_w ? load_elem(a.pre_w, a.dtype, i) : 1.0f;
    const float postw = a.post_w ? load_elem(a.post_w, a.dtype, i) : 1.0f;
    const float postb = a.post_b ? load_elem(a.post_b, a.dtype, i) : 0.0f;
    for (int64_t m = 0; m < a.M; m++) {
        const int64_t o = m * a.D + i, go = (m / a.gate_rows) * a.D + i;
        const float* st = a.stats + 4 * m;
        float g = a.dr_out ? load_elem(a.dr_out, a.r_dtype, o) : 0.0f;
        if (a.pre != NORM_NONE) {
            const float dn = load_elem(a.dn, a.dtype, o), hat = (load_elem(a.r_out, a.r_dtype, o) - st[2]) * st[3];
            g += (dn * prew - c[2 * m] - hat * c[2 * m + 1]) * st[3];
            pw = fmaf(dn, hat, pw);
            pb += dn;
        }
        if (!a.y) continue;
        float hat = load_elem(a.y, a.dtype, o), p = hat;
        if (a.post != NORM_NONE) {
            hat = (hat - st[0]) * st[1];
            p = fmaf(hat, postw, postb);
        }
        const float dp = a.scale * (a.gate ? load_elem(a.gate, a.dtype, go) : 1.0f) * g;
        qw = fmaf(dp, hat, qw);
        qb += dp;
        dg = fmaf(a.scale * g, p, dg);
        if (a.dgate && (m + 1 == a.M || (m + 1) % a.gate_rows == 0)) {
            store_elem(a.dgate, a.dtype, go, dg);
            dg = 0.0f;
        }
    }
    if (a.pre_dw) a.pre_dw[i] = pw;
    if (a.pre_db) a.pre_db[i] = pb;
    if (a.post_dw) a.post_dw[i] = qw;
    if (a.post_db) a.post_db[i] = qb;
}

int64_t norm_grad_workspace_bytes(int64_t M, int64_t, int64_t) { return M * 8; }

hipError_t launch_block_norm_grad(const NormGradArgs& a, void* ws, hipStream_t s) {
    float* c = static_cast<float*>(ws);
    hipLaunchKernelGGL(k_norm_grad_simple, dim3((unsigned)a.M), dim3(256), 0, s, a);
    hipLaunchKernelGGL(k_norm_rows_simple, dim3((unsigned)a.M), dim3(256), 0, s, a, c);
    hipLaunchKernelGGL(k_norm_cols_simple, dim3((unsigned)((a.D + 63) / 64)), dim3(64), 0, s, a, c);
    return hipGetLastError();
}

}  // namespace q4
