// linear.hip -- q4_linear, q4_gated and their gradients: which kernels a call
// takes and how it divides its workspace.
#include "linear_few.hpp"
#include "tile_image.hpp"

namespace q4 {

namespace {

// Rows that the few-row kernel takes, in two launches above its own 32: the
// weights are streamed twice, but not written as an image (12288 x 4096, 33 to 64
// rows: 2 x 21 us against 30 for the image and 22 for its product).
constexpr int64_t kFewCallMaxM = 2 * kFewMaxM;

int64_t up256(int64_t n) { return (n + 255) / 256 * 256; }

// The workspace of a product over images: weights, activations, row
// exponents, parts of a split sum, column sums.
struct Layout {
    TilePlan plan;
    int64_t slices, w_panels, x_panels, x_at, exp_at, part_at, sums_at, total;
};
Layout layout(const TilePlan& plan, int64_t w_panels, int64_t slices, int64_t M, int64_t sums) {
    Layout l{};
    l.plan = plan;
    l.slices = slices;
    l.w_panels = w_panels;
    l.x_panels = (M + 31) / 32;
    l.x_at = up256(w_panels * slices * kUnit);
    l.exp_at = l.x_at + l.x_panels * slices * kUnit;
    l.part_at = l.exp_at + up256(M);
    l.sums_at = l.part_at + partial_bytes(plan, M, w_panels);
    l.total = l.sums_at + sums;
    return l;
}
Layout forward_layout(int nmat, int64_t M, int64_t N, int64_t K) {
    return layout(plan_tiles(nmat, M, N, K), (N + 31) / 32 * nmat, image_slices(K), M, 0);
}
Layout backward_layout(int nmat, int64_t M, int64_t N, int64_t K) {
    const int64_t slices = image_slices(N) * nmat;
    return layout(plan_tiles(1, M, K, slices * 16), K / 32, slices, M, grad_sums_bytes(nmat, M, N));
}

TileArgs tile_args(const Layout& l, uint8_t* ws) {
    TileArgs t{};
    t.wimg = ws;
    t.ximg = ws + l.x_at;
    t.xexp = reinterpret_cast<const int8_t*>(ws + l.exp_at);
    t.slices = l.slices;
    t.w_panels = l.w_panels;
    t.x_panels = l.x_panels;
    t.part = reinterpret_cast<float*>(ws + l.part_at);
    return t;
}

}  // namespace

int64_t linear_workspace_bytes(int, int nmat, int64_t M, int64_t N, int64_t K) {
    return M <= kFewCallMaxM ? 0 : forward_layout(nmat, M, N, K).total;
}

// The few-row kernel on rows m0 .. m0 + count - 1.
static hipError_t launch_few(const LinearArgs& a, int64_t m0, int64_t count, hipStream_t s) {
    LinearArgs t = a;
    auto rows = [&](const void* p, int64_t width) {
        return p ? const_cast<char*>(static_cast<const char*>(p)) + m0 * width * 2 : nullptr;
    };
    t.M = count;
    t.x = rows(a.x, a.K);
    t.y = rows(a.y, a.N);
    t.residual = rows(a.residual, a.N);
    for (int i = 0; i < 2; i++) t.pre[i] = rows(a.pre[i], a.N);
    return t.wf == WF_Q4_0 ? launch_few_q4_0(t, s) : t.wf == WF_AFFINE4 ? launch_few_affine4(t, s) : launch_few_affine8(t, s);
}

hipError_t launch_linear(const LinearArgs& a, void* workspace, hipStream_t s) {
    if (a.M <= kFewCallMaxM) {
        const int64_t first = a.M <= kFewMaxM ? a.M : (a.M + 1) / 2;
        const hipError_t e = launch_few(a, 0, first, s);
        return e != hipSuccess || first == a.M ? e : launch_few(a, first, a.M - first, s);
    }
    const Layout l = forward_layout(a.nmat, a.M, a.N, a.K);
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    hipError_t e = launch_pack_weights(a.wf, a.nmat, a.w, a.N, a.K, false, ws, s);
    if (e == hipSuccess)
        e = launch_pack_x(a.x, a.dtype, a.M, a.K, ws + l.x_at, reinterpret_cast<int8_t*>(ws + l.exp_at), s);
    if (e != hipSuccess) return e;
    TileArgs t = tile_args(l, ws);
    t.epi.act = a.act;
    t.epi.dtype = a.dtype;
    t.epi.M = a.M;
    t.epi.N = a.N;
    for (int i = 0; i < 2; i++) {
        t.epi.bias[i] = a.bias[i];
        t.epi.pre[i] = a.pre[i];
    }
    t.epi.residual = a.residual;
    t.epi.y = a.y;
    return launch_tile_gemm(l.plan, a.nmat, t, s);
}

int64_t linear_grad_workspace_bytes(int, int nmat, int64_t M, int64_t N, int64_t K) {
    return backward_layout(nmat, M, N, K).total;
}

hipError_t launch_linear_grad(const LinearGradArgs& a, void* workspace, hipStream_t s) {
    const Layout l = backward_layout(a.nmat, a.M, a.N, a.K);
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    hipError_t e = launch_pack_weights(a.wf, a.nmat, a.w, a.N, a.K, true, ws, s);
    if (e == hipSuccess)
        e = launch_pack_dz(a, ws + l.x_at, reinterpret_cast<int8_t*>(ws + l.exp_at),
                           reinterpret_cast<float*>(ws + l.sums_at), s);
    if (e != hipSuccess) return e;
    TileArgs t = tile_args(l, ws);
    t.epi.act = ACT_NONE;
    t.epi.dtype = DT_BF16;
    t.epi.M = a.M;
    t.epi.N = a.K;
    t.epi.y = a.dx;
    return launch_tile_gemm(l.plan, 1, t, s);
}

}  // namespace q4
