// linear.hip -- q4_linear, q4_gated and their gradients: which kernels a call
// takes and how it divides its workspace.
#include "linear_few.hpp"
#include "tile_image.hpp"

namespace q4 {

namespace {

// Rows that the few-row kernel takes, in two launches above its own 32: the
// weights are streamed twice, but not written as an image (Q4_0, 64 rows: 12288 x
// 4096 2 x 21 us against 57, of which 23 for the image and 21 for its product; 4096 x
// 14336 2 x 23 + 5 against 80; 2048 x 2048, 33 rows, 14 against 22).
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
// rest: the sum runs over the weights rounded to binary16, then over what the
// rounding left of them.
Layout forward_layout(int nmat, bool rest, int64_t M, int64_t N, int64_t K) {
    if (rest) K *= 2;
    return layout(plan_tiles(nmat, M, N, K), (N + 31) / 32 * nmat, image_slices(K), M, 0);
}
// A weight rounded to binary16 puts about as much error into a sum as the
// rounding of a binary16 output does.  One such error (q4_linear with no
// activation, or relu) leaves the output within 1.41 of its own rounding's; the
// two of a gated product and a curved activation's slope made it 1.6 to 1.8
// (affine4, 200 rows), so there the remainders are summed too, at twice the matrix
// work (12288 x 4096, 512 rows, gated: 291 us against 148).  bfloat16 outputs are
// eight times coarser.
bool sums_rest(int nmat, int dtype, int act) {
    return dtype == DT_F16 && (nmat == 2 || (act != ACT_NONE && act != ACT_RELU));
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

// A workgroup reads all of x that its steps meet, so one that has few column
// tiles and a long K is bound by x, and few workgroups leave CUs idle.  Above
// four rows a K of 32 steps or more is split into parts of 8 steps at least, to
// two workgroups a CU at most, and joined (about 4 us): 4096 x 14336, 32 rows,
// 38.7 us whole against 23.9 + 3.9 in 4 parts (16 rows 22.4, 16.2 + 3.9); 512 x
// 12288 26.2 against 7.8 + 4.8.  Not split: 2048 x 2048 (8 steps) 7.5, in 4 parts
// 7.1 + 3.6; 8192 x 4096 (16 steps) 15.6, in 2 15.2 + 4.0; up to four rows, where
// x is small (512 x 12288, one row: 7.4, in 4 parts 4.9 + 2.2).
//
// Column tiles of a workgroup: one pair at q4_gated (12288 x 4096: 17.6 us at
// one row against 18.1 with three pairs, 41.0 at 32 rows against 42.7 with two).
// At q4_linear two where they fill the CUs (8192 x 4096, 32 rows: 15.6 against 19.2
// with one; 512 x 12288 in 8 parts: 9.0, with one 7.8).  Three, of which a CU holds
// one workgroup, where they make one round over the CUs and two would make a
// ragged one: more than two tiles a CU and at most three.  K = 4096, Q4_0, 16 rows:
// N = 8448 12.3 us against 13.7 with two, 12288 13.8 against 14.6, but 16384 23.2
// against 15.1; 32 rows 17.1 against 20.4, 19.2 / 21.1, 33.5 / 22.6; one row (K = 2048)
// 6.4 / 7.0, 6.9 / 7.3, 11.3 / 8.0, and 31.0 / 22.9 at N = 65536.  At 8 bits only at
// 5 to 16 rows (K = 2048, N = 8448, 16 rows 9.9 / 10.7; one row 9.7 / 9.3, and 32 rows
// 16.1 / 13.8, where the accumulators beside two dwords of codes spill).
// Eight waves where the workgroups do not outnumber the CUs (4096 x 4096 gated, 32
// rows: 16.4 against 20.8 with four).
FewPlan plan_few(int wf, int nmat, int64_t M, int64_t N, int64_t K) {
    const int64_t step = wf == WF_AFFINE8 ? 128 : 256, steps = (K + step - 1) / step;
    const int64_t tiles = (N + 15) / 16, cus = current_cu_count(), pairs = (tiles + 1) / 2;
    const int64_t most = M > 4 && steps >= 32 ? steps / 8 : 1;
    const bool fills = most > 1 ? pairs * most >= cus : tiles > cus;
    const bool three = most == 1 && tiles > 2 * cus && tiles <= 3 * cus && few_three(wf, M);
    FewPlan p{};
    p.tiles = nmat == 2 || !fills ? 1 : three ? 3 : 2;
    const int64_t groups = (tiles + p.tiles - 1) / p.tiles, room = 2 * cus / groups;
    const int64_t parts = room < 1 ? 1 : room < most ? room : most;
    p.per = (int)((steps + parts - 1) / parts);
    p.parts = (int)((steps + p.per - 1) / p.per);
    p.waves = M <= 4 || groups * p.parts <= cus ? 8 : 4;
    return p;
}

static int64_t few_rows_of(int64_t M) { return M <= kFewMaxM ? M : (M + 1) / 2; }
static int64_t few_part_row(int nmat, int64_t N) { return (N + 31) / 32 * nmat * 32; }

// Whatever the activation.
int64_t linear_workspace_bytes(int wf, int nmat, int dtype, int64_t M, int64_t N, int64_t K) {
    if (M > kFewCallMaxM) {
        const int64_t one = forward_layout(nmat, false, M, N, K).total;
        const int64_t two = dtype == DT_F16 ? forward_layout(nmat, true, M, N, K).total : 0;
        return one > two ? one : two;
    }
    const FewPlan p = plan_few(wf, nmat, few_rows_of(M), N, K);
    return p.parts > 1 ? p.parts * M * few_part_row(nmat, N) * 4 : 0;
}

// The few-row kernel on rows m0 .. m0 + count - 1.
static hipError_t launch_few(const LinearArgs& a, const FewPlan& p, int64_t m0, int64_t count, float* part, hipStream_t s) {
    LinearArgs t = a;
    auto rows = [&](const void* v, int64_t width) {
        return v ? const_cast<char*>(static_cast<const char*>(v)) + m0 * width * 2 : nullptr;
    };
    t.M = count;
    t.x = rows(a.x, a.K);
    t.y = rows(a.y, a.N);
    t.residual = rows(a.residual, a.N);
    for (int i = 0; i < 2; i++) t.pre[i] = rows(a.pre[i], a.N);
    FewSplit split{};
    split.rows = a.M;
    split.np = few_part_row(a.nmat, a.N);
    split.part = p.parts > 1 ? part + m0 * split.np : nullptr;
    return t.wf == WF_Q4_0      ? launch_few_q4_0(t, p, split, s)
           : t.wf == WF_AFFINE4 ? launch_few_affine4(t, p, split, s)
                                : launch_few_affine8(t, p, split, s);
}

static EpilogueArgs epilogue_args(const LinearArgs& a) {
    EpilogueArgs e{};
    e.act = a.act;
    e.dtype = a.dtype;
    e.M = a.M;
    e.N = a.N;
    for (int i = 0; i < 2; i++) {
        e.bias[i] = a.bias[i];
        e.pre[i] = a.pre[i];
    }
    e.residual = a.residual;
    e.y = a.y;
    return e;
}

hipError_t launch_linear(const LinearArgs& a, void* workspace, hipStream_t s) {
    if (a.M <= kFewCallMaxM) {
        const int64_t first = few_rows_of(a.M);
        const FewPlan p = plan_few(a.wf, a.nmat, first, a.N, a.K);
        float* part = static_cast<float*>(workspace);
        hipError_t e = launch_few(a, p, 0, first, part, s);
        if (e == hipSuccess && first < a.M) e = launch_few(a, p, first, a.M - first, part, s);
        if (e != hipSuccess || p.parts == 1) return e;
        TileArgs t{};
        t.part = part;
        t.parts = p.parts;
        t.unit = few_unit(a.wf, a.dtype);
        t.w_panels = (a.N + 31) / 32 * a.nmat;
        t.epi = epilogue_args(a);
        return launch_tile_join(a.nmat, t, s);
    }
    const bool rest = sums_rest(a.nmat, a.dtype, a.act);
    const Layout l = forward_layout(a.nmat, rest, a.M, a.N, a.K);
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    hipError_t e = launch_pack_weights(a.wf, a.nmat, a.w, a.N, a.K, false, rest, ws, s);
    if (e == hipSuccess)
        e = launch_pack_x(a.x, a.dtype, a.M, a.K, rest, ws + l.x_at, reinterpret_cast<int8_t*>(ws + l.exp_at), s);
    if (e != hipSuccess) return e;
    TileArgs t = tile_args(l, ws);
    t.epi = epilogue_args(a);
    return launch_tile_gemm(l.plan, a.nmat, t, s);
}

int64_t linear_grad_workspace_bytes(int, int nmat, int64_t M, int64_t N, int64_t K) {
    return backward_layout(nmat, M, N, K).total;
}

hipError_t launch_linear_grad(const LinearGradArgs& a, void* workspace, hipStream_t s) {
    const Layout l = backward_layout(a.nmat, a.M, a.N, a.K);
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    hipError_t e = launch_pack_weights(a.wf, a.nmat, a.w, a.N, a.K, true, false, ws, s);
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
