// mx_tile.hip -- mx_linear and mx_gated on MX x at many rows: Z[m][n] = sum_k
// X[m][k] W[n][k] straight from the planes on the scaled matrix instruction
// (v_mfma_scale_f32_32x32x64_f8f6f4), which takes 4-bit or 8-bit codes and a
// scale byte for each row and block of 32.
//
// Operands.  Lane l of the instruction holds row l & 31; with h = l >> 5, 4-bit
// codes of block h (16 bytes), 8-bit codes 16 h .. + 15 and 32 + 16 h .. + 15 of the
// 64, and in both cases the scale of block h.
//
// A workgroup of four waves owns a tile of 2 NT x 2 MT panels of 32 (columns x
// rows), each wave NT x MT of them.  The sum runs in steps of 128 k through a ring
// of three LDS slots that direct-to-LDS copies fill from the planes: a copy is 16
// rows by 64 bytes (8 rows by 128 at 8 bits), so that four (eight) neighbouring
// lanes read whole lines, and the 16-byte pieces of a row are placed by an XOR with
// the row, so that the reads of an operand, 32 rows apart by a row's pitch, meet no
// bank twice.  The scales come from images (k_mx_scales), a dword for lane and 256
// k, and pass through LDS too.  What a copy would read past a row's end or behind
// the last row it takes from the row's last piece or from the last row: those
// blocks have the scale 2^-127 on both sides (nothing is left of their
// products), those rows are never stored.
#include "mx_tile.hpp"
#include "tile_epilogue.hpp"

namespace q4 {

namespace {

constexpr int kRing = 3;
constexpr int kScaleUnit = 256;            // bytes of a panel's scales for 256 k

typedef int i32x8_t __attribute__((ext_vector_type(8)));

}  // namespace

// ---- scales ----------------------------------------------------------------------
//
// [t = k / 256][panel][lane]: byte s of the dword is the scale of row lane & 31 of
// the panel, block 8 t + 2 s + (lane >> 5): what the instruction s of those 256 k
// takes.  Blocks past K and rows past the last are 0.  A thread takes 512 k of a
// row, 16 neighbouring scales.
__global__ __launch_bounds__(256) void k_mx_scales(const MxTileArgs a) {
    const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t pairs = (a.groups + 1) / 2, row_id = id >> 5;
    const int64_t panel = row_id / pairs, t = row_id % pairs * 2;
    if (panel >= a.w_pad + a.x_pad) return;
    const bool is_w = panel < a.w_pad;
    const int64_t p = is_w ? panel : panel - a.w_pad, rows = is_w ? a.N : a.epi.M;
    const uint8_t* s = is_w ? a.ws[a.nmat == 2 ? p & 1 : 0] : a.xs;
    const int64_t row = (is_w ? p / a.nmat : p) * 32 + (id & 31), nb = a.K / 32, first = t * 8;
    uint32_t v[4] = {0u, 0u, 0u, 0u};
    if (row < rows) {
        const uint8_t* q = s + row * nb + first;
        typedef u32x4_t u32x4_b __attribute__((aligned(1)));
        if (first + 16 <= nb) {
            const u32x4_t r = *reinterpret_cast<const u32x4_b*>(q);
#pragma unroll
            for (int e = 0; e < 4; e++) v[e] = r[e];
        } else {
#pragma unroll
            for (int e = 0; e < 16; e++)
                if (first + e < nb) v[e >> 2] |= (uint32_t)q[e] << (8 * (e & 3));
        }
    }
    uint32_t* img = is_w ? a.w_scales : a.x_scales;
    const int64_t panels = is_w ? a.w_pad : a.x_pad;
#pragma unroll
    for (int g = 0; g < 2; g++) {
        if (t + g >= a.groups) break;
        uint32_t* out = img + ((t + g) * panels + p) * 64 + (id & 31);
        out[0] = __builtin_amdgcn_perm(v[2 * g + 1], v[2 * g], 0x06040200u);
        out[32] = __builtin_amdgcn_perm(v[2 * g + 1], v[2 * g], 0x07050301u);
    }
}

// ---- the product -------------------------------------------------------------------

template <int NT, int MT, int XT, int EPI>
__global__ __launch_bounds__(256, 1) void k_mx_tile(const MxTileArgs a) {
    static_assert(EPI != EPI_GATED || NT % 2 == 0, "gate and up panels come in pairs");
    constexpr bool k8 = XT == XT_MXFP8;
    constexpr int kXR = k8 ? 2 : 1;                         // reads of an x fragment, copies of 16 rows of x
    constexpr int kWPanel = 2048, kXPanel = 2048 * kXR;     // bytes of a panel and step
    constexpr int kSlot = 2 * NT * kWPanel + 2 * MT * kXPanel;
    constexpr int kCopies = NT + MT * kXR;                  // of a wave and step, without the scales'
    constexpr int kScaleSlot = 2 * (NT + MT) * kScaleUnit;  // of two steps
    constexpr int kRowF = tile_row_floats<NT>();
    constexpr int kData = kRing * kSlot, kLoop = kData + 2 * kScaleSlot, kTail = 4 * 32 * kRowF * 4;
    __shared__ __attribute__((aligned(1024))) uint8_t lds[kLoop > kTail ? kLoop : kTail];

    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wn = wave & 1, wm = wave >> 1;

    // ---- the tile: workgroup b runs on XCD b mod 8; consecutive tiles v go to one
    // XCD, down the rows first, in groups of eight row tiles (as in tile_gemm.hip) ----
    const int64_t x_panels = (a.epi.M + 31) / 32;
    const int64_t tiles_n = (a.w_panels + 2 * NT - 1) / (2 * NT), tiles_m = (x_panels + 2 * MT - 1) / (2 * MT);
    const int64_t G = gridDim.x, xcd = blockIdx.x % 8, each = G / 8, rest = G % 8;
    int64_t v = xcd * each + (xcd < rest ? xcd : rest) + blockIdx.x / 8;
    const int part = (int)(v / (tiles_n * tiles_m));
    v -= part * (tiles_n * tiles_m);
    const int64_t group = v / (8 * tiles_n), left_m = tiles_m - group * 8;
    const int64_t high = left_m < 8 ? left_m : 8;
    v -= group * 8 * tiles_n;
    const int64_t pn0 = v / high * (2 * NT), pm0 = (group * 8 + v % high) * (2 * MT);

    // ---- copies.  The sum's groups of 256 k (two steps) t0 .. of this part ----
    const int64_t t0 = a.groups * part / a.parts, t1 = a.groups * (part + 1) / a.parts;
    const int64_t all_steps = (a.K + 127) / 128;
    const int S = (int)((2 * t1 < all_steps ? 2 * t1 : all_steps) - 2 * t0);
    const uint32_t row_w = (uint32_t)(a.K / 2), row_x = (uint32_t)(k8 ? a.K : a.K / 2);
    const uint8_t* src[kCopies];                            // the first row of a copy's unit
    uint32_t at[kCopies];                                   // the lane's row in it, in bytes
#pragma unroll
    for (int t = 0; t < kCopies; t++) {
        const bool w = t < NT;
        // unit 4 t + wave of the tile's W (x): 16 rows of a panel, 8 at 8 bits
        const int u = (w ? t : t - NT) * 4 + wave, per = w || !k8 ? 2 : 4, height = 32 / per;
        int64_t p = (w ? pn0 : pm0) + u / per;
        const int64_t last_p = (w ? a.w_panels : x_panels) - 1;
        p = p < last_p ? p : last_p;
        const uint8_t* base = w ? a.wq[a.nmat == 2 ? p & 1 : 0] : a.xq;
        const int64_t rows = w ? a.N : a.epi.M, pitch = w ? row_w : row_x;
        int64_t first = (w ? p / a.nmat : p) * 32 + u % per * height;
        first = first < rows ? first : rows - 1;
        const int64_t in = rows - 1 - first, r = lane / (64 / height);
        src[t] = base + first * pitch;
        at[t] = (uint32_t)((r < in ? r : in) * pitch);
    }
    // the lane's piece of a row: the XOR is by the row mod 16 (the unit's parity at 8 bits)
    const int wr = lane >> 2, xr = k8 ? (lane >> 3) + 8 * (wave & 1) : wr;
    auto swz4 = [](int r) { return ((r >> 1) & 3) ^ ((r >> 3) & 1); };
    auto swz8 = [](int r) { return (r & 7) ^ ((r >> 3) & 1); };
    const uint32_t piece_w = (uint32_t)((lane & 3) ^ swz4(wr)) + (uint32_t)(8 * t0);
    const uint32_t piece_x = k8 ? (uint32_t)((lane & 7) ^ swz8(xr)) + (uint32_t)(16 * t0) : piece_w;
    const uint32_t last_w = row_w / 16 - 1, last_x = row_x / 16 - 1;
    const uint32_t lds0 = (uint32_t)reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) uint8_t*)lds);
    // The step that copies stand at; after the last one it is copied again (and
    // never read), so that a wait counts alike.
    int ahead = 0;
    uint32_t off_w = 0, off_x = 0;
    auto stand = [&]() __attribute__((always_inline)) {
        const uint32_t step = (uint32_t)(ahead < S ? ahead : S - 1);
        const uint32_t pw = piece_w + step * 4, px = piece_x + step * (k8 ? 8 : 4);
        off_w = (pw < last_w ? pw : last_w) * 16;
        off_x = (px < last_x ? px : last_x) * 16;
    };
    auto copy = [&](int t, int slot) __attribute__((always_inline)) {
        const bool w = t < NT;
        copy_unit(src[t], at[t] + (w ? off_w : off_x),
                  lds0 + (uint32_t)(slot * kSlot + (w ? 0 : 2 * NT * kWPanel) + ((w ? t : t - NT) * 4 + wave) * 1024));
    };
    // the scales of a group of 256 k: NT / 2 units of 1 KiB of W, MT / 2 of x; a wave
    // copies one (some twice)
    constexpr int kUnitsW = NT / 2, kUnitsS = NT / 2 + MT / 2;
    const int su = wave < kUnitsS ? wave : 0;
    const uint32_t* s_src = su < kUnitsW ? a.w_scales + (pn0 * 64 + su * 256) : a.x_scales + (pm0 * 64 + (su - kUnitsW) * 256);
    const int64_t s_pitch = (su < kUnitsW ? a.w_pad : a.x_pad) * 64;
    auto copy_scales = [&](int g) __attribute__((always_inline)) {       // group g of this part
        const int64_t t = t0 + g < t1 ? t0 + g : t1 - 1;
        copy_unit(reinterpret_cast<const uint8_t*>(s_src + t * s_pitch), (uint32_t)lane * 16,
                  lds0 + (uint32_t)(kData + (g & 1) * kScaleSlot + su * 1024));
    };

    floatx16_t acc[NT][MT];
#pragma unroll
    for (int i = 0; i < NT; i++)
#pragma unroll
        for (int j = 0; j < MT; j++)
#pragma unroll
            for (int e = 0; e < 16; e++) acc[i][j][e] = 0.0f;

    // ---- fragments of 64 k: half kk of a step ----
    const int r = lane & 31, h = lane >> 5;
    uint32_t at_w[2], at_x[2][kXR];                          // of the wave's first panel
#pragma unroll
    for (int kk = 0; kk < 2; kk++) {
        at_w[kk] = (uint32_t)(wn * NT * kWPanel + r * 64 + (((2 * kk + h) ^ swz4(r & 15)) * 16));
#pragma unroll
        for (int e = 0; e < kXR; e++)
            at_x[kk][e] = (uint32_t)(2 * NT * kWPanel + wm * MT * kXPanel +
                                     (k8 ? r * 128 + (((4 * kk + 2 * e + h) ^ swz8(r & 15)) * 16)
                                         : r * 64 + (((2 * kk + h) ^ swz4(r & 15)) * 16)));
    }
    constexpr int kFrags = NT + MT * kXR;                    // reads of a half: W0, x .., W1 ..
    struct Frags {
        u32x4_t w[NT], x[MT][kXR];
    };
    Frags fa, fb;
    auto read = [&](int f, const uint8_t* slot, int kk, Frags& fr) __attribute__((always_inline)) {
        if (f == 0 || f > MT * kXR) {
            const int i = f == 0 ? 0 : f - MT * kXR;
            fr.w[i] = *reinterpret_cast<const u32x4_t*>(slot + at_w[kk] + i * kWPanel);
        } else {
            const int j = (f - 1) / kXR, e = (f - 1) % kXR;
            fr.x[j][e] = *reinterpret_cast<const u32x4_t*>(slot + at_x[kk][e] + j * kXPanel);
        }
    };
    uint32_t sc[NT + MT], next_sc[NT + MT];
    auto read_scales = [&](int g, uint32_t (&to)[NT + MT]) __attribute__((always_inline)) {
        const uint32_t* p = reinterpret_cast<const uint32_t*>(lds + kData + (g & 1) * kScaleSlot);
#pragma unroll
        for (int i = 0; i < NT; i++) to[i] = p[(wn * NT + i) * 64 + lane];
#pragma unroll
        for (int j = 0; j < MT; j++) to[NT + j] = p[(2 * NT + wm * MT + j) * 64 + lane];
    };
    auto mfma = [&](int q, const Frags& fr, auto byte) __attribute__((always_inline)) {
        constexpr int kByte = decltype(byte)::value;
        const int i = q / MT, j = q % MT;
        i32x8_t w = {}, x = {};
#pragma unroll
        for (int e = 0; e < 4; e++) {
            w[e] = (int)fr.w[i][e];
            x[e] = (int)fr.x[j][0][e];
            if constexpr (k8) x[4 + e] = (int)fr.x[j][1][e];
        }
        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(w, x, acc[i][j], 4, k8 ? 0 : 4, kByte, (int)sc[i], kByte,
                                                                    (int)sc[NT + j]);
    };

    // ---- the schedule of a step: T MFMAs, the reads and copies between them ----
    constexpr int kM = NT * MT, T = 2 * kM;
    constexpr int B = 3 * T / 4;                            // the barrier stands before MFMA B
    constexpr int kEarly = MT * kXR + 2;                    // W0, x, W1 of half 0: read after the step before's barrier
    constexpr int kLate = 2 * kFrags - kEarly;              // the rest, and half 1: read before this step's barrier
    constexpr int kLead = T / 4 < 4 ? T / 4 : 4;            // MFMAs between the last of them and the barrier
    static_assert(B - kLead > 0, "room for the reads");
    // copies of the step after next but one run from a barrier to the next one's
    constexpr int kAfter = (kCopies * (T - B) + T - 1) / T;          // of them before the step's end

    auto step = [&](int i, auto odd) __attribute__((always_inline)) {
        constexpr int kOdd = decltype(odd)::value;
        const int slot = i % kRing, next = (i + 1) % kRing, third = (i + 2) % kRing;
        const uint8_t* here = lds + slot * kSlot;
        const uint8_t* there = lds + next * kSlot;
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int q = 0; q < T; q++) {
            if (q == B) {
                // the next step has landed (and its scales), the one after it is in flight
                step_barrier<kCopies + (kOdd ? 0 : 1)>();
                ahead++;
                stand();
                __builtin_amdgcn_sched_barrier(0);
                if (kOdd) read_scales((i >> 1) + 1, next_sc);
            }
            if (q < kM) mfma(q, fa, std::integral_constant<int, 2 * kOdd>{});
            else mfma(q - kM, fb, std::integral_constant<int, 2 * kOdd + 1>{});
#pragma unroll
            for (int f = 0; f < kLate; f++)
                if (f * (B - kLead) / kLate == q) {
                    if (f < kFrags - kEarly) read(f + kEarly, here, 0, fa);
                    else read(f - (kFrags - kEarly), here, 1, fb);
                }
#pragma unroll
            for (int f = 0; f < kEarly; f++)
                if (B + f * (T - B) / kEarly == q) read(f, there, 0, fa);
#pragma unroll
            for (int t = 0; t < kCopies; t++) {
                // into the slot just read, for the step after next but one; the rest of the one before
                if (t < kAfter && B + t * (T - B) / kAfter == q) copy(t, slot);
                if (t >= kAfter && (t - kAfter) * B / (kCopies - kAfter) == q) copy(t, third);
            }
            if (!kOdd && q == 1) copy_scales((i >> 1) + 1);
            __builtin_amdgcn_sched_barrier(0);
        }
        if constexpr (kOdd) {
#pragma unroll
            for (int e = 0; e < NT + MT; e++) sc[e] = next_sc[e];
        }
    };

    if (S > 0) {
        copy_scales(0);
        for (int p = 0; p < kRing - 1; p++) {
            stand();
#pragma unroll
            for (int t = 0; t < kCopies; t++) copy(t, p);
            ahead++;
        }
        stand();
#pragma unroll
        for (int t = 0; t < kAfter; t++) copy(t, kRing - 1);
        step_barrier<kCopies + kAfter>();
        read_scales(0, sc);
#pragma unroll
        for (int f = 0; f < kEarly; f++) read(f, lds, 0, fa);
        int i = 0;
        for (; i + 1 < S; i += 2) {
            step(i, std::integral_constant<int, 0>{});
            step(i + 1, std::integral_constant<int, 1>{});
        }
        if (i < S) step(i, std::integral_constant<int, 0>{});
    }

    // every copy has landed and every wave has read its last fragments
    step_barrier<0>();
    tile_epilogue<NT, MT, EPI>(acc, reinterpret_cast<float*>(lds) + wave * 32 * kRowF, a.epi, a.part, part, a.w_panels,
                               EPI == EPI_GATED ? (pn0 + wn * NT) * 16 : (pn0 + wn * NT) * 32, (pm0 + wm * MT) * 32,
                               [](int64_t) __attribute__((always_inline)) { return 1.0f; });
}

// ---- host ------------------------------------------------------------------------

namespace {

int64_t panels_of(int64_t rows) { return (rows + 31) / 32; }
int64_t padded(int64_t panels) { return (panels + 7) / 8 * 8; }
int64_t up256(int64_t n) { return (n + 255) / 256 * 256; }

// Cost of a plan in cycles (tile_gemm.hip's, on this kernel's steps).
double plan_cost(int nt, int mt, int parts, bool k8, int64_t w_panels, int64_t x_panels, int64_t steps, int cus) {
    const int64_t tiles = ((w_panels + 2 * nt - 1) / (2 * nt)) * ((x_panels + 2 * mt - 1) / (2 * mt));
    const int64_t rounds = (tiles * parts + cus - 1) / cus;
    const double mfma = 2.0 * (k8 ? 64.0 : 32.0) * nt * mt, lds = 96.0 * (nt + (k8 ? 2 : 1) * mt);
    const double step = (mfma > lds ? mfma : lds) + 100.0;
    const double one = 5000.0 + step * (double)((steps + parts - 1) / parts);
    const double join = parts > 1 ? 6000.0 + 8.0 * parts * (double)(x_panels * w_panels) * 1024.0 / 2000.0 : 0.0;
    return rounds * one + join;
}

TilePlan plan_mx(int x_type, int nmat, int64_t M, int64_t N, int64_t K) {
    const int64_t w_panels = panels_of(N) * nmat, x_panels = panels_of(M), steps = (K + 127) / 128;
    const int cus = current_cu_count();
    TilePlan best{4, 4, 1};
    double least = -1.0;
    constexpr int kShapes[][2] = {{4, 4}, {4, 2}, {2, 4}, {2, 2}};
    for (const auto& sh : kShapes)
        for (int parts = 1; parts <= 16; parts *= 2) {
            if (parts > 1 && steps / parts < 8) break;
            const double c = plan_cost(sh[0], sh[1], parts, x_type == XT_MXFP8, w_panels, x_panels, steps, cus);
            if (least < 0.0 || c < least) {
                least = c;
                best = TilePlan{sh[0], sh[1], parts};
            }
        }
    return best;
}

struct Layout {
    TilePlan plan;
    int64_t w_panels, w_pad, x_pad, groups, x_at, part_at, total;
};
Layout layout(int x_type, int nmat, int64_t M, int64_t N, int64_t K) {
    Layout l{};
    l.plan = plan_mx(x_type, nmat, M, N, K);
    l.w_panels = panels_of(N) * nmat;
    l.w_pad = padded(l.w_panels);
    l.x_pad = padded(panels_of(M));
    l.groups = (K + 255) / 256;
    l.x_at = up256(l.groups * l.w_pad * kScaleUnit);
    l.part_at = l.x_at + up256(l.groups * l.x_pad * kScaleUnit);
    l.total = l.part_at + partial_bytes(l.plan, M, l.w_panels);
    return l;
}

template <int NT, int MT, int XT>
void launch_shape(int epi, const MxTileArgs& a, unsigned grid, hipStream_t s) {
    if (epi == EPI_PARTIAL) hipLaunchKernelGGL((k_mx_tile<NT, MT, XT, EPI_PARTIAL>), dim3(grid), dim3(256), 0, s, a);
    else if (epi == EPI_GATED) hipLaunchKernelGGL((k_mx_tile<NT, MT, XT, EPI_GATED>), dim3(grid), dim3(256), 0, s, a);
    else hipLaunchKernelGGL((k_mx_tile<NT, MT, XT, EPI_LINEAR>), dim3(grid), dim3(256), 0, s, a);
}
template <int XT>
void launch_type(const TilePlan& p, int epi, const MxTileArgs& a, unsigned grid, hipStream_t s) {
    if (p.nt == 4 && p.mt == 4) launch_shape<4, 4, XT>(epi, a, grid, s);
    else if (p.nt == 4) launch_shape<4, 2, XT>(epi, a, grid, s);
    else if (p.mt == 4) launch_shape<2, 4, XT>(epi, a, grid, s);
    else launch_shape<2, 2, XT>(epi, a, grid, s);
}

}  // namespace

int64_t mx_tile_workspace_bytes(int x_type, int nmat, int64_t M, int64_t N, int64_t K) {
    return layout(x_type, nmat, M, N, K).total;
}

hipError_t launch_mx_tile(const MxLinearArgs& p, const EpilogueArgs& epi, void* workspace, hipStream_t s) {
    const LinearArgs& l = p.a;
    const Layout at = layout(p.x_type, l.nmat, l.M, l.N, l.K);
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    MxTileArgs a{};
    a.nmat = l.nmat;
    for (int i = 0; i < l.nmat; i++) {
        a.wq[i] = l.w[i].q;
        a.ws[i] = reinterpret_cast<const uint8_t*>(l.w[i].s);
    }
    a.xq = static_cast<const uint8_t*>(l.x);
    a.xs = p.x_s;
    a.w_scales = reinterpret_cast<uint32_t*>(ws);
    a.x_scales = reinterpret_cast<uint32_t*>(ws + at.x_at);
    a.part = reinterpret_cast<float*>(ws + at.part_at);
    a.N = l.N;
    a.K = l.K;
    a.w_panels = at.w_panels;
    a.w_pad = at.w_pad;
    a.x_pad = at.x_pad;
    a.groups = at.groups;
    a.parts = at.plan.parts;
    a.epi = epi;
    const int64_t threads = (at.w_pad + at.x_pad) * ((at.groups + 1) / 2) * 32;
    const TilePlan& plan = at.plan;
    const int64_t tiles = ((at.w_panels + 2 * plan.nt - 1) / (2 * plan.nt)) *
                          ((panels_of(l.M) + 2 * plan.mt - 1) / (2 * plan.mt)) * plan.parts;
    if (!launchable((threads + 255) / 256, 256) || !launchable(tiles, 256)) return hipErrorInvalidValue;
    hipLaunchKernelGGL(k_mx_scales, dim3((unsigned)((threads + 255) / 256)), dim3(256), 0, s, a);
    const int which = plan.parts > 1 ? EPI_PARTIAL : l.nmat == 2 ? EPI_GATED : EPI_LINEAR;
    if (p.x_type == XT_MXFP8) launch_type<XT_MXFP8>(plan, which, a, (unsigned)tiles, s);
    else launch_type<XT_MXFP4>(plan, which, a, (unsigned)tiles, s);
    if (plan.parts > 1) {
        TileArgs t{};
        t.part = a.part;
        t.parts = plan.parts;
        t.unit = 1.0f;
        t.w_panels = a.w_panels;
        t.epi = epi;
        return launch_tile_join(l.nmat, t, s);
    }
    return hipGetLastError();
}

}  // namespace q4
