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
// of LDS slots (mx_ring) that direct-to-LDS copies fill from the planes: a copy is 16
// rows by 64 bytes (8 rows by 128 at 8 bits), so that four (eight) neighbouring
// lanes read whole lines, and the 16-byte pieces of a row are placed by an XOR with
// the row, so that the reads of an operand, 32 rows apart by a row's pitch, meet no
// bank twice.  The scales pass through LDS too, eight bytes a row and 256 k, which a
// shift by 8 h bits brings to the bytes that the instructions take (0 and 2 of
// either dword: blocks h, 2 + h, 4 + h, 6 + h).  What a copy would read past a row's end or behind
// the last row it takes from the row's last piece or from the last row: those
// blocks have the scale 2^-127 on both sides (nothing is left of their
// products), those rows are never stored.
//
// Bounds.  8-bit x: the matrix pipe and the power that it draws; 8192 x 8192 x 8192 in 409 us,
// 2.69 PFLOP/s (a loop of nothing but these instructions reaches 3.74, a library's 8-bit
// product 3.07), a step of 4 x 4 panels 2450 cycles of which 2048 are its MFMAs.
// Shorter sums pay the start and the end of a tile, 9000 to 22000 cycles: 2048 x 4096 x
// 12288 88 us, the gated pair of 2048 x 12288 x 4096 186 with both projections stored, 160 without.
// 4-bit x: 2048 x 12288 x 4096 in 79 us; a step of 4 x 4 panels takes 1880 cycles for 1024 of
// MFMAs.  Neither memory nor LDS is what it lacks: 4096 x 4096 x 16384 takes 151 us, 147 with every copy
// from the same lines, 124 without copies, and LDS is busy for 0.17 of its cycles, without a bank conflict.
// Its waves wait at the counters and barriers for 0.19 of their time, as many cycles as with 8-bit x, whose
// MFMAs take twice as long (matrix pipe 0.52 busy; 8 bits 0.79, 0.15): the schedule, in MFMAs, is that of
// 8-bit x.  Eight waves a workgroup instead of four (half the tile each, two waves a SIMD to hide each other's
// waits) were no faster: 81 us, and 98.5 against 97 at 2048 x 12288 x 4096 with 8-bit x.
#include "mx_tile.hpp"
#include "tile_epilogue.hpp"

namespace q4 {

namespace {

constexpr int kScaleUnit = 256;            // bytes of a panel's scales for 256 k

// copy_unit for four bytes a lane.
__device__ __forceinline__ void copy_dwords(const uint8_t* src, uint32_t voff, uint32_t m0) {
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dword %0, %1" : : "v"(voff), "s"(src), "s"(m0) : "memory", "m0");
}

typedef int i32x8_t __attribute__((ext_vector_type(8)));

// An address that is the same in all lanes, in scalar registers.
__device__ __forceinline__ const uint8_t* scalar(const uint8_t* p) {
    const uint64_t v = reinterpret_cast<uint64_t>(p);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)v), hi = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(v >> 32));
    return reinterpret_cast<const uint8_t*>((uint64_t)hi << 32 | lo);
}

}  // namespace

// ---- scales ----------------------------------------------------------------------
//
// A group of 256 k takes eight neighbouring scales of a row.  Where K is a multiple
// of 256 they are copied from the planes, else from images of them, [k / 256][row][8]
// with zeros past K: a thread takes a row's eight.
__global__ __launch_bounds__(256) void k_mx_scales(const MxTileArgs a) {
    const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t all = a.N * a.nmat + a.epi.M, t = id / all, i = id % all, nb = a.K / 32;
    if (t >= a.groups) return;
    const bool is_w = i < a.N * a.nmat;
    const int mat = is_w && i >= a.N ? 1 : 0;
    const int64_t row = is_w ? i - mat * a.N : i - a.N * a.nmat;
    const uint8_t* s = (is_w ? a.ws[mat] : a.xs) + row * nb;
    typedef u32x2_t u32x2_b __attribute__((aligned(1)));
    u32x2_t v = {0u, 0u};
    if (8 * t + 8 <= nb) {
        v = *reinterpret_cast<const u32x2_b*>(s + 8 * t);
    } else {
#pragma unroll
        for (int e = 0; e < 8; e++)
            if (8 * t + e < nb) v[e >> 2] |= (uint32_t)s[8 * t + e] << (8 * (e & 3));
    }
    reinterpret_cast<u32x2_t*>(a.scales)[t * all + i] = v;
}

// ---- the product -------------------------------------------------------------------

// Slots of the ring: what LDS holds, six at most -- from a copy to its use lie kRing - 1
// steps, 1400 cycles each at 4 x 2 panels, and memory may take two of them.  2 x 2
// panels take half of LDS, so that two workgroups share a CU.
template <int NT, int MT>
constexpr int mx_ring(int slot, int scale_slot) {
    const int lds = (NT * MT == 4 ? 80 : 160) * 1024;
    for (int r = 6; r > 3; r--)
        if (r * slot + (r / 2 + 1) * scale_slot <= lds) return r;
    return 3;
}
template <int NT, int MT, int EPI>
constexpr int wave_lds() {
    if constexpr (EPI == EPI_GATED) return 0;
    else return RowEpilogue<NT, MT, EPI>::kWaveB;
}

template <int NT, int MT, int XT, int EPI>
__global__ __launch_bounds__(256, 1) void k_mx_tile(const MxTileArgs a) {
    static_assert(EPI != EPI_GATED || NT % 2 == 0, "gate and up panels come in pairs");
    constexpr bool k8 = XT == XT_MXFP8;
    constexpr int kXR = k8 ? 2 : 1;                         // reads of an x fragment, copies of 16 rows of x
    constexpr int kWPanel = 2048, kXPanel = 2048 * kXR;     // bytes of a panel and step
    constexpr int kSlot = 2 * NT * kWPanel + 2 * MT * kXPanel;
    constexpr int kCopies = NT + MT * kXR;                  // of a wave and step, without the scales'
    constexpr int kScaleSlot = 2 * (NT + MT) * kScaleUnit;  // of two steps
    constexpr int kRing = mx_ring<NT, MT>(kSlot, kScaleSlot), kScaleRing = kRing / 2 + 1;
    constexpr int kData = kRing * kSlot, kLoop = kData + kScaleRing * kScaleSlot;
    constexpr int kWaveB = wave_lds<NT, MT, EPI>();          // the epilogue's tiles lie where the operands were
    constexpr int kScaleCopies = (NT + MT) / 2;             // of a wave and two steps
    __shared__ __attribute__((aligned(1024))) uint8_t lds[kLoop > 4 * kWaveB ? kLoop : 4 * kWaveB];

    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wn = wave & 1, wm = wave >> 1;

    // ---- the tile: workgroup b runs on XCD b mod 8; consecutive tiles v go to one
    // XCD, down the rows first, in groups of eight row tiles (as in tile_gemm.hip) ----
    // (counts of panels and tiles stay below 2^31: the launch's own limits)
    const uint32_t w_panels = (uint32_t)a.w_panels, x_panels = (uint32_t)((a.epi.M + 31) / 32);
    const uint32_t tiles_n = (w_panels + 2 * NT - 1) / (2 * NT), tiles_m = (x_panels + 2 * MT - 1) / (2 * MT);
    const uint32_t G = gridDim.x, xcd = blockIdx.x % 8, each = G / 8, rest = G % 8;
    uint32_t v = xcd * each + (xcd < rest ? xcd : rest) + blockIdx.x / 8;
    const int part = a.parts > 1 ? (int)(v / (tiles_n * tiles_m)) : 0;
    v -= (uint32_t)part * (tiles_n * tiles_m);
    const uint32_t group = v / (8 * tiles_n), left_m = tiles_m - group * 8;
    const uint32_t high = left_m < 8 ? left_m : 8;
    v -= group * 8 * tiles_n;
    const uint32_t pn0 = v / high * (2 * NT), pm0 = (group * 8 + v % high) * (2 * MT);

    // ---- copies.  The sum's groups of 256 k (two steps) t0 .. of this part ----
    const uint32_t groups = (uint32_t)a.groups;
    const int t0 = (int)((uint64_t)groups * part / a.parts), t1 = (int)((uint64_t)groups * (part + 1) / a.parts);
    const int S = 2 * (t1 - t0);                             // steps; one wholly past K has scales of zero
    const uint32_t row_w = (uint32_t)(a.K / 2), row_x = (uint32_t)(k8 ? a.K : a.K / 2);
    const uint32_t rows_w = (uint32_t)a.N, rows_x = (uint32_t)a.epi.M;
    const uint8_t* src[kCopies];                            // the first row of a copy's unit
    uint32_t at[kCopies];                                   // the lane's row in it, in bytes
#pragma unroll
    for (int t = 0; t < kCopies; t++) {
        const bool w = t < NT;
        // unit 4 t + wave of the tile's W (x): 16 rows of a panel, 8 at 8 bits
        const uint32_t u = (uint32_t)((w ? t : t - NT) * 4 + wave), per = w || !k8 ? 2 : 4, height = 32 / per;
        uint32_t p = (w ? pn0 : pm0) + u / per;
        const uint32_t last_p = (w ? w_panels : x_panels) - 1;
        p = p < last_p ? p : last_p;
        const bool up = w && a.nmat == 2 && (p & 1);
        const uint8_t* base = w ? (up ? a.wq[1] : a.wq[0]) : a.xq;
        const uint32_t rows = w ? rows_w : rows_x, pitch = w ? row_w : row_x;
        uint32_t first = (w && a.nmat == 2 ? p >> 1 : p) * 32 + u % per * height;
        first = first < rows ? first : rows - 1;
        const uint32_t in = rows - 1 - first, r = (uint32_t)lane / (64 / height);
        src[t] = base + (uint64_t)first * pitch;
        at[t] = (r < in ? r : in) * pitch;
    }
    // the lane's piece of a row: the XOR is by the row mod 16 (the unit's parity at 8 bits)
    const int wr = lane >> 2, xr = k8 ? (lane >> 3) + 8 * (wave & 1) : wr;
    auto swz4 = [](int r) { return ((r >> 1) & 3) ^ ((r >> 3) & 1); };
    auto swz8 = [](int r) { return (r & 7) ^ ((r >> 3) & 1); };
    const uint32_t piece_w = (uint32_t)(((lane & 3) ^ swz4(wr)) + 8 * t0);
    const uint32_t piece_x = k8 ? (uint32_t)(((lane & 7) ^ swz8(xr)) + 16 * t0) : piece_w;
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
    // the scales of a group: a copy is a panel's 32 rows by eight bytes
    const uint8_t* s_src[kScaleCopies];
    uint32_t s_at[kScaleCopies];
#pragma unroll
    for (int t = 0; t < kScaleCopies; t++) {
        const uint32_t u = (uint32_t)(t * 4 + wave);          // panel of the tile: W, then x
        const bool w = u < 2 * NT;
        uint32_t p = w ? pn0 + u : pm0 + u - 2 * NT;
        const uint32_t last_p = (w ? w_panels : x_panels) - 1;
        p = p < last_p ? p : last_p;
        const bool up = w && a.nmat == 2 && (p & 1);
        const uint32_t first = (w && a.nmat == 2 ? p >> 1 : p) * 32, in = (w ? rows_w : rows_x) - 1 - first, r = (uint32_t)lane >> 1;
        s_src[t] = scalar((w ? (up ? a.w_scales[1] : a.w_scales[0]) : a.x_scales) + (uint64_t)first * a.scale_row);
        s_at[t] = (r < in ? r : in) * a.scale_row + (uint32_t)(lane & 1) * 4;
    }
    auto copy_scales = [&](int g) __attribute__((always_inline)) {       // group g of this part
        const int t = t0 + g < t1 ? t0 + g : t1 - 1;
#pragma unroll
        for (int e = 0; e < kScaleCopies; e++)
            copy_dwords(scalar(s_src[e] + (int64_t)t * a.scale_group), s_at[e],
                        lds0 + (uint32_t)(kData + g % kScaleRing * kScaleSlot + (e * 4 + wave) * kScaleUnit));
    };

    floatx16_t acc[NT][MT];

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
    typedef uint64_t scale_t;
    scale_t sc[NT + MT], next_sc[NT + MT];
    auto read_scales = [&](int g, scale_t (&to)[NT + MT]) __attribute__((always_inline)) {
        const scale_t* p = reinterpret_cast<const scale_t*>(lds + kData + g % kScaleRing * kScaleSlot);
#pragma unroll
        for (int i = 0; i < NT; i++) to[i] = p[(wn * NT + i) * 32 + r];
#pragma unroll
        for (int j = 0; j < MT; j++) to[NT + j] = p[(2 * NT + wm * MT + j) * 32 + r];
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
        constexpr int kOp = 2 * (kByte & 1), kDword = 32 * (kByte >> 1);
        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(w, x, acc[i][j], 4, k8 ? 0 : 4, kOp, (int)(sc[i] >> kDword),
                                                                    kOp, (int)(sc[NT + j] >> kDword));
    };

    // ---- the schedule of a step: T MFMAs, the reads and copies between them ----
    constexpr int kM = NT * MT, T = 2 * kM;
    constexpr int B = 3 * T / 4;                            // the barrier stands before MFMA B
    constexpr int kEarly = MT * kXR + 2;                    // W0, x, W1 of half 0: read after the step before's barrier
    constexpr int kLate = 2 * kFrags - kEarly;              // the rest, and half 1: read before this step's barrier
    constexpr int kLead = T / 4 < 4 ? T / 4 : 4;            // MFMAs between the last of them and the barrier
    static_assert(B - kLead > 0, "room for the reads");
    // a step's copies run from a barrier to the next one's
    constexpr int kAfter = (kCopies * (T - B) + T - 1) / T;          // of them before the step's end

    auto step = [&](int i, auto odd) __attribute__((always_inline)) {
        constexpr int kOdd = decltype(odd)::value;
        const int slot = i % kRing, next = (i + 1) % kRing, before = (i + kRing - 1) % kRing;
        // the step whose copies end in this one is i + kRing - 1; the scales go with the even ones
        constexpr bool kScales = (kOdd + kRing - 1) % 2 == 0;
        constexpr int kAhead = kRing - 2, kAheadScales = (kAhead + (kOdd ? 0 : 1)) / 2;      // in flight at the barrier
        const uint8_t* here = lds + slot * kSlot;
        const uint8_t* there = lds + next * kSlot;
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int q = 0; q < T; q++) {
            if (q == B) {
                // the next step has landed (and its scales), the one after it is in flight
                step_barrier<kAhead * kCopies + kAheadScales * kScaleCopies>();
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
                // into the slot just read, for step i + kRing; the rest of the one before
                if (t < kAfter && B + t * (T - B) / kAfter == q) copy(t, slot);
                if (t >= kAfter && (t - kAfter) * B / (kCopies - kAfter) == q) copy(t, before);
            }
            if (kScales && q == 1) copy_scales((i + kRing - 1) >> 1);
            __builtin_amdgcn_sched_barrier(0);
        }
        if constexpr (kOdd) {
#pragma unroll
            for (int e = 0; e < NT + MT; e++) sc[e] = next_sc[e] >> (8 * h);
        }
    };

    auto clear = [&]() __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < NT; i++)
#pragma unroll
            for (int j = 0; j < MT; j++)
#pragma unroll
                for (int e = 0; e < 16; e++) acc[i][j][e] = 0.0f;
    };
    if (S > 0) {
#pragma unroll
        for (int p = 0; p < kRing - 1; p++) {
            if (p % 2 == 0) copy_scales(p / 2);
            stand();
#pragma unroll
            for (int t = 0; t < kCopies; t++) copy(t, p);
            ahead++;
        }
        stand();
#pragma unroll
        for (int t = 0; t < kAfter; t++) copy(t, kRing - 1);
        clear();                                             // while the copies travel
        step_barrier<(kRing - 2) * kCopies + (kRing - 2) / 2 * kScaleCopies + kAfter>();
        read_scales(0, sc);
#pragma unroll
        for (int e = 0; e < NT + MT; e++) sc[e] >>= 8 * h;
#pragma unroll
        for (int f = 0; f < kEarly; f++) read(f, lds, 0, fa);
        for (int i = 0; i < S; i += 2) {
            step(i, std::integral_constant<int, 0>{});
            step(i + 1, std::integral_constant<int, 1>{});
        }
    } else {
        clear();
    }

    // every copy has landed and every wave has read its last fragments
    step_barrier<0>();
    const int64_t n0 = (int64_t)(pn0 + wn * NT) * (EPI == EPI_GATED ? 16 : 32), m0 = (int64_t)(pm0 + wm * MT) * 32;
    auto finish = [&](auto vec, auto dtype) __attribute__((always_inline)) {
        constexpr bool kVec = decltype(vec)::value;
        constexpr int kDt = decltype(dtype)::value;
        if constexpr (EPI == EPI_GATED) gate_epilogue<NT, MT, kVec, kDt>(acc, a.epi, n0, m0);
        else row_epilogue<NT, MT, EPI, kVec, kDt>(acc, lds + wave * kWaveB, a.epi, a.part, part, a.w_panels, n0, m0);
    };
    using std::integral_constant;
    if constexpr (EPI == EPI_PARTIAL) {
        finish(integral_constant<bool, true>{}, integral_constant<int, DT_F32>{});
    } else if (a.epi.dtype == DT_BF16) {
        if (a.epi.N % 8 == 0) finish(integral_constant<bool, true>{}, integral_constant<int, DT_BF16>{});
        else finish(integral_constant<bool, false>{}, integral_constant<int, DT_BF16>{});
    } else {
        if (a.epi.N % 8 == 0) finish(integral_constant<bool, true>{}, integral_constant<int, DT_F16>{});
        else finish(integral_constant<bool, false>{}, integral_constant<int, DT_F16>{});
    }
}

// ---- host ------------------------------------------------------------------------

namespace {

int64_t panels_of(int64_t rows) { return (rows + 31) / 32; }
int64_t up256(int64_t n) { return (n + 255) / 256 * 256; }

// Cost of a plan in cycles: rounds of workgroups over the CUs, each a start and an
// end and its steps, as measured (8-bit x: 4 x 4 panels 2450 a step, of which 2048 its
// MFMAs; 4-bit x: 1880 of which 1024).  Rounds are counted by one workgroup a CU, also of 2 x 2
// panels, two of which share one: what sharing gains them is not measured.
double plan_cost(int nt, int mt, int parts, bool k8, int64_t w_panels, int64_t x_panels, int64_t steps, int cus) {
    const int64_t tiles = ((w_panels + 2 * nt - 1) / (2 * nt)) * ((x_panels + 2 * mt - 1) / (2 * mt));
    const int64_t rounds = (tiles * parts + cus - 1) / cus;
    const int size = nt * mt;                                // 16, 8 or 4
    const double ends = size == 16 ? 22000.0 : size == 8 ? 15000.0 : 9000.0;
    const double step = size == 16 ? (k8 ? 2450.0 : 1880.0) : size == 8 ? (k8 ? 1450.0 : 1300.0) : (k8 ? 800.0 : 700.0);
    // the parts' sums travel to memory and back, and a join is a launch more
    const double join = parts > 1 ? 6000.0 + 8.0 * parts * (double)(x_panels * w_panels) * 1024.0 / 2000.0 : 0.0;
    return rounds * (ends + step * (double)((steps + parts - 1) / parts)) + join;
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
    int64_t w_panels, groups, part_at, total;
    bool images;               // of the scales
};
Layout layout(int x_type, int nmat, int64_t M, int64_t N, int64_t K) {
    Layout l{};
    l.plan = plan_mx(x_type, nmat, M, N, K);
    l.w_panels = panels_of(N) * nmat;
    l.groups = (K + 255) / 256;
    l.images = K % 256 != 0;
    l.part_at = l.images ? up256(l.groups * (N * nmat + M) * 8) : 0;
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
    a.part = reinterpret_cast<float*>(ws + at.part_at);
    a.N = l.N;
    a.K = l.K;
    a.w_panels = at.w_panels;
    a.groups = at.groups;
    a.parts = at.plan.parts;
    a.epi = epi;
    const int64_t rows = l.N * l.nmat + l.M, threads = at.groups * rows;
    a.scales = ws;
    for (int i = 0; i < 2; i++) a.w_scales[i] = at.images ? ws + i * l.N * 8 : a.ws[i];
    a.x_scales = at.images ? ws + l.N * l.nmat * 8 : a.xs;
    a.scale_row = (uint32_t)(at.images ? 8 : l.K / 32);
    a.scale_group = at.images ? rows * 8 : 8;
    const TilePlan& plan = at.plan;
    const int64_t tiles = ((at.w_panels + 2 * plan.nt - 1) / (2 * plan.nt)) *
                          ((panels_of(l.M) + 2 * plan.mt - 1) / (2 * plan.mt)) * plan.parts;
    if (!launchable((threads + 255) / 256, 256) || !launchable(tiles, 256)) return hipErrorInvalidValue;
    if (at.images) hipLaunchKernelGGL(k_mx_scales, dim3((unsigned)((threads + 255) / 256)), dim3(256), 0, s, a);
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
