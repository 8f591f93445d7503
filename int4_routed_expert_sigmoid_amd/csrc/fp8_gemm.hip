// Grouped products of FP8 rows with FP8 matrices: y[r][n] = sum over blocks b of 128 columns of
// sa[r][b] sw[n / 128][b] <a[r], w_e(r)[n]>_b, rows sorted by expert.
//
// v_mfma_f32_16x16x128_f8f6f4 multiplies 16 rows by 16 rows over one block: a lane holds 32 of the block's 128
// columns of row l % 16, here the 16-byte units l / 16 and l / 16 + 4 (a block's columns may be taken in any order,
// as long as both sides take the same). The block's sum (for its accuracy, and what results of 32 bits take in its
// place, see fp8.h) starts from 0 and enters the row's f32 sum by one multiplication: scales are any f32 numbers,
// so they cannot go into the instruction, which takes powers of two. The matrix rows are the first operand: result
// lane l then holds outputs n = 4 (l / 16) .. + 3 of one row m = l % 16, whose scale for the block is one number a
// lane, as the 16 matrix rows have one together.
//
// Bounds and times on one MI355X, where a copy moves 4.7 TB/s and a CU takes in about 35 GB/s from beyond its LDS:
//  - few rows: the matrices' bytes. 8192 x 8192, one to 16 rows, 67 MB: 17 us (4.0 TB/s); SwiGLU of 8 of 256
//    experts of 2048 x 6144, 201 MB: 41 (4.9).
//  - many rows: the matrix unit, in which a block of a tile takes 1.2 us of the 1.73 that it takes altogether. What
//    keeps the rest: a tile of 256 by 256 brings in 64 KB a block, 1.8 us at a CU's rate if nothing hits a cache
//    near by; and the four scalings of a product share the issue slots with the matrix instructions. 8191 x 8192 x
//    8192 into bf16: 446 to 474 us on several cards, 2.3 to 2.5 PFLOP/s; of 460 on one of them 16 go if every load
//    hits the L2 cache, 63 with no loads.
//  - SwiGLU of all of 256 experts of 2048 x 6144, 6.4 GB: 1.19 ms (5.6 TB/s) for 1 to 8 rows an expert and more.
#include <algorithm>
#include <cmath>

#include "fp8.h"

namespace coli {
namespace {

// FP8 rows as an output type of the SwiGLU epilogue; f32 rows on their way there (few_rows: exact products), or parts
// of sums on their way to 16 bits or to kFewValues FP8 values and more (tiles: the FP8 instruction's, as without parts).
struct Fp8Out {};
struct RawOut {};

// FP8 rows from exact products (fp8.h). A sum decides a code, and one that falls to the other side of a rounding
// border moves its value by up to an eighth: of the FP8 instruction's sums one in about 4000 does. Over a million
// values that is 1e-3 of a layer's output (509 tokens of 256 experts: 2.6e-3 off the 64-bit form, with exact sums
// 2.4e-3, bf16's own rounding), but of a few thousand a single large one can show (26 tokens, inter 288: 6.3e-3).
// Below kFewValues, and wherever few_rows runs (whose time is the matrices' bytes), FP8 rows therefore take exact
// products; above, the tiles' blocks would take 1.85 us in place of 1.03 (SwiGLU of 256 of 2048 x 6144, 16384 rows 1690
// in place of 1180, 8192 rows of one 349 / 185, the layer of 509 tokens 1373 / 1050).
struct ExactFp8Out {};
constexpr int64_t kFewValues = 1 << 20;

template <typename Out>
struct StoredAs {
    typedef Out type;
};
template <>
struct StoredAs<RawOut> {
    typedef float type;
};

typedef __attribute__((address_space(4))) const float const_f32;
typedef __attribute__((address_space(1))) const float global_float;

template <bool EXACT>
__device__ __forceinline__ f32x4 block_sum(const Frag& w, const Frag& a) {
    const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
    if constexpr (EXACT) return wide_mfma(widen(w, 1.f), widen(a, 1.f), zero);
    // 0: e4m3 operands; scale operands 0 select the form without scales
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(words8(w), words8(a), zero, 0, 0, 0, 0, 0, 0);
}

__device__ __forceinline__ void add_scaled(f32x4& acc, const f32x4& p, float s) {
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] = fmaf(p[i], s, acc[i]);
}

// The scale of a block of 128 h of a row from its largest |h|, and four of its codes.
__device__ __forceinline__ uint32_t codes4(const f32x4& h, float inv) { return fp8_codes4(h[0], h[1], h[2], h[3], inv); }

__device__ __forceinline__ uint32_t top4(const f32x4& h) {
    return max(max(abs_bits(h[0]), abs_bits(h[1])), max(abs_bits(h[2]), abs_bits(h[3])));
}

// ------------------------------------------------------------ few rows
// Workgroup: WN x KS waves, each NF fragments of 16 matrix rows (SwiGLU: gate and up in turn) by up to 16
// rows. KS waves take chunks of CB blocks in turn, and their sums meet in LDS in wave order. Everything
// goes straight into the instruction's registers; those of a block, one cache line of every row, are
// refilled for the wave's next chunk as soon as they are used. Whole chunks only (TAIL false) or any
// number of columns.
template <typename Out, bool SWIGLU, int NF, int WN, int KS, int CB, bool TAIL>
__global__ __launch_bounds__(64 * WN * KS) void fp8_few_rows_kernel(Fp8GemmArgs a, int NT) {
    constexpr bool kFp8 = std::is_same<Out, Fp8Out>::value;
    constexpr bool EXACT = kFp8 || std::is_same<Out, RawOut>::value || std::is_same<Out, float>::value;
    constexpr int kWaves = WN * KS, kCols = (SWIGLU ? NF / 2 : NF) * WN * kFrag;   // outputs of a tile
    static_assert(!kFp8 || kCols == kFp8Block, "a tile holds one block of h");
    __shared__ f32x4 part[KS][WN * NF][64];
    __shared__ uint32_t tops[8][kFrag];
    Unit u;
    if (!find_unit<kFrag>(a, NT, &u)) return;
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wn = wave % WN, ks = wave / WN;
    const int KB = (a.K + kFp8Block - 1) / kFp8Block, KU = a.K / kFp8Unit, chunks = (KB + CB - 1) / CB;
    const uint32_t row_bytes = a.K;
    const int n_tile = u.nt * kCols;
    const uint8_t* a_base = a.a + (int64_t)u.m0 * row_bytes;
    const int mr = min(r, u.rows - 1);
    const float* as_row = a.as + (int64_t)(u.m0 + mr) * KB;
    const uint8_t* w_base[2] = {u.blob + a.q_off + (int64_t)n_tile * row_bytes,
                                SWIGLU ? u.blob + a.up_q + (int64_t)n_tile * row_bytes : nullptr};
    uint32_t nr[NF];                             // the row of the tile, in bytes
    const_f32* ws_row[NF];
#pragma unroll
    for (int f = 0; f < NF; ++f) {
        const int x = wn * NF + f, at = (SWIGLU ? x / 2 : x) * kFrag;
        nr[f] = (uint32_t)min(at + r, a.N - 1 - n_tile) * row_bytes;
        ws_row[f] = (const_f32*)(u.blob + (SWIGLU && f % 2 ? a.up_s : a.s_off)) +
                    (int64_t)(min(n_tile + at, a.N - 1) / kFp8Block) * KB;
    }

    Frag w[CB][NF], av[CB];
    float as[CB], ws[CB][NF];
    auto load_block = [&](int c, int s) {
        const int b = c * CB + s;
        int u0 = b * 8 + g, u1 = u0 + 4;
        if (TAIL) u0 = min(u0, KU - 1), u1 = min(u1, KU - 1);
#pragma unroll
        for (int f = 0; f < NF; ++f) {
            const uint8_t* base = w_base[SWIGLU ? f % 2 : 0];
            w[s][f].lo = load16(base + (nr[f] + u0 * 16));
            w[s][f].hi = load16(base + (nr[f] + u1 * 16));
        }
        av[s].lo = load16(a_base + (mr * row_bytes + u0 * 16));
        av[s].hi = load16(a_base + (mr * row_bytes + u1 * 16));
    };
    auto load_scales = [&](int c) {
#pragma unroll
        for (int s = 0; s < CB; ++s) {
            const int b = TAIL ? min(c * CB + s, KB - 1) : c * CB + s;
            as[s] = *(global_float*)(as_row + b);
#pragma unroll
            for (int f = 0; f < NF; ++f) ws[s][f] = ws_row[f][b];
        }
    };
    f32x4 acc[NF];
#pragma unroll
    for (int f = 0; f < NF; ++f) acc[f] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (ks < chunks) {
        load_scales(ks);
#pragma unroll
        for (int s = 0; s < CB; ++s) load_block(ks, s);
    }
    for (int c = ks; c < chunks; c += KS) {
        const bool more = c + KS < chunks;
        float as_c[CB], ws_c[CB][NF];
#pragma unroll
        for (int s = 0; s < CB; ++s) {
            const bool behind = TAIL && c * CB + s >= KB;     // (0 on both sides: the other may be infinite)
            as_c[s] = behind ? 0.f : as[s];
#pragma unroll
            for (int f = 0; f < NF; ++f) ws_c[s][f] = behind ? 0.f : ws[s][f];
        }
        if (more) load_scales(c + KS);
#pragma unroll
        for (int s = 0; s < CB; ++s) {
            Frag x = av[s];
            if (TAIL) {                          // units behind the row: 0 on one side
                const int u0 = (c * CB + s) * 8 + g;
                if (u0 >= KU) x.lo = u32x4{0, 0, 0, 0};
                if (u0 + 4 >= KU) x.hi = u32x4{0, 0, 0, 0};
            }
            f32x4 p[NF];
#pragma unroll
            for (int f = 0; f < NF; ++f) p[f] = block_sum<EXACT>(w[s][f], x);
#pragma unroll
            for (int f = 0; f < NF; ++f) add_scaled(acc[f], p[f], as_c[s] * ws_c[s][f]);
            hold(acc);
            if (more) load_block(c + KS, s);
        }
    }
#pragma unroll
    for (int f = 0; f < NF; ++f) part[ks][wn * NF + f][lane] = acc[f];
    __syncthreads();
    auto sum = [&](int f) {
        f32x4 v = part[0][f][lane];
#pragma unroll
        for (int k = 1; k < KS; ++k) v += part[k][f][lane];
        return v;
    };
    const bool live = r < u.rows;
    const int m = u.m0 + r;
    if constexpr (!SWIGLU) {
        for (int o = wave; o < WN * NF; o += kWaves) {
            const f32x4 v = sum(o);
            const int n0 = n_tile + o * kFrag + 4 * g;
            if (live && n0 < a.N) store4<Out>(a, m, n0, a.N, v);
        }
    } else {
        constexpr int kOut = WN * NF / 2, kPer = (kOut + kWaves - 1) / kWaves;
        f32x4 h[kPer];
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int o = i * kWaves + wave;
            if (o >= kOut) break;
            const f32x4 gv = sum(2 * o), uv = sum(2 * o + 1);
#pragma unroll
            for (int x = 0; x < 4; ++x) h[i][x] = silu_mul(gv[x], uv[x]);
            const int n0 = n_tile + o * kFrag + 4 * g;
            if constexpr (kFp8) {
                uint32_t top = n0 < a.N ? top4(h[i]) : 0u;
                top = umax_step<16>(top);
                top = umax_step<32>(top);
                if (g == 0) tops[o][r] = top;
            } else {
                if (live && n0 < a.N) store4<typename StoredAs<Out>::type>(a, m, n0, a.N, h[i]);
            }
        }
        if constexpr (kFp8) {
            __syncthreads();
            uint32_t top = 0;
#pragma unroll
            for (int o = 0; o < kOut; ++o) top = max(top, tops[o][r]);
            const int code = fp8_scale_code(top);
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const int o = i * kWaves + wave, n0 = n_tile + o * kFrag + 4 * g;
                if (o < kOut && live && n0 < a.N)
                    *(uint32_t*)((uint8_t*)a.y + (int64_t)m * a.N + n0) = codes4(h[i], fp8_scale_inverse(code));
            }
            if (wave == 0 && g == 0 && live) a.ys[(int64_t)m * fp8_blocks(a.N) + u.nt] = fp8_scale_value(code);
        }
    }
}

// ------------------------------------------------------------ many rows: both sides over LDS
// Persistent workgroups of WM x WN waves, each MT fragments of rows (those with number i * WM + wm) by NF
// fragments of matrix rows (SwiGLU: gate and up in turn). Codes and scales go from memory straight into
// LDS, a block of 128 columns (one cache line of every row) at a time, STAGES blocks ahead and on into the
// workgroup's next unit. A wave waits for its own loads of a block by count and meets the others at one
// barrier a block, once it has the block's last fragments in registers: from there on the slot is filled
// again while the last row of fragments is multiplied and the next block's first ones are read.
// A product is scaled into its sum while the next row's are in the matrix unit: the four multiply-adds of one
// product take half of its time there.
// Tiles of 256 rows in two stages of 64 KB and tiles of 128 in three of 48: two workgroups a CU would leave each half
// of the rows and read everything twice (8191 x 8192 x 8192: 534 us by tiles of 128).
// FAST: K in multiples of 512 and rows of scales on 16-byte boundaries: scales come 16 bytes, four blocks, a
// row, and every unit is whole. Otherwise one block's at a time, and zeros behind the last column.
// PARTS: each unit once for every part of the columns, into an output of its own (product_parts).
template <typename Out, bool SWIGLU, int MT, int NF, int WM, int WN, int STAGES, bool FAST>
struct LineTile {
    static constexpr bool kFp8 = std::is_same<Out, Fp8Out>::value || std::is_same<Out, ExactFp8Out>::value;
    static constexpr int BM = WM * MT * kFrag, BN = WN * NF * kFrag, kWaves = WM * WN, kThreads = 64 * kWaves;
    static constexpr int U = kBlockUnits;
    static constexpr int kCols = SWIGLU ? BN / 2 : BN;        // outputs of a tile
    static constexpr int kLoads = (BM + BN) * U / kThreads;   // code loads of a wave and block
    static constexpr int kARows = BM * U / kThreads;          // of them for the rows
    static constexpr int kScaleLoads = BM / 64 + 1;           // 64 rows each, and the matrix' blocks
    static constexpr int kGroup = FAST ? 4 : 1;               // blocks whose scales come together
    static constexpr int kStores = kFp8 ? MT : SWIGLU ? MT * NF / 2 : MT * (int)sizeof(typename StoredAs<Out>::type);   // of a wave and whole tile
    static_assert(BM * U % kThreads == 0 && BN * U % kThreads == 0, "whole loads for every wave");
    static_assert(kScaleLoads <= kWaves && BM % 64 == 0, "one scale load a wave");
    static_assert((MT == 4 || MT == 8) && NF == 4 && kWaves == 8, "the ring of row fragments; 64 columns and 8 rows a wave");
    static_assert(STAGES == 2 || STAGES == 3, "the stores that a wait may leave in flight");
    static_assert(kCols % kFp8Block == 0 && NF * kFrag <= kFp8Block, "a wave's fragments share their scales");
    struct Lds {
        u32x4 code[STAGES][(BM + BN) * U];                    // rows, then matrix rows
        // The scales of a group of blocks: rows, then the matrix' blocks. A slot is filled again STAGES groups
        // later, for a block at least STAGES behind the last one that reads it.
        float scale[STAGES][(BM + 64) * kGroup];
        uint32_t first[kMaxExperts];                          // first unit of every expert
        uint32_t top[kFp8 ? WN * BM : 1];
    };
};

struct Place {
    void* y;
    int64_t ld;
};

struct PartUnit : LineUnit {
    int lo, hi, part;                        // blocks of columns
};

template <typename Out, bool SWIGLU, int MT, int NF, int WM, int WN, int STAGES, bool FAST, bool PARTS>
__global__ __launch_bounds__(64 * WM * WN, 2) void fp8_line_kernel(Fp8GemmArgs a, int NT) {
    typedef typename StoredAs<Out>::type Stored;
    typedef LineTile<Out, SWIGLU, MT, NF, WM, WN, STAGES, FAST> T;
    constexpr int U = T::U, kGroup = T::kGroup, kW = SWIGLU ? 2 : 1;
    constexpr bool EXACT = std::is_same<Out, float>::value || std::is_same<Out, ExactFp8Out>::value;
    __shared__ typename T::Lds lds;
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wn = wave % WN, wm = wave / WN;
    const int KB = (a.K + kFp8Block - 1) / kFp8Block, KU = a.K / kFp8Unit;
    const uint32_t row_bytes = a.K;

    const uint32_t units = scan_units<T::BM, T::kThreads>(a, NT, lds.first, (uint32_t*)lds.scale[0]);
    const uint32_t total = PARTS ? units * a.parts : units;
    const uint32_t per = (total + kXcds - 1) / kXcds, xcd = blockIdx.x % kXcds, step = gridDim.x / kXcds;
    auto unit_at = [&](uint32_t x) {
        const uint32_t w = xcd * per + x;
        const bool live = x < per && w < total;
        PartUnit u;
        u.part = PARTS && live ? w / units : 0;
        (LineUnit&)u = line_unit<T::BM>(a, NT, lds.first, w - u.part * units, live);
        const int groups = (KB + 3) / 4;     // whole groups of scales to a part
        u.lo = PARTS ? groups * u.part / a.parts * 4 : 0;
        u.hi = PARTS ? min(groups * (u.part + 1) / a.parts * 4, KB) : KB;
        return u;
    };
    uint32_t at = blockIdx.x / kXcds;        // this workgroup's units: at, at + step, ... of its XCD's `per`
    PartUnit u = unit_at(at);
    if (u.rows <= 0) return;

    // the unit that is being loaded
    uint32_t load_at = at;
    const uint8_t *w_base, *a_base, *scale_base;
    int lc = 0, load_hi = 0;                 // its next block, and the one behind its last
    bool loading = true;
    uint32_t a_max, w_max;                   // a lane's place in the last row, and in the last matrix row
    const int sx = min(wave, T::kScaleLoads - 1);
    // A load takes 8 rows, lane l row l / 8, position l % 8; of a wave's loads i each is kStep rows below the
    // one before. SwiGLU: the tile's fragments are gate's and up's in turn, two loads each, and as there are 8
    // waves, all of a wave's are of one matrix.
    const int unit = (lane & 7) ^ (lane >> 3);
    constexpr int kStepA = 8 * T::kWaves, kStepW = SWIGLU ? kStepA / 2 : kStepA;
    const int a_row = wave * 8 + (lane >> 3);
    const int w_row = SWIGLU ? wave / 4 * kFrag + wave % 2 * 8 + (lane >> 3) : a_row;
    const bool up = SWIGLU && wave / 2 % 2 == 1;
    const uint32_t a_lane = a_row * row_bytes + unit * 16, w_lane = w_row * row_bytes + unit * 16;
    auto set_unit = [&](const PartUnit& v) {
        const int n_tile = v.nt * T::kCols;
        const int m_last = v.rows - 1, n_last = a.N - 1 - n_tile;
        a_max = m_last * row_bytes + unit * 16;
        w_max = min(n_last, T::BN) * row_bytes + unit * 16;
        w_base = v.blob + (up ? a.up_q : a.q_off) + (int64_t)n_tile * row_bytes;
        a_base = a.a + (int64_t)v.m0 * row_bytes;
        // rows' scales: 64 rows from sx * 64 on; the matrix': lane 0 and 1 its two blocks, or gate's and up's
        if (sx < T::BM / 64) {
            scale_base = (const uint8_t*)(a.as + (int64_t)(v.m0 + min(sx * 64 + lane, m_last)) * KB);
        } else {
            const int block = n_tile / kFp8Block, last = (a.N - 1) / kFp8Block;
            const size_t off = SWIGLU && lane > 0 ? a.up_s : a.s_off;
            const int b = SWIGLU ? block : min(block + min(lane, T::BN / kFp8Block - 1), last);
            scale_base = v.blob + off + (int64_t)b * KB * 4;
        }
        lc = v.lo;
        load_hi = v.hi;
    };
    // Load i of this wave for the block. Behind the last unit the same number of loads goes out, so that the
    // counts hold, of its first block again and into slots that are not read.
    auto load_codes = [&](int slot, int i) {
        const bool rows = i < T::kARows;
        const int j = rows ? i : i - T::kARows, below = j * (rows ? kStepA : kStepW);
        // (rows behind the last are the last)
        const uint32_t off = min((rows ? a_lane : w_lane) + (uint32_t)below * row_bytes, rows ? a_max : w_max);
        const uint8_t* p = (rows ? a_base : w_base) + (uint32_t)lc * kFp8Block + off;
        if (!FAST && lc * U + unit >= KU) p = (const uint8_t*)&kZeroUnit;
        load_to_lds(p, lds.code[slot] + ((rows ? 0 : T::BM / 8) + j * T::kWaves + wave) * 64);
    };
    int fill_scale = 0;                      // the scale slot that is filled next
    auto load_scales = [&]() {
        if (!loading || lc % kGroup != 0) return;
        float* dst = lds.scale[fill_scale] + sx * 64 * kGroup;
        if constexpr (FAST) load_to_lds(scale_base + lc * 4, (u32x4*)dst);
        else load4_to_lds(scale_base + lc * 4, (uint32_t*)dst);
        fill_scale = fill_scale == STAGES - 1 ? 0 : fill_scale + 1;
    };
    auto advance = [&]() {                   // to the block that is loaded next
        if (!loading || ++lc < (PARTS ? load_hi : KB)) return;
        lc = 0;
        load_at += step;
        const PartUnit v = unit_at(load_at);
        loading = v.rows > 0;
        if (loading) set_unit(v);
    };

    set_unit(u);
    __syncthreads();                         // the scan's scratch is a scale slot
#pragma unroll
    for (int c = 0; c < STAGES; ++c) {
        load_scales();
#pragma unroll
        for (int i = 0; i < T::kLoads; ++i) load_codes(c, i);
        advance();
    }

    // fragments: rows 16 apart have the same place in their unit's permutation
    const int m_lds = wm * kFrag + r, n_lds = T::BM + wn * NF * kFrag + r;
    const int lo = g ^ (r & 7), hi = (g + 4) ^ (r & 7);
    int slot = 0, scales = 0;                // of the block that is multiplied
    auto code = [&](int row, int below) {
        const u32x4* p = lds.code[slot] + below * U;
        return Frag{p[row * U + lo], p[row * U + hi]};
    };
    const int ws_row = T::BM + (SWIGLU ? 0 : wn * NF * kFrag / kFp8Block);
    // The steps of a block, a product each: row by row, and of the last two rows, from step kMeet on, both with one
    // matrix fragment after the other, so that the next block's can be read one by one meanwhile. The row
    // fragments take turns in a few registers.
    constexpr int kMeet = (MT - 2) * NF;
    auto row_of = [](int n) constexpr { return n < kMeet ? n / NF : MT - 2 + (n - kMeet) % 2; };
    auto frag_of = [](int n) constexpr { return n < kMeet ? n % NF : (n - kMeet) / 2; };
    auto ring = [](int i) constexpr { return MT == 4 || i < 2 ? i : i < 4 ? i - 2 : i == 4 ? 2 : i - 5; };   // 0 1 0 1 2 0 1 2
    constexpr int kRing = MT == 4 ? 4 : 3;
    Frag w[NF], av[kRing];
    float as[kRing], ws[kW], s_last[2 * kW];  // s_last: the scales of the block before, rows MT - 2 and MT - 1
    f32x4 acc[MT][NF], p[4];
    auto read_scales = [&](int b) {
#pragma unroll
        for (int x = 0; x < kW; ++x) ws[x] = lds.scale[scales][(ws_row + x) * kGroup + b % kGroup];
    };
    auto read_row = [&](int i, int b) {
        av[ring(i)] = code(m_lds, i * WM * kFrag);
        as[ring(i)] = lds.scale[scales][m_lds * kGroup + b % kGroup + i * WM * kFrag * kGroup];
    };
    // How many tiles' stores may be in flight behind the loads of the block that is waited for next: those of
    // the last STAGES - 1 blocks' units.
    int stores[2] = {0, 0};
    wait_loads<(STAGES - 1) * T::kLoads>();
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
#pragma unroll
    for (int f = 0; f < NF; ++f) w[f] = code(n_lds, f * kFrag);
    read_scales(0);
    read_row(0, 0);
    if constexpr (MT == 4) read_row(1, 0);
    while (true) {
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int f = 0; f < NF; ++f) acc[i][f] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int x = 0; x < 4; ++x) p[x] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int x = 0; x < 2 * kW; ++x) s_last[x] = 0.f;
#pragma unroll 1
        for (int c = PARTS ? u.lo : 0; c < (PARTS ? u.hi : KB); ++c) {
            const int fill = slot, next = c + 1 == (PARTS ? u.hi : KB) ? 0 : c + 1;   // (a part begins with a group of scales)
            float s[MT][kW];
            Wide ww[EXACT ? NF : 1], aw[EXACT ? 2 : 1];
            if constexpr (EXACT) {
#pragma unroll
                for (int f = 0; f < NF; ++f) ww[f] = widen(w[f], 1.f);
            }
            // four steps by bf16 in turn, as the four instructions of one wait for each other
            auto wide_steps = [&](int n) {
                if (n <= kMeet) aw[0] = widen(av[ring(row_of(n))], 1.f);
                if (n == kMeet) aw[EXACT] = widen(av[ring(MT - 1)], 1.f);
#pragma unroll
                for (int x = 0; x < 4; ++x) p[x] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int k = 0; k < 4; ++k)
#pragma unroll
                    for (int x = 0; x < 4; ++x)
                        p[x] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ww[EXACT ? frag_of(n + x) : 0].v[k],
                                                                       aw[EXACT && row_of(n + x) == MT - 1].v[k], p[x], 0, 0, 0);
            };
#pragma unroll
            for (int n = 0; n < MT * NF; ++n) {
                const int i = row_of(n), f = frag_of(n);
                if (n == kMeet) {
                    // The next block and its scales (issued before its codes) have arrived, the codes of the
                    // STAGES - 2 behind it may not have, and this one is read.
                    wait_behind_stores<(STAGES - 2) * T::kLoads, T::kStores>(STAGES == 3 ? stores[0] + stores[1] : stores[0]);
                    if constexpr (STAGES == 3) stores[1] = stores[0];
                    stores[0] = 0;
                    __builtin_amdgcn_s_barrier();
                    asm volatile("" ::: "memory");
                    slot = slot == STAGES - 1 ? 0 : slot + 1;
                    if (next % kGroup == 0) scales = scales == STAGES - 1 ? 0 : scales + 1;
                    load_scales();
                }
                if (f == 0) {
#pragma unroll
                    for (int x = 0; x < kW; ++x) s[i][x] = as[ring(i)] * ws[x];
                }
                if (n < kMeet && f == 0) {               // rows of this block
                    if (MT == 4 && i == 0) read_row(2, c), read_row(3, c);
                    if (MT == 8) read_row(i + 1, c);
                    if (MT == 8 && i == MT - 3) read_row(MT - 1, c);
                }
                if (n == kMeet + 1) read_row(0, next);   // of the next
                if (n == kMeet + 3 && MT == 4) read_row(1, next);
                // the product of four steps before into its sum
                const int m = (n + MT * NF - 4) % (MT * NF), mi = row_of(m), mf = frag_of(m), mx = SWIGLU ? mf % 2 : 0;
                add_scaled(acc[mi][mf], p[n % 4], n < 4 ? s_last[(mi - (MT - 2)) * kW + mx] : s[mi][mx]);
                if constexpr (!EXACT) p[n % 4] = block_sum<false>(w[f], av[ring(i)]);
                else if (n % 4 == 3) wide_steps(n - 3);
                asm volatile("" : "+v"(acc[mi][mf])::"memory");
                if (n >= kMeet) {
                    if (i == MT - 1) w[f] = code(n_lds, f * kFrag);
                    const int q = n - kMeet;
#pragma unroll
                    for (int x = q * T::kLoads / 8; x < (q + 1) * T::kLoads / 8; ++x) load_codes(fill, x);
                }
                if (n == kMeet + 2) read_scales(next);   // (those of this block's last rows are multiplied)
            }
#pragma unroll
            for (int x = 0; x < 2 * kW; ++x) s_last[x] = s[MT - 2 + x / kW][x % kW];
            advance();
        }
#pragma unroll
        for (int n = MT * NF - 4; n < MT * NF; ++n) {
            const int i = row_of(n), f = frag_of(n);
            add_scaled(acc[i][f], p[n % 4], s_last[(i - (MT - 2)) * kW + (SWIGLU ? f % 2 : 0)]);
        }
        // outputs
        const int n_wave = u.nt * T::kCols + wn * (SWIGLU ? NF / 2 : NF) * kFrag;
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            const int row = m_lds + i * WM * kFrag, m = u.m0 + row;
            const bool there = row < u.rows;
            if constexpr (!SWIGLU) {
                const int m0 = (i * WM + wm) * kFrag;
                Stored* y = (Stored*)a.y + (PARTS ? (int64_t)u.part * a.rows * a.ld : 0);
                if (n_wave + NF * kFrag <= a.N) {         // uniform
                    store64<Stored>(y + (int64_t)(u.m0 + m0) * a.ld + n_wave, a.ld, u.rows - m0, acc[i][0], acc[i][1], acc[i][2],
                                    acc[i][3]);
                } else if (there) {
#pragma unroll
                    for (int f = 0; f < NF; ++f) {
                        const int n0 = n_wave + f * kFrag + 4 * g;
                        if (n0 < a.N) store4<Stored>(Place{y, a.ld}, m, n0, a.N, acc[i][f]);
                    }
                }
            } else if constexpr (PARTS) {                 // gate's sums and up's, N each a row
                float* y = (float*)a.y + (int64_t)u.part * a.rows * a.ld;
#pragma unroll
                for (int f = 0; f < NF; ++f) {
                    const int n0 = n_wave + f / 2 * kFrag + 4 * g;
                    if (there && n0 < a.N) store4<float>(Place{y + (f % 2 ? a.N : 0), a.ld}, m, n0, a.N, acc[i][f]);
                }
            } else {
#pragma unroll
                for (int x = 0; x < NF / 2; ++x) {
                    f32x4 h;
#pragma unroll
                    for (int y = 0; y < 4; ++y) h[y] = silu_mul(acc[i][2 * x][y], acc[i][2 * x + 1][y]);
                    acc[i][2 * x] = h;
                    const int n0 = n_wave + x * kFrag + 4 * g;
                    if constexpr (!T::kFp8) {
                        if (there && n0 < a.N) store4<Out>(a, m, n0, a.N, h);
                    }
                }
            }
        }
        if constexpr (T::kFp8) {
            // a row's largest |h| of the tile's 128, a wave's 32 of them at a time
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                uint32_t top = 0;
#pragma unroll
                for (int x = 0; x < NF / 2; ++x)
                    if (n_wave + x * kFrag + 4 * g < a.N) top = max(top, top4(acc[i][2 * x]));
                top = umax_step<16>(top);
                top = umax_step<32>(top);
                if (g == 0) lds.top[wn * T::BM + m_lds + i * WM * kFrag] = top;
            }
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            __builtin_amdgcn_s_barrier();
            asm volatile("" ::: "memory");
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                const int row = m_lds + i * WM * kFrag, m = u.m0 + row;
                uint32_t top = 0;
#pragma unroll
                for (int x = 0; x < WN; ++x) top = max(top, lds.top[x * T::BM + row]);
                const int code = fp8_scale_code(top);
                const float inv = fp8_scale_inverse(code);
                // 8 neighbouring codes a lane
                uint32_t q[2] = {codes4(acc[i][0], inv), codes4(acc[i][2], inv)};
                swap_quarters(q[0], q[1]);
                if (row >= u.rows) continue;
                typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
                uint8_t* y = (uint8_t*)a.y + (int64_t)m * a.N + n_wave + 8 * g;
                if (n_wave + 8 * g < a.N) *(u32x2*)y = u32x2{q[0], q[1]};          // N comes in multiples of 16
                if (wn == 0 && g == 0) a.ys[(int64_t)m * fp8_blocks(a.N) + u.nt] = fp8_scale_value(code);
            }
        }
        // Of a whole tile every lane's stores have gone out: at least as many as are counted.
        if (u.rows == T::BM && (u.nt + 1) * T::kCols <= a.N) stores[0] = 1;
        u = unit_at(at += step);
        if (u.rows <= 0) break;
    }
    wait_loads<0>();                         // nothing lands in LDS after the workgroup
}

template <typename Out, bool SWIGLU, int MT, int NF, int WM, int WN, int STAGES, bool PARTS = false>
coli_status lines(const Fp8GemmArgs& a, hipStream_t stream) {
    typedef LineTile<Out, SWIGLU, MT, NF, WM, WN, STAGES, true> T;
    const int NT = (a.N + T::kCols - 1) / T::kCols;
    uint32_t grid;
    if (coli_status st = grid_of(a, T::BM, NT * (PARTS ? a.parts : 1), 1, "fp8 product", &grid)) return st;
    grid = std::min(grid, kCus);             // LDS holds one workgroup a CU
    const bool fast = a.K % (4 * kFp8Block) == 0 && (uintptr_t)a.as % 16 == 0 && a.s_off % 16 == 0 && (!SWIGLU || a.up_s % 16 == 0);
    if (fast) launch(fp8_line_kernel<Out, SWIGLU, MT, NF, WM, WN, STAGES, true, PARTS>, dim3(grid), dim3(T::kThreads), 0, stream, a, NT);
    else launch(fp8_line_kernel<Out, SWIGLU, MT, NF, WM, WN, STAGES, false, PARTS>, dim3(grid), dim3(T::kThreads), 0, stream, a, NT);
    COLI_CHECK_LAUNCH("fp8 product kernel launch");
    return COLI_OK;
}

template <typename Out, bool SWIGLU, int NF, int WN, int KS, int CB>
coli_status few_rows(const Fp8GemmArgs& a, hipStream_t stream) {
    constexpr int kCols = (SWIGLU ? NF / 2 : NF) * WN * kFrag;
    const int NT = (a.N + kCols - 1) / kCols;
    uint32_t grid;
    if (coli_status st = grid_of(a, kFrag, NT, 64 * WN * KS, "fp8 product", &grid)) return st;
    if (a.K % (CB * kFp8Block) == 0)
        launch(fp8_few_rows_kernel<Out, SWIGLU, NF, WN, KS, CB, false>, dim3(grid), dim3(64 * WN * KS), 0, stream, a, NT);
    else
        launch(fp8_few_rows_kernel<Out, SWIGLU, NF, WN, KS, CB, true>, dim3(grid), dim3(64 * WN * KS), 0, stream, a, NT);
    COLI_CHECK_LAUNCH("fp8 product kernel launch");
    return COLI_OK;
}

// SwiGLU of few rows into FP8. A block of 128 h is one workgroup's, whose CU takes in about 35 GB/s, so that fewer
// workgroups than CUs leave the device idle: then, with a workspace for h in f32, it is formed 16 columns a
// workgroup and quantised by a launch of its own (K 6144, inter 2048: 8 rows of 8 of 256 experts 41 us against 58,
// one row 11 against 51; from 256 workgroups on, 40 rows of 40 experts, 188 against the one launch's 186).
int64_t few_rows_blocks(const Fp8GemmArgs& a) {
    const int64_t experts = a.offsets ? std::min(a.E, a.rows) : 1;
    return experts * ((a.rows + experts * kFrag - 1) / (experts * kFrag)) * fp8_blocks(a.N);
}

coli_status few_rows_fp8(const Fp8GemmArgs& a, hipStream_t stream) {
    if (a.ws == nullptr) return few_rows<Fp8Out, true, 2, 8, 1, 4>(a, stream);
    Fp8GemmArgs h = a;
    h.y = a.ws;
    h.ld = a.N;
    if (coli_status st = few_rows<RawOut, true, 2, 1, 4, 4>(h, stream)) return st;
    return launch_quantize_fp8(a.ws, COLI_F32, a.rows, a.N, a.N, (uint8_t*)a.y, a.ys, stream, a.offsets, a.E);
}

// y = the sum of the parts, in their order; a thread has 4 neighbouring columns of a row. Rows outside the offsets
// stay.
template <typename T>
__global__ __launch_bounds__(256) void part_sum_kernel(const float* __restrict__ part, Fp8GemmArgs a, uint32_t per_row) {
    const uint32_t i = blockIdx.x * 256 + threadIdx.x, m = i / per_row;
    const int n0 = (int)(i - m * per_row) * 4;
    if (m >= (uint32_t)a.rows || (a.offsets && ((int)m < a.offsets[0] || (int)m >= a.offsets[a.E]))) return;
    const int64_t all = (int64_t)a.rows * a.N;
    const float* p = part + (int64_t)m * a.N + n0;
    T* y = (T*)a.y + (int64_t)m * a.ld + n0;
    if (n0 + 4 <= a.N) {
        float v[4], x[4];
        load_f32<float, 4>(p, v);
#pragma unroll 4
        for (int s = 1; s < a.parts; ++s) {
            load_f32<float, 4>(p + s * all, x);
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] += x[j];
        }
        store_f32<T, 4>(y, v);
    } else {
        for (int j = 0; n0 + j < a.N; ++j) {
            float v = p[j];
            for (int s = 1; s < a.parts; ++s) v += p[s * all + j];
            y[j] = (T)v;
        }
    }
}

// The same for gate's sums and up's (N each a row) and SwiGLU; 32 lanes have a block of 128 h.
template <typename Out>
__global__ __launch_bounds__(256) void part_swiglu_kernel(const float* __restrict__ part, Fp8GemmArgs a, uint32_t per_row) {
    constexpr bool kFp8 = std::is_same<Out, Fp8Out>::value;
    const uint32_t i = blockIdx.x * 256 + threadIdx.x, m = i / per_row;
    const int n0 = (int)(i - m * per_row) * 4;
    if (m >= (uint32_t)a.rows || (a.offsets && ((int)m < a.offsets[0] || (int)m >= a.offsets[a.E]))) return;   // 32 lanes alike
    const int64_t ld = 2 * (int64_t)a.N, all = a.rows * ld;
    const float* p = part + m * ld + n0;
    f32x4 h = {0.f, 0.f, 0.f, 0.f};
    if (n0 + 4 <= a.N) {
        float g[4], u[4], x[4];
        load_f32<float, 4>(p, g);
        load_f32<float, 4>(p + a.N, u);
#pragma unroll 4
        for (int s = 1; s < a.parts; ++s) {
            load_f32<float, 4>(p + s * all, x);
#pragma unroll
            for (int j = 0; j < 4; ++j) g[j] += x[j];
            load_f32<float, 4>(p + s * all + a.N, x);
#pragma unroll
            for (int j = 0; j < 4; ++j) u[j] += x[j];
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) h[j] = silu_mul(g[j], u[j]);
    } else {
#pragma unroll
        for (int j = 0; j < 3; ++j) {
            if (n0 + j >= a.N) break;
            float g = p[j], u = p[a.N + j];
            for (int s = 1; s < a.parts; ++s) g += p[s * all + j], u += p[s * all + a.N + j];
            h[j] = silu_mul(g, u);
        }
    }
    if constexpr (kFp8) {
        const int code = fp8_scale_code(lanes_umax<32>(top4(h)));
        if (n0 < a.N) *(uint32_t*)((uint8_t*)a.y + (int64_t)m * a.N + n0) = codes4(h, fp8_scale_inverse(code));
        if (threadIdx.x % 32 == 0) a.ys[(int64_t)m * fp8_blocks(a.N) + n0 / kFp8Block] = fp8_scale_value(code);
    } else {
        if (n0 < a.N) store4<Out>(a, (int)m, n0, a.N, h);
    }
}

bool exact_products(const Fp8GemmArgs& a, bool f32, bool fp8) { return f32 || (fp8 && a.rows * (int64_t)a.N < kFewValues); }

// The product in a.parts parts of its columns, f32 sums in the workspace, and their sum.
template <typename Out, bool SWIGLU>
coli_status product_parts(const Fp8GemmArgs& a, hipStream_t stream) {
    Fp8GemmArgs p = a;
    p.y = a.ws;
    p.ld = (SWIGLU ? 2 : 1) * (int64_t)a.N;
    const bool exact = exact_products(a, std::is_same<Out, float>::value, std::is_same<Out, Fp8Out>::value);
    if (coli_status st = exact ? lines<float, SWIGLU, 4, 4, 2, 4, 3, true>(p, stream) : lines<RawOut, SWIGLU, 4, 4, 2, 4, 3, true>(p, stream))
        return st;
    const uint32_t per_row = SWIGLU ? (uint32_t)fp8_blocks(a.N) * 32 : ((uint32_t)a.N + 3) / 4;
    const dim3 grid((uint32_t)(((int64_t)a.rows * per_row + 255) / 256));
    if constexpr (SWIGLU) launch(part_swiglu_kernel<Out>, grid, dim3(256), 0, stream, (const float*)a.ws, a, per_row);
    else launch(part_sum_kernel<Out>, grid, dim3(256), 0, stream, (const float*)a.ws, a, per_row);
    COLI_CHECK_LAUNCH("fp8 product kernel launch");
    return COLI_OK;
}

template <typename Out, bool SWIGLU>
coli_status product(const Fp8GemmArgs& a, hipStream_t stream) {
    constexpr bool kFp8 = std::is_same<Out, Fp8Out>::value, kWide = std::is_same<Out, float>::value;
    if (a.parts > 1) return product_parts<Out, SWIGLU>(a, stream);
    const bool exact = exact_products(a, kWide, kFp8);
    switch (choose_fp8_kernel(a, SWIGLU, exact)) {
        case kFp8FewRows16:                  // (not of SwiGLU's)
            if constexpr (!SWIGLU) return few_rows<Out, SWIGLU, 1, 1, 4, 4>(a, stream);
        case kFp8FewRows32:
            if constexpr (kFp8) return few_rows_fp8(a, stream);
            else return few_rows<Out, SWIGLU, 2, 1, 4, 4>(a, stream);
        case kFp8Lines256:
            // (32-bit results have no registers for it, as their operands are twice as wide, and are not sent here)
            if constexpr (!kWide) return lines<Out, SWIGLU, 8, 4, 2, 4, 2>(a, stream);
        default:
            if constexpr (kFp8) {
                if (exact) return lines<ExactFp8Out, SWIGLU, 4, 4, 2, 4, 3>(a, stream);
            }
            return lines<Out, SWIGLU, 4, 4, 2, 4, 3>(a, stream);
    }
}

}  // namespace

// Which kernel, by estimates of each one's time in us, from times on one MI355X (graphs, warm caches):
//  - few_rows reads a matrix once per 16 rows, 5.5 TB/s the first time and 6 from the caches, and a workgroup takes
//    in its rows no faster than about 35 GB/s: 1.3 us per 1024 columns; 1024 workgroups take 3 at least. One matrix
//    of 8192 x 8192, 17 / 64 / 128 / 256 rows 25.7 / 47 / 90 / 176; 2048 x 6144 (N, K), 64 / 256 rows 11.4 / 35; 64
//    of 2048 x 2048, 1024 rows 71; SwiGLU of 256 of 2048 x 6144, 512 / 2048 rows 928 / 1166.
//  - lines takes 2 for a unit's ends and a time a block of columns: tiles of 128 rows 0.78 while they leave half of
//    the CUs idle, 1.03 where they do not, of 256 rows 1.8, for 32-bit results 1.5 to 1.85; and 5.4 TB/s. 8192 x
//    8192: 17 to 512 rows 56 (f32 103 to 108), 1024 rows 72 against 103 for tiles of 256, 2048 rows 135 against
//    121, 8192 rows 534 against 453; 2048 x 6144, 17 to 256 rows 43; 64 of 2048 x 2048, 1024 rows 49; the SwiGLU of
//    256 988 / 1102.
// few_rows with 16 matrix rows a workgroup in place of 32 where that leaves no more workgroups than CUs.
struct Fp8Estimate {
    Fp8Kernel kernel;
    int parts;                               // with a workspace, if more than 1
};

Fp8Estimate estimate_fp8(const Fp8GemmArgs& a, bool swiglu, bool wide) {
    const int64_t experts = a.offsets ? std::min(a.E, a.rows) : 1;
    const double per = (double)a.rows / experts, KB = (double)fp8_blocks(a.K);
    const double bytes = (double)experts * a.N * a.K * (swiglu ? 2 : 1);
    // (of several experts, the last tile of each is half full on average)
    auto tiles = [&](int rows) { return experts > 1 ? std::max(1.0, per / rows + 0.5) : std::ceil(per / rows); };
    auto units = [&](int rows) { return experts * tiles(rows) * std::ceil(a.N / (swiglu ? 128.0 : 256.0)); };
    auto line_us = [&](int rows, double block, double idle) {
        const double u = units(rows);
        return 4 + std::max((2 + KB * (u <= kCus / 2 ? idle : block)) * std::ceil(u / kCus), bytes / 5.4e6);
    };
    const double again = experts > 1 ? std::max(0.0, per / kFrag - 0.4) : tiles(kFrag) - 1;
    const double groups = experts * (1 + again) * std::ceil(a.N / (swiglu ? 16.0 : 32.0));
    const double few = 3 + std::max({1.3 * a.K / 1024, bytes / 5.5e6 + again * bytes / 6e6, 3 * groups / 1024});
    const double l128 = wide ? line_us(128, 1.85, 1.5) : line_us(128, 1.03, 0.78);
    const double l256 = wide ? l128 : line_us(256, 1.8, 1.7);
    // (as many workgroups as few_rows may need must fit a launch)
    const int64_t stretches = a.offsets ? (int64_t)a.rows / kFrag + std::min(a.E, a.rows) : ((int64_t)a.rows + kFrag - 1) / kFrag;
    const bool fits = stretches * ((a.N + 15) / 16) < int64_t(1) << 23;
    Fp8Estimate best = {l256 < l128 ? kFp8Lines256 : kFp8Lines128, 1};
    double least = std::min(l128, l256);
    if (fits && few < least) {
        const bool half = !swiglu && experts * tiles(kFrag) * std::ceil(a.N / 16.0) <= kCus;
        best.kernel = half ? kFp8FewRows16 : kFp8FewRows32;
        least = few;
    }
    // Tiles of 128 rows that leave CUs idle, in parts of the columns: as many blocks less, a second launch (5) and
    // the sums' way through the caches. One matrix of 8192 x 8192 into 16 bits: 64 rows 24 in place of 46, 128 28 /
    // 55, 256 33 / 54; into f32 64 rows 31 / 48, 256 49 / 105, 512 77 / 105; 512 rows of 2048 x 6144 25 / 43.
    // SwiGLU of two of 2048 x 6144, 128 / 256 / 512 rows 22 / 24 / 30 in place of 35 / 46 / 46.
    least -= 5;                              // (what the second launch and the workspace cost the host)
    const double u = units(128), block = wide ? 1.85 : 1.03, sums = (swiglu ? 2.0 : 1.0) * a.rows * a.N;
    for (int s = 2; s <= 16 && s * u <= kCus && 4 * s <= KB; ++s) {
        const double us = 4 + std::max(2 + (std::ceil(KB / 4 / s) * 4) * block, bytes / 5.4e6) + 5 + s * sums * 8 / 8e6;
        if (us < least) best.parts = s, least = us;
    }
    return best;
}

Fp8Kernel choose_fp8_kernel(const Fp8GemmArgs& a, bool swiglu, bool wide) { return estimate_fp8(a, swiglu, wide).kernel; }

size_t plan_fp8_ws(Fp8GemmArgs& a, bool swiglu, int32_t dtype) {
    if (a.rows == 0) return 0;
    const Fp8Estimate e = estimate_fp8(a, swiglu, exact_products(a, dtype == COLI_F32, dtype == COLI_FP8));
    a.parts = e.parts;
    if (e.parts > 1) return (size_t)e.parts * a.rows * a.N * (swiglu ? 8 : 4);
    // SwiGLU of few rows into FP8 in two launches. (One row, inter 2048, K 512 / 1024 / 1536 / 4096: 6.9 / 11.0 /
    // 15.0 / 34.4 us in one launch, 4.7 / 5.1 / 5.8 / 8.1 in two, which cost the host 4.5 more.)
    const bool two = swiglu && dtype == COLI_FP8 && e.kernel == kFp8FewRows32 && fp8_blocks(a.K) > 8 && few_rows_blocks(a) < kCus;
    return two ? (size_t)a.rows * a.N * 4 : 0;
}

coli_status launch_fp8_gemm(const Fp8GemmArgs& a, bool swiglu, int32_t dtype, hipStream_t stream) {
    if (swiglu && dtype == COLI_FP8) return product<Fp8Out, true>(a, stream);
    return with_elem(dtype, [&](auto e) -> coli_status {
        using T = decltype(e);
        return swiglu ? product<T, true>(a, stream) : product<T, false>(a, stream);
    });
}

}  // namespace coli
