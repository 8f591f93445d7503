// Grouped products of FP8 rows with FP8 matrices: y[r][n] = sum over blocks b of 128 columns of
// sa[r][b] sw[n / 128][b] <a[r], w_e(r)[n]>_b, rows sorted by expert.
//
// v_mfma_f32_16x16x128_f8f6f4 multiplies 16 rows by 16 rows over one block: a lane holds 32 of the
// block's 128 columns of row l % 16, here the 16-byte units l / 16 and l / 16 + 4 (a block's columns
// may be taken in any order, as long as both sides take the same). The block's sum, exact products
// summed in f32, starts from 0 and enters the row's f32 sum by one multiplication: scales are any f32
// numbers, so they cannot go into the instruction, which takes powers of two. The matrix rows are the
// first operand: result lane l then holds outputs n = 4 (l / 16) .. + 3 of one row m = l % 16, whose
// scale for the block is one number a lane, as the 16 matrix rows have one together.
#include <algorithm>
#include <cmath>

#include "fp8.h"

namespace coli {
namespace {

// FP8 rows as an output type of the SwiGLU epilogue.
struct Fp8Out {};

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
            as_c[s] = TAIL && c * CB + s >= KB ? 0.f : as[s];
#pragma unroll
            for (int f = 0; f < NF; ++f) ws_c[s][f] = ws[s][f];
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
            for (int f = 0; f < NF; ++f) p[f] = block_sum<std::is_same<Out, float>::value>(w[s][f], x);
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
                if (live && n0 < a.N) store4<Out>(a, m, n0, a.N, h[i]);
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
// again while the last two rows of fragments are multiplied and the next block's first ones are read.
// Scales come 16 bytes, four blocks, a row where rows of scales are on 16-byte boundaries (wide).
constexpr int kBlockUnits = kFp8Block / kFp8Unit;       // 16-byte units of a row's block

// What lanes behind the last column load (TAIL).
__device__ const u32x4 kZeroUnit = {0, 0, 0, 0};

__device__ __forceinline__ void load4_to_lds(const uint8_t* p, uint32_t* dst) {
    __builtin_amdgcn_global_load_lds((global_void*)p, (lds_void*)dst, 4, 0, 0);
}

template <typename Out, bool SWIGLU, int MT, int NF, int WM, int WN, int STAGES>
struct LineTile {
    static constexpr int BM = WM * MT * kFrag, BN = WN * NF * kFrag, kWaves = WM * WN, kThreads = 64 * kWaves;
    static constexpr int U = kBlockUnits;
    static constexpr int kCols = SWIGLU ? BN / 2 : BN;        // outputs of a tile
    static constexpr int kLoads = (BM + BN) * U / kThreads;   // code loads of a wave and block
    static constexpr int kARows = BM * U / kThreads;          // of them for the rows
    static constexpr int kScaleLoads = BM / 64 + 1;           // 64 rows each, and the matrix' blocks
    static_assert(BM * U % kThreads == 0 && BN * U % kThreads == 0, "whole loads for every wave");
    static_assert(kScaleLoads <= kWaves && BM % 64 == 0, "one scale load a wave");
    static_assert(MT % 4 == 0 && kLoads % 2 == 0, "the ring of row fragments; two shares of loads");
    static_assert(kCols % kFp8Block == 0 && NF * kFrag <= kFp8Block, "a wave's fragments share their scales");
    struct Lds {
        u32x4 code[STAGES][(BM + BN) * U];                    // rows, then matrix rows
        // The scales of a group of blocks (4, or 1): rows, then the matrix' blocks. A slot is filled again
        // STAGES groups later, for a block at least STAGES behind the last one that reads it.
        u32x4 scale[STAGES][BM + 64];
        uint32_t first[kMaxExperts];                          // first unit of every expert
        uint32_t top[std::is_same<Out, Fp8Out>::value ? WN * BM : 1];
    };
};

template <typename Out, bool SWIGLU, int MT, int NF, int WM, int WN, int STAGES, bool TAIL>
__global__ __launch_bounds__(64 * WM * WN, 2) void fp8_line_kernel(Fp8GemmArgs a, int NT, int wide) {
    typedef LineTile<Out, SWIGLU, MT, NF, WM, WN, STAGES> T;
    constexpr int U = T::U;
    constexpr bool EXACT = std::is_same<Out, float>::value;
    __shared__ typename T::Lds lds;
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wn = wave % WN, wm = wave / WN;
    const int KB = (a.K + kFp8Block - 1) / kFp8Block, KU = a.K / kFp8Unit;
    const uint32_t row_bytes = a.K;

    const uint32_t total = scan_units<T::BM, T::kThreads>(a, NT, lds.first, (uint32_t*)lds.scale[0]);
    const uint32_t per = (total + kXcds - 1) / kXcds, xcd = blockIdx.x % kXcds, step = gridDim.x / kXcds;
    auto unit_at = [&](uint32_t x) {
        const uint32_t w = xcd * per + x;
        return line_unit<T::BM>(a, NT, lds.first, w, x < per && w < total);
    };
    uint32_t at = blockIdx.x / kXcds;        // this workgroup's units: at, at + step, ... of its XCD's `per`
    LineUnit u = unit_at(at);
    if (u.rows <= 0) return;

    // the unit that is being loaded
    uint32_t load_at = at;
    const uint8_t *w_base[SWIGLU ? 2 : 1], *a_base, *scale_base;
    int m_last, n_last, scale_last;          // its last row and matrix row; of the scales that this wave loads
    int lc = 0;                              // its next block
    bool loading = true;
    const int sx = min(wave, T::kScaleLoads - 1);
    auto set_unit = [&](const LineUnit& v) {
        const int n_tile = v.nt * T::kCols;
        m_last = v.rows - 1, n_last = a.N - 1 - n_tile;
        w_base[0] = v.blob + a.q_off + (int64_t)n_tile * row_bytes;
        if constexpr (SWIGLU) w_base[1] = v.blob + a.up_q + (int64_t)n_tile * row_bytes;
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
        lc = 0;
    };
    // Load i of this wave for the block: 8 rows into a slot, lane l row l / 8, position l % 8. Behind the last
    // unit the same number of loads goes out, so that the counts hold, into slots that are not read again.
    const int unit = (lane & 7) ^ (lane >> 3);
    auto load_codes = [&](int slot, int i) {
        const bool rows = i < T::kARows;
        const int x = (rows ? i : i - T::kARows) * T::kWaves + wave;         // 8 rows of the tile
        const uint8_t* base;
        uint32_t row;
        if (rows) {
            base = a_base;
            row = min(x * 8 + (lane >> 3), m_last);
        } else if constexpr (SWIGLU) {                                      // fragments of gate and up in turn
            base = w_base[x / 2 % 2];
            row = min(x / 4 * kFrag + x % 2 * 8 + (lane >> 3), n_last);
        } else {
            base = w_base[0];
            row = min(x * 8 + (lane >> 3), n_last);
        }
        const uint8_t* p = base + (loading ? __umul24(row, row_bytes) + (uint32_t)(lc * U + unit) * 16 : 0u);
        if (TAIL && lc * U + unit >= KU) p = (const uint8_t*)&kZeroUnit;
        load_to_lds(p, lds.code[slot] + (rows ? x : T::BM / 8 + x) * 64);
    };
    int fill_scale = 0;                      // the scale slot that is filled next
    auto load_scales = [&]() {
        if (!loading || (wide && lc % 4 != 0)) return;
        if (wide) load_to_lds(scale_base + lc * 4, lds.scale[fill_scale] + sx * 64);
        else load4_to_lds(scale_base + lc * 4, (uint32_t*)lds.scale[fill_scale] + sx * 64);
        fill_scale = fill_scale == STAGES - 1 ? 0 : fill_scale + 1;
    };
    auto advance = [&]() {                   // to the block that is loaded next
        if (++lc < KB || !loading) return;
        load_at += step;
        const LineUnit v = unit_at(load_at);
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

    const int m_lds = wm * kFrag + r, n_lds = T::BM + wn * NF * kFrag + r;
    auto code = [&](int slot, int row) {
        return Frag{lds.code[slot][lds_unit<U>(row, g)], lds.code[slot][lds_unit<U>(row, g + 4)]};
    };
    const int per_row = wide ? 4 : 1;
    auto scale = [&](int from, int row, int b) {                // block b of the group's
        return ((const float*)lds.scale[from])[row * per_row + (wide ? b % 4 : 0)];
    };
    constexpr int kW = SWIGLU ? 2 : 1;
    const int ws_row = T::BM + (SWIGLU ? 0 : wn * NF * kFrag / kFp8Block);
    Frag w[NF], av[4];
    float as[4], ws[kW];
    f32x4 acc[MT][NF];
    int slot = 0, scales = 0;                // of the block that is multiplied
    auto read_scales = [&](int b) {
#pragma unroll
        for (int x = 0; x < kW; ++x) ws[x] = scale(scales, ws_row + x, b);
    };
    auto read_row = [&](int i, int b) {
        av[i % 4] = code(slot, m_lds + i * WM * kFrag);
        as[i % 4] = scale(scales, m_lds + i * WM * kFrag, b);
    };
    wait_loads<(STAGES - 1) * T::kLoads>();
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
#pragma unroll
    for (int f = 0; f < NF; ++f) w[f] = code(0, n_lds + f * kFrag);
    read_scales(0);
    read_row(0, 0);
    read_row(1, 0);
    while (true) {
        const int live = (u.rows - wm * kFrag + WM * kFrag - 1) / (WM * kFrag);   // fragments with rows
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int f = 0; f < NF; ++f) acc[i][f] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
        for (int c = 0; c < KB; ++c) {
            auto multiply = [&](int i) {
                if (MT > 4 || i < live) {
                    f32x4 p[NF];
#pragma unroll
                    for (int f = 0; f < NF; ++f) p[f] = block_sum<EXACT>(w[f], av[i % 4]);
#pragma unroll
                    for (int f = 0; f < NF; ++f) add_scaled(acc[i][f], p[f], as[i % 4] * ws[SWIGLU ? f % 2 : 0]);
                    hold(acc[i]);
                }
            };
#pragma unroll
            for (int i = 0; i < MT - 2; ++i) {
                read_row(i + 2, c);
                multiply(i);
            }
            // The next block and its scales (issued before its codes) have arrived, the codes of the
            // STAGES - 2 behind it may not have, and this one is read.
            wait_loads<(STAGES - 2) * T::kLoads>();
            __builtin_amdgcn_s_barrier();
            asm volatile("" ::: "memory");
            const int fill = slot, next = c + 1 == KB ? 0 : c + 1;
            slot = slot == STAGES - 1 ? 0 : slot + 1;
            const float ws_old[2] = {ws[0], ws[kW - 1]}, as_old[2] = {as[2], as[3]};
            if (!wide || next % 4 == 0) scales = scales == STAGES - 1 ? 0 : scales + 1;
            load_scales();
            // the last two rows, matrix fragment by matrix fragment, the one before scaled meanwhile
            const bool last = MT > 4 || MT - 2 < live;
            f32x4 p[2][2];
            auto add_last = [&](int f) {
#pragma unroll
                for (int x = 0; x < 2; ++x)
                    add_scaled(acc[MT - 2 + x][f], p[x][f % 2], as_old[x] * ws_old[SWIGLU ? f % 2 : 0]);
                asm volatile("" : "+v"(acc[MT - 2][f]), "+v"(acc[MT - 1][f])::"memory");
            };
#pragma unroll
            for (int f = 0; f < NF; ++f) {
                if (last) {
                    p[0][f % 2] = block_sum<EXACT>(w[f], av[2]);
                    p[1][f % 2] = block_sum<EXACT>(w[f], av[3]);
                    if (f > 0) add_last(f - 1);
                }
                w[f] = code(slot, n_lds + f * kFrag);
                if (f == 0) read_row(0, next);
                if (f == 1) read_row(1, next);
                if (f == 2) read_scales(next);
#pragma unroll
                for (int x = f * T::kLoads / NF; x < (f + 1) * T::kLoads / NF; ++x) load_codes(fill, x);
            }
            if (last) add_last(NF - 1);
            advance();
        }
        // outputs
        const int n_wave = u.nt * T::kCols + wn * (SWIGLU ? NF / 2 : NF) * kFrag;
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            const int row = m_lds + i * WM * kFrag, m = u.m0 + row;
            const bool there = row < u.rows;
            if constexpr (!SWIGLU) {
#pragma unroll
                for (int f = 0; f < NF; f += 2) store32<Out>(a, m, n_wave + f * kFrag, a.N, there, acc[i][f], acc[i][f + 1]);
            } else {
#pragma unroll
                for (int p = 0; p < NF / 2; ++p) {
                    f32x4 h;
#pragma unroll
                    for (int x = 0; x < 4; ++x) h[x] = silu_mul(acc[i][2 * p][x], acc[i][2 * p + 1][x]);
                    acc[i][2 * p] = h;
                    const int n0 = n_wave + p * kFrag + 4 * g;
                    if constexpr (!std::is_same<Out, Fp8Out>::value) {
                        if (there && n0 < a.N) store4<Out>(a, m, n0, a.N, h);
                    }
                }
            }
        }
        if constexpr (std::is_same<Out, Fp8Out>::value) {
            // a row's largest |h| of the tile's 128, a wave's 32 of them at a time
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                uint32_t top = 0;
#pragma unroll
                for (int p = 0; p < NF / 2; ++p)
                    if (n_wave + p * kFrag + 4 * g < a.N) top = max(top, top4(acc[i][2 * p]));
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
                if (row >= u.rows) continue;
#pragma unroll
                for (int p = 0; p < NF / 2; ++p) {
                    const int n0 = n_wave + p * kFrag + 4 * g;
                    if (n0 < a.N) *(uint32_t*)((uint8_t*)a.y + (int64_t)m * a.N + n0) = codes4(acc[i][2 * p], fp8_scale_inverse(code));
                }
                if (wn == 0 && g == 0) a.ys[(int64_t)m * fp8_blocks(a.N) + u.nt] = fp8_scale_value(code);
            }
        }
        at += step;
        u = unit_at(at);
        if (u.rows <= 0) break;
    }
    wait_loads<0>();                         // nothing lands in LDS after the workgroup
}

template <typename Out, bool SWIGLU, int MT, int NF, int WM, int WN, int STAGES>
coli_status lines(const Fp8GemmArgs& a, hipStream_t stream) {
    typedef LineTile<Out, SWIGLU, MT, NF, WM, WN, STAGES> T;
    const int NT = (a.N + T::kCols - 1) / T::kCols;
    uint32_t grid;
    if (coli_status st = grid_of(a, T::BM, NT, 1, "fp8 product", &grid)) return st;
    grid = std::min(grid, kCus);             // LDS holds one workgroup a CU
    const int wide = fp8_blocks(a.K) % 4 == 0 && (uintptr_t)a.as % 16 == 0 && a.s_off % 16 == 0 && (!SWIGLU || a.up_s % 16 == 0);
    if (a.K % kFp8Block == 0)
        launch(fp8_line_kernel<Out, SWIGLU, MT, NF, WM, WN, STAGES, false>, dim3(grid), dim3(T::kThreads), 0, stream, a, NT, wide);
    else
        launch(fp8_line_kernel<Out, SWIGLU, MT, NF, WM, WN, STAGES, true>, dim3(grid), dim3(T::kThreads), 0, stream, a, NT, wide);
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

template <typename Out, bool SWIGLU>
coli_status product(const Fp8GemmArgs& a, hipStream_t stream) {
    constexpr bool kFp8 = std::is_same<Out, Fp8Out>::value, kWide = std::is_same<Out, float>::value;
    switch (choose_fp8_kernel(a, SWIGLU)) {
        case kFp8FewRows2:
        case kFp8FewRows4:
            if constexpr (kFp8) return few_rows<Out, SWIGLU, 4, 4, 2, 4>(a, stream);
            else return few_rows<Out, SWIGLU, 2, 1, 4, 4>(a, stream);
        case kFp8Lines256:
            // (32-bit results have no registers for it: operands are twice as wide)
            if constexpr (!kWide) return lines<Out, SWIGLU, 8, 4, 2, 4, 2>(a, stream);
        default: return lines<Out, SWIGLU, 4, 4, 2, 4, 3>(a, stream);
    }
}

}  // namespace

Fp8Kernel choose_fp8_kernel(const Fp8GemmArgs& a, bool swiglu) {
    const int64_t experts = a.offsets ? std::min(a.E, a.rows) : 1;
    const double per = (double)a.rows / experts;
    const int cols = swiglu ? 128 : 256;
    auto units = [&](int bm) { return experts * (int64_t)std::ceil(per / bm) * ((a.N + cols - 1) / cols); };
    if (per <= 4 || (per <= 32 && units(128) < kCus)) return kFp8FewRows4;
    return per >= 512 ? kFp8Lines256 : kFp8Lines128;
}

coli_status launch_fp8_gemm(const Fp8GemmArgs& a, bool swiglu, int32_t dtype, hipStream_t stream) {
    if (swiglu && dtype == COLI_FP8) return product<Fp8Out, true>(a, stream);
    return with_elem(dtype, [&](auto e) -> coli_status {
        using T = decltype(e);
        return swiglu ? product<T, true>(a, stream) : product<T, false>(a, stream);
    });
}

}  // namespace coli
