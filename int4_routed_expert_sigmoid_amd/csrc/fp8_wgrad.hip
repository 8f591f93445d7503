// Every expert's matrix gradient from FP8 rows and output gradients: dw_e[n][k] = sum over the expert's rows r of
// g[r][n] x[r][k], both quantised over 128 of its rows (a block of the sum) by one column and laid out by columns,
// so that the sum runs along the rows of both operands.
//
// The scales are powers of two and go into the matrix instruction (one E8M0 byte for each row of an operand and
// block), or into the conversion to bf16 for 32-bit results (fp8.h), so that sums stay in the instruction's
// registers from block to block.
//
// What bounds it: the gradients that it writes where experts have few rows (64 experts of 2048 x 6144, 256 rows
// each, one MI355X, repeated by itself: 3.2 GB of f32 in 710 to 820 us, 3.9 to 4.5 TB/s, added to what is there 1206
// to 1244, 5.2 TB/s; bf16 384 to 417 and 773 to 782; in a pass behind the rows' gradient the f32 one takes 940),
// the bf16 matrix instructions where there are many and results have 32 bits (6144 x 8192 from 4095 rows, 0.41
// TFLOP: 337 us, 1.22 PFLOP/s, where a large bf16 product reaches 1.34; bf16 162, 2.5 PFLOP/s).
#include <algorithm>

#include "fp8.h"

namespace coli {
namespace {

// Persistent workgroups of WM x WN waves, each MT fragments of g's columns (n) by NF fragments of x's (k), as
// fp8_gemm.hip's lines: codes and scales straight into LDS, a block of 128 rows at a time, STAGES blocks ahead and
// on into the workgroup's next unit (a tile of one expert's gradient, whose sum has as many blocks as the expert
// has rows for, none where it has no rows). x is the first operand: a lane's four results are four neighbouring k.
// Results of 32 bits have tiles of 128 n in three stages (256 would leave the operands' bf16 form no registers),
// the others of 256 in two. Where they are added to what is there (ADD), which is loaded at a tile's end all at
// once (row by row: 1880 us for the 1244 above), all have 128.
template <typename T, int MT, int NF, int WM, int WN, int STAGES>
struct WgradTile {
    static constexpr int BM = WM * MT * kFrag, BN = WN * NF * kFrag, kWaves = WM * WN, kThreads = 64 * kWaves;
    static constexpr int U = kBlockUnits;
    static constexpr int kLoads = (BM + BN) * U / kThreads;   // code loads of a wave and block
    static constexpr int kARows = BM * U / kThreads;          // of them for g
    static constexpr int kStores = MT * sizeof(T);            // of a wave and whole tile (store64)
    static_assert(STAGES == 2 || STAGES == 3, "the stores that a wait may leave in flight");
    static_assert(BM * U % kThreads == 0 && BN * U % kThreads == 0, "whole loads for every wave");
    static_assert(NF == 4, "a wave's columns are one store64");
    static_assert(BM <= 256 && BN <= 256 && (MT == 4 || MT == 8), "a wave loads 256 scales; the ring of fragments");
    struct Lds {
        u32x4 code[STAGES][(BM + BN) * U];                    // g's columns, then x's
        uint32_t scale[STAGES][2][64];                        // 256 bytes of each
        uint32_t first[kMaxExperts];                          // first block of every expert
    };
};

struct WgradUnit {
    int e, n_tile, k_tile, first, count;     // e: of the outputs, expert + E * part; count -1: no unit
};

template <typename T, int MT, int NF, int WM, int WN, int STAGES, bool ADD>
__global__ __launch_bounds__(64 * WM * WN, 2) void wgrad_kernel(Fp8WgradArgs a, int NT, int KT) {
    typedef WgradTile<T, MT, NF, WM, WN, STAGES> W;
    constexpr int U = W::U;
    constexpr bool EXACT = std::is_same<T, float>::value;
    __shared__ typename W::Lds lds;
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wn = wave % WN, wm = wave / WN;

    const RowGroups groups = {a.offsets, nullptr, a.rows, a.E};
    const int blocks = min((int)scan_units<kFp8Block, W::kThreads>(groups, 1, lds.first, lds.scale[0][0]), a.blocks);
    const uint32_t per_expert = (uint32_t)NT * KT, total = per_expert * a.E * a.splits;
    // Units in order of expert, stretches of `tall` tiles of n, k, n, round all workgroups, and with them round the
    // XCDs: the device writes neighbouring tiles at a time. With KT a multiple of 4 and tall 1 an XCD reads an
    // eighth or a quarter of x's columns, with tall 8 a stretch of its own of g's. (An eighth of the units for each
    // XCD in place of it: 64 experts' 2048 x 6144 in f32 799 us in place of 780, 16 of 2048 x 6400 326 in place of
    // 298, 4 of 5008 x 1280 in bf16 251 in place of 213; tall 1 where KT is 7 184 in place of 177, tall 8 where it
    // is 32 367 in place of 349.)
    const uint32_t tall = KT % 4 == 0 ? 1 : 8;
    auto unit_at = [&](uint32_t w) {
        WgradUnit u = {0, 0, 0, 0, -1};
        if (w >= total) return u;
        u.e = w / per_expert;
        const uint32_t rest = w - u.e * per_expert;
        const uint32_t block = rest / (tall * KT), in = rest - block * tall * KT, high = min(tall, NT - block * tall);
        u.n_tile = (block * tall + in % high) * W::BM;
        u.k_tile = in / high * W::BN;
        // (offsets that are not ascending may count more blocks than there are)
        const int part = u.e / a.E, e = u.e - part * a.E;
        u.first = min(__builtin_amdgcn_readfirstlane((int)lds.first[e]), blocks);
        u.count = (e + 1 < a.E ? min(__builtin_amdgcn_readfirstlane((int)lds.first[min(e + 1, a.E - 1)]), blocks) : blocks) - u.first;
        if (a.splits > 1 && u.count > 0) {
            const int lo = (int)((int64_t)u.count * part / a.splits), hi = (int)((int64_t)u.count * (part + 1) / a.splits);
            u.first += lo;
            u.count = hi - lo;
        }
        return u;
    };
    uint32_t at = blockIdx.x;                // this workgroup's units: at, at + step, ...
    const uint32_t step = gridDim.x;
    WgradUnit u = unit_at(at);
    if (u.count < 0) return;

    // the block that is loaded next
    uint32_t load_at = at;
    const uint8_t *g_base = nullptr, *x_base = nullptr, *scale_base = nullptr;
    int lc = 0, load_count = 0;
    const uint32_t unit16 = ((lane & 7) ^ (lane >> 3)) * 16, lane_off = (wave * 8 + (lane >> 3)) * kFp8Block + unit16;
    uint32_t g_max = 0, x_max = 0;           // a lane's place in the last column of each
    bool loading = true;
    uint32_t scale_step = 0;
    auto set_unit = [&](const WgradUnit& v) {
        const int g_last = a.N - 1 - v.n_tile, x_last = a.K - 1 - v.k_tile;
        g_max = min(g_last, W::BM) * kFp8Block + unit16;
        x_max = min(x_last, W::BN) * kFp8Block + unit16;
        g_base = a.g + ((int64_t)v.first * a.N + v.n_tile) * kFp8Block;
        x_base = a.x + ((int64_t)v.first * a.K + v.k_tile) * kFp8Block;
        // wave 0: g's scales, the others: x's; four a lane
        scale_base = wave == 0 ? a.gs + (int64_t)v.first * a.N + v.n_tile + min(lane * 4, g_last - 3)
                               : a.xs + (int64_t)v.first * a.K + v.k_tile + min(lane * 4, x_last - 3);
        scale_step = wave == 0 ? a.N : a.K;
        load_count = v.count;
        lc = 0;
    };
    auto find = [&](WgradUnit v) {           // from unit v (load_at) on, the next that has blocks
        while (v.count == 0) v = unit_at(load_at += step);
        loading = v.count > 0;
        if (loading) set_unit(v);
    };
    // Load i of this wave: 8 columns into a slot, lane l column l / 8, position l % 8, kStep columns below the one
    // before. Behind the last unit the same number of loads goes out, so that the counts hold.
    auto load_codes = [&](int slot, int i) {
        const bool of_g = i < W::kARows;
        const int j = of_g ? i : i - W::kARows;
        const uint32_t off = min(lane_off + j * 8 * W::kWaves * kFp8Block, of_g ? g_max : x_max);   // (behind the last column: the last)
        const uint8_t* p = (of_g ? g_base + (int64_t)lc * a.N * kFp8Block : x_base + (int64_t)lc * a.K * kFp8Block) + off;
        load_to_lds(loading ? p : (const uint8_t*)&kZeroUnit, lds.code[slot] + ((of_g ? 0 : W::BM / 8) + j * W::kWaves + wave) * 64);
    };
    auto load_scales = [&](int slot) {
        load4_to_lds(loading ? scale_base + (int64_t)lc * scale_step : (const uint8_t*)&kZeroUnit, lds.scale[slot][min(wave, 1)]);
    };
    auto advance = [&]() {
        if (!loading || ++lc < load_count) return;
        find(unit_at(load_at += step));
    };

    find(u);
    __syncthreads();                         // the scan's scratch is a scale slot
#pragma unroll
    for (int c = 0; c < STAGES; ++c) {
        load_scales(c);
#pragma unroll
        for (int i = 0; i < W::kLoads; ++i) load_codes(c, i);
        advance();
    }

    // fragments: columns 16 apart have the same place in their unit's permutation
    const int m_lds = wm * kFrag + r, n_lds = wn * NF * kFrag + r;
    const int lo = g ^ (r & 7), hi = (g + 4) ^ (r & 7);
    int slot = 0;                            // of the block that is multiplied
    auto code = [&](int row, int below) {
        const u32x4* p = lds.code[slot] + below * U;
        return Frag{p[row * U + lo], p[row * U + hi]};
    };
    auto scale = [&](int which, int row) { return (int)((const uint8_t*)lds.scale[slot][which])[row]; };
    // The steps of a block as in fp8_gemm.hip: row by row, the last two rows, from step kMeet on, together.
    constexpr int kMeet = (MT - 2) * NF;
    auto row_of = [](int n) constexpr { return n < kMeet ? n / NF : MT - 2 + (n - kMeet) % 2; };
    auto frag_of = [](int n) constexpr { return n < kMeet ? n % NF : (n - kMeet) / 2; };
    auto ring = [](int i) constexpr { return MT == 4 || i < 2 ? i : i < 4 ? i - 2 : i == 4 ? 2 : i - 5; };   // 0 1 0 1 2 0 1 2
    constexpr int kRing = MT == 4 ? 4 : 3;
    Frag w[NF], av[kRing];
    int ws[NF], as[kRing];
    f32x4 acc[MT][NF];
    // How many tiles' stores may be in flight behind the loads of the block that is waited for next: those
    // of the last STAGES - 1 blocks' units (of units without blocks, whose stores follow each other, one).
    int stores[2] = {0, 0};
    auto read_x = [&](int f) {
        w[f] = code(n_lds, W::BM + f * kFrag);
        ws[f] = scale(1, n_lds + f * kFrag);
    };
    auto read_g = [&](int i) {
        av[ring(i)] = code(m_lds, i * WM * kFrag);
        as[ring(i)] = scale(0, m_lds + i * WM * kFrag);
    };
    wait_loads<(STAGES - 1) * W::kLoads>();
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
#pragma unroll
    for (int f = 0; f < NF; ++f) read_x(f);
    read_g(0);
    if constexpr (MT == 4) read_g(1);
    while (true) {
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int f = 0; f < NF; ++f) acc[i][f] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
        for (int c = 0; c < u.count; ++c) {
            Wide ww[EXACT ? NF : 1], gw[EXACT ? 2 : 1];
            if constexpr (EXACT) {
#pragma unroll
                for (int f = 0; f < NF; ++f) ww[f] = widen(w[f], fp8_scale_value(ws[f]));
            }
            // four steps by bf16 in turn, as the four instructions of one wait for each other
            auto wide_steps = [&](int n) {
                if (n <= kMeet) gw[0] = widen(av[ring(row_of(n))], fp8_scale_value(as[ring(row_of(n))]));
                if (n == kMeet) gw[EXACT] = widen(av[ring(MT - 1)], fp8_scale_value(as[ring(MT - 1)]));
#pragma unroll
                for (int k = 0; k < 4; ++k)
#pragma unroll
                    for (int x = n; x < n + 4; ++x) {
                        f32x4& y = acc[row_of(x)][frag_of(x)];
                        y = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ww[EXACT ? frag_of(x) : 0].v[k],
                                                                    gw[EXACT && row_of(x) == MT - 1].v[k], y, 0, 0, 0);
                    }
            };
            const int fill = slot;
#pragma unroll
            for (int n = 0; n < MT * NF; ++n) {
                const int i = row_of(n), f = frag_of(n);
                if (n < kMeet && f == 0) {               // rows of this block
                    if (MT == 4 && i == 0) read_g(2), read_g(3);
                    if (MT == 8) read_g(i + 1);
                    if (MT == 8 && i == MT - 3) read_g(MT - 1);
                }
                if (n == kMeet) {
                    // The next block and its scales (issued before its codes) have arrived, the codes of the
                    // STAGES - 2 behind it may not have, and this one is read.
                    wait_behind_stores<(STAGES - 2) * W::kLoads, W::kStores>(STAGES == 3 ? stores[0] + stores[1] : stores[0]);
                    if constexpr (STAGES == 3) stores[1] = stores[0];
                    stores[0] = 0;
                    __builtin_amdgcn_s_barrier();
                    asm volatile("" ::: "memory");
                    slot = slot == STAGES - 1 ? 0 : slot + 1;
                    load_scales(fill);
                }
                if constexpr (EXACT) {
                    if (n % 4 == 0) wide_steps(n);
                } else {
                    acc[i][f] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(words8(w[f]), words8(av[ring(i)]), acc[i][f],
                                                                                 0, 0, 0, ws[f], 0, as[ring(i)]);
                }
                asm volatile("" : "+v"(acc[i][f])::"memory");
                if (n >= kMeet) {
                    if (n == kMeet + 1) read_g(0);       // of the next block
                    if (n == kMeet + 3 && MT == 4) read_g(1);
                    if (i == MT - 1) read_x(f);
                    const int q = n - kMeet;
#pragma unroll
                    for (int x = q * W::kLoads / 8; x < (q + 1) * W::kLoads / 8; ++x) load_codes(fill, x);
                }
            }
            advance();
        }
        const int k_wave = u.k_tile + wn * NF * kFrag;
        const bool whole = k_wave + NF * kFrag <= a.K;                        // uniform
        auto row_at = [&](int i) { return (T*)a.dw + ((int64_t)u.e * a.N + u.n_tile + (i * WM + wm) * kFrag) * a.ld + k_wave; };
        if (ADD && whole) {                  // all loads before the first is waited for
            Old64<T> old[MT];
#pragma unroll
            for (int i = 0; i < MT; ++i) old[i].load(row_at(i), a.ld, a.N - u.n_tile - (i * WM + wm) * kFrag);
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                old[i].add_to(acc[i]);
                if constexpr (!EXACT) hold(acc[i]);      // (one after the other: fewer registers)
            }
        }
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            const int n0 = u.n_tile + (i * WM + wm) * kFrag, n = n0 + r;
            T* row = row_at(i);
            if (whole) {
                store64<T>(row, a.ld, a.N - n0, acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
                continue;
            }
            if (n >= a.N) continue;
#pragma unroll
            for (int f = 0; f < NF; ++f) {
                if (k_wave + f * kFrag + 4 * g >= a.K) continue;              // K comes in multiples of 16
                T* p = row + r * a.ld + f * kFrag + 4 * g;
                float v[4] = {acc[i][f][0], acc[i][f][1], acc[i][f][2], acc[i][f][3]};
                if (ADD) {
                    float o[4];
                    load_f32<T, 4>(p, o);
#pragma unroll
                    for (int x = 0; x < 4; ++x) v[x] += o[x];
                }
                store_f32<T, 4>(p, v);
            }
        }
        // Of a whole tile every lane's stores have gone out: as many as are counted.
        if (u.n_tile + W::BM <= a.N && u.k_tile + W::BN <= a.K) stores[0] = 1;
        u = unit_at(at += step);
        if (u.count < 0) break;
    }
    wait_loads<0>();                         // nothing lands in LDS after the workgroup
}

template <typename T, int MT, int NF, int WM, int WN, int STAGES, bool ADD>
coli_status wgrad(const Fp8WgradArgs& a, hipStream_t stream) {
    typedef WgradTile<T, MT, NF, WM, WN, STAGES> W;
    const int64_t NT = (a.N + W::BM - 1) / W::BM, KT = (a.K + W::BN - 1) / W::BN;
    if (NT * KT > INT32_MAX / a.E / a.splits) return fail(COLI_EUNSUPPORTED, "fp8_wgrad: more than 2^31 tiles");
    constexpr int64_t kPerCu = 163840 / sizeof(typename W::Lds);
    const uint32_t grid = (uint32_t)std::min<int64_t>(kCus * kPerCu, NT * KT * a.E * a.splits);
    launch(wgrad_kernel<T, MT, NF, WM, WN, STAGES, ADD>, dim3(grid), dim3(W::kThreads), 0, stream, a, (int)NT, (int)KT);
    COLI_CHECK_LAUNCH("fp8_wgrad kernel launch");
    return COLI_OK;
}

// dw = the sum of the parts, in their order (+ dw); 4 neighbouring columns a thread.
template <typename T>
__global__ __launch_bounds__(256) void wgrad_sum_kernel(const float* __restrict__ part, int64_t rows, int K, int splits, bool add,
                                                        T* __restrict__ dw, int64_t ld) {
    const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
    if (i >= rows * K) return;
    f32x4 v = *(const f32x4*)(part + i);
#pragma unroll 4
    for (int s = 1; s < splits; ++s) v += *(const f32x4*)(part + s * rows * K + i);
    T* p = dw + i / K * ld + i % K;
    float x[4] = {v[0], v[1], v[2], v[3]};
    if (add) {
        float o[4];
        load_f32<T, 4>(p, o);
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] += o[j];
    }
    store_f32<T, 4>(p, x);
}

// Into how many parts an expert's rows are divided: a tile takes about 1.5 us a block of rows, however few tiles
// there are, and the parts' sum a launch (5) and its bytes. (One gradient of 1024 x 256 from 65536 rows: 732 us in
// one part, 55 in 32; 2048 x 2048 from 16384 192 and 129 in 2; 256 x 1168 from 3274 44 and 19 in 8; 48 x 80 from
// 1400 21 and 12 in 5.)
int wgrad_splits(const Fp8WgradArgs& a) {
    const int64_t units = (int64_t)((a.N + 127) / 128) * ((a.K + 255) / 256) * a.E;
    const double blocks = (double)a.rows / kFp8Block / a.E, one = 1.6 * blocks;
    int best = 1;
    double least = one - 4;                      // (what the second launch costs the host)
    for (int s = 2; s <= 32 && s * units <= kCus && 2 * s <= blocks + 1; ++s) {
        const double us = one / s + 5 + (double)s * a.E * a.N * a.K * 8 / 4e6;
        if (us < least) best = s, least = us;
    }
    return best;
}

}  // namespace

size_t fp8_wgrad_ws(const Fp8WgradArgs& a) {
    const int splits = wgrad_splits(a);
    return splits > 1 ? (size_t)splits * a.E * a.N * a.K * 4 : 0;
}

coli_status launch_fp8_wgrad(const Fp8WgradArgs& args, int32_t dtype, hipStream_t stream) {
    Fp8WgradArgs a = args;
    a.splits = 1;
    if (a.ws) {                                  // (f32 sums of exact products whatever the type, as they are stored)
        a.splits = wgrad_splits(a);
        a.dw = a.ws;
        a.ld = a.K;
        if (coli_status st = wgrad<float, 4, 4, 2, 4, 3, false>(a, stream)) return st;
        return with_elem(dtype, [&](auto e) -> coli_status {
            using T = decltype(e);
            const int64_t rows = (int64_t)a.E * a.N;
            launch(wgrad_sum_kernel<T>, dim3((uint32_t)((rows * a.K / 4 + 255) / 256)), dim3(256), 0, stream, (const float*)a.ws, rows,
                   (int)a.K, (int)a.splits, args.accumulate, (T*)args.dw, args.ld);
            COLI_CHECK_LAUNCH("fp8_wgrad kernel launch");
            return COLI_OK;
        });
    }
    return with_elem(dtype, [&](auto e) -> coli_status {
        using T = decltype(e);
        constexpr int MT = std::is_same<T, float>::value ? 4 : 8;
        if (a.accumulate) return wgrad<T, 4, 4, 2, 4, 3, true>(a, stream);
        return wgrad<T, MT, 4, 2, 4, MT == 4 ? 3 : 2, false>(a, stream);
    });
}

}  // namespace coli
