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
    if constexpr (std::is_same<Out, Fp8Out>::value) return few_rows<Out, SWIGLU, 4, 4, 2, 4>(a, stream);
    else return few_rows<Out, SWIGLU, 2, 1, 4, 4>(a, stream);
}

}  // namespace

Fp8Kernel choose_fp8_kernel(const Fp8GemmArgs& a, bool swiglu) { return kFp8FewRows4; }

coli_status launch_fp8_gemm(const Fp8GemmArgs& a, bool swiglu, int32_t dtype, hipStream_t stream) {
    if (swiglu && dtype == COLI_FP8) return product<Fp8Out, true>(a, stream);
    return with_elem(dtype, [&](auto e) -> coli_status {
        using T = decltype(e);
        return swiglu ? product<T, true>(a, stream) : product<T, false>(a, stream);
    });
}

}  // namespace coli
