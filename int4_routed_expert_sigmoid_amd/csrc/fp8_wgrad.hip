// Every expert's matrix gradient from FP8 rows and output gradients: dw_e[n][k] = sum over the expert's
// rows r of g[r][n] x[r][k], both quantised over 128 of its rows (a block of the sum) by one column and
// laid out by columns, so that the sum runs along the rows of both operands.
//
// The scales are powers of two and go into the matrix instruction (one E8M0 byte for each row of an
// operand and block), or into the conversion to bf16 for 32-bit results (fp8.h), so that sums stay in
// the instruction's registers from block to block.
#include <algorithm>

#include "fp8.h"

namespace coli {
namespace {

// The first block of expert e and how many it has, by a wave.
__device__ __forceinline__ void expert_blocks(const Fp8WgradArgs& a, int e, int* first, int* count) {
    if (a.offsets == nullptr) {
        *first = 0;
        *count = (int)fp8_blocks(a.rows);
        return;
    }
    const int lane = threadIdx.x & 63;
    int before = 0;
    for (int i = lane; i < e; i += 64) {
        const int lo = min(max(a.offsets[i], 0), a.rows), hi = min(max(a.offsets[i + 1], lo), a.rows);
        before += (int)fp8_blocks(hi - lo);
    }
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) before += __shfl_xor(before, o);
    const int lo = min(max(a.offsets[e], 0), a.rows), hi = min(max(a.offsets[e + 1], lo), a.rows);
    *first = __builtin_amdgcn_readfirstlane(before);
    *count = __builtin_amdgcn_readfirstlane((int)fp8_blocks(hi - lo));
    // offsets that are not ascending may count more blocks than there are
    const int all = (int)(a.ld_t / kFp8Block);
    *first = min(*first, all);
    *count = min(*count, all - *first);
}

// A workgroup of 4 waves: 128 x 128 of one expert's gradient, a wave 64 x 64 of it.
template <typename T>
__global__ __launch_bounds__(256) void wgrad_kernel(Fp8WgradArgs a, int tiles_n, int tiles_k) {
    constexpr int NF = 4;
    const uint32_t per = (uint32_t)tiles_n * tiles_k, e = blockIdx.x / per, at = blockIdx.x % per;
    const int n_tile = at / tiles_k * 128, k_tile = at % tiles_k * 128;
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4, wave = threadIdx.x >> 6;
    const int n_wave = n_tile + (wave >> 1) * 64, k_wave = k_tile + (wave & 1) * 64;
    int first, count;
    expert_blocks(a, e, &first, &count);
    f32x4 acc[NF][NF];
#pragma unroll
    for (int i = 0; i < NF; ++i)
#pragma unroll
        for (int j = 0; j < NF; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    // x is the first operand: a lane's four results are four neighbouring k
    const uint8_t *xp[NF], *gp[NF], *xsp[NF], *gsp[NF];
#pragma unroll
    for (int i = 0; i < NF; ++i) {
        const int k = min(k_wave + i * kFrag + r, a.K - 1), n = min(n_wave + i * kFrag + r, a.N - 1);
        xp[i] = a.x + k * a.ld_t + (int64_t)first * kFp8Block + g * 16;
        gp[i] = a.g + n * a.ld_t + (int64_t)first * kFp8Block + g * 16;
        xsp[i] = a.xs + (int64_t)first * a.K + k;
        gsp[i] = a.gs + (int64_t)first * a.N + n;
    }
    for (int b = 0; b < count; ++b) {
        Frag xv[NF], gv[NF];
        int xs[NF], gs[NF];
#pragma unroll
        for (int i = 0; i < NF; ++i) {
            xv[i] = Frag{load16(xp[i]), load16(xp[i] + 64)};
            gv[i] = Frag{load16(gp[i]), load16(gp[i] + 64)};
            xs[i] = load1(xsp[i]), gs[i] = load1(gsp[i]);
            xp[i] += kFp8Block, gp[i] += kFp8Block, xsp[i] += a.K, gsp[i] += a.N;
        }
        if constexpr (std::is_same<T, float>::value) {
            Wide xw[NF];
#pragma unroll
            for (int j = 0; j < NF; ++j) xw[j] = widen(xv[j], fp8_scale_value(xs[j]));
#pragma unroll
            for (int i = 0; i < NF; ++i) {
                const Wide gw = widen(gv[i], fp8_scale_value(gs[i]));
#pragma unroll
                for (int j = 0; j < NF; ++j) acc[i][j] = wide_mfma(xw[j], gw, acc[i][j]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < NF; ++i)
#pragma unroll
                for (int j = 0; j < NF; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(words8(xv[j]), words8(gv[i]), acc[i][j], 0, 0,
                                                                                 0, xs[j], 0, gs[i]);
        }
    }
#pragma unroll
    for (int i = 0; i < NF; ++i) {
        const int n = n_wave + i * kFrag + r;
        if (n >= a.N) continue;
        T* row = (T*)a.dw + ((int64_t)e * a.N + n) * a.ld;
#pragma unroll
        for (int j = 0; j < NF; ++j) {
            const int k = k_wave + j * kFrag + 4 * g;
            if (k >= a.K) continue;              // K comes in multiples of 16
            float v[4] = {acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]};
            if (a.accumulate) {
                float o[4];
                load_f32<T, 4>(row + k, o);
#pragma unroll
                for (int x = 0; x < 4; ++x) v[x] += o[x];
            }
            store_f32<T, 4>(row + k, v);
        }
    }
}

}  // namespace

coli_status launch_fp8_wgrad(const Fp8WgradArgs& a, int32_t dtype, hipStream_t stream) {
    const int64_t tn = (a.N + 127) / 128, tk = (a.K + 127) / 128;
    if (tn * tk * a.E > (int64_t(1) << 32) / 256 - 1) return fail(COLI_EUNSUPPORTED, "fp8_wgrad: more than 2^32 threads");
    return with_elem(dtype, [&](auto e) -> coli_status {
        using T = decltype(e);
        launch(wgrad_kernel<T>, dim3((uint32_t)(tn * tk * a.E)), dim3(256), 0, stream, a, (int)tn, (int)tk);
        COLI_CHECK_LAUNCH("fp8_wgrad kernel launch");
        return COLI_OK;
    });
}

}  // namespace coli
