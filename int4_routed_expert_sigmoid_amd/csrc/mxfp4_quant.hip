// MXFP4 rows: E2M1 codes with one E8M0 scale per 32 columns, and back.
//
// Quantising, a lane takes 16 bytes (4 or 8 neighbouring columns), so that a wave
// reads 1 KiB in one piece, and a block is 8 or 4 lanes: its largest |x| is the
// largest in the lane and over the lanes by DPP exchanges. The conversion itself
// is the hardware's scaled E2M1 convert (half to even, saturating).
//
// Both directions are bound by HBM: 4 (f32) or 2 bytes a value on one side,
// 17/32 byte on the other; the wide side goes past the caches. 98304 x 2048 f32 to
// MXFP4 157 us, 5.8 TB/s (200 us with cached loads of 8 columns a lane); with the
// way back to bf16 229 us, 6.2 TB/s (243 with cached stores).
#include "mxfp4.h"

namespace coli {
namespace {

constexpr int kThreads = 256;
constexpr int kUnit = 8;                          // columns per lane, dequantising

// Position of unit `u`: its row and the unit's number within it. Rows that
// follow each other without a gap are one long row (a block never crosses a
// row end: columns come in 32s), which needs no division.
struct UnitMap {
    int64_t units;       // units in all
    int64_t per_row;     // units of a row (all of them for gapless rows)
    int64_t ld;          // elements from row to row
    int32_t gu_base;     // codes' row placement, as launch_quantize_mxfp4
};

__device__ __forceinline__ void locate(const UnitMap& m, int64_t u, int64_t* row, int64_t* at) {
    if (m.per_row == m.units) {
        *row = 0;
        *at = u;
    } else if (m.units <= 0xffffffffll) {
        const uint32_t r = (uint32_t)u / (uint32_t)m.per_row;
        *row = r;
        *at = (uint32_t)u - r * (uint32_t)m.per_row;
    } else {
        *row = u / m.per_row;
        *at = u - *row * m.per_row;
    }
}

// A unit a thread (two to eight, loaded before the first is converted, were 1 to 3%
// slower).
template <typename T>
__global__ __launch_bounds__(kThreads) void quantize_kernel(const T* __restrict__ x, UnitMap m,
                                                            uint8_t* __restrict__ q,
                                                            uint8_t* __restrict__ s) {
    constexpr int N = 16 / sizeof(T), kLanes = kMxBlock / N;      // columns a lane, lanes a block
    const int64_t u = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (u >= m.units) return;                     // whole blocks: their lanes come together
    int64_t row, at;
    locate(m, u, &row, &at);
    float v[N];
    load_f32_once<T, N>(x + row * m.ld + at * N, v);
    uint32_t top = 0;
#pragma unroll
    for (int c = 0; c < N; ++c) top = max(top, abs_bits(v[c]));
    top = mx_quad_max(top);
    if constexpr (kLanes == 8)                    // the other quad of the eight
        top = max(top, (uint32_t)__builtin_amdgcn_mov_dpp((int)top, 0x141, 0xf, 0xf, true));
    const int code = mx_scale_code(top);
    const float scale = mx_scale_value(code);
    const int64_t out = (m.gu_base < 0 ? row : gu_row(row) + m.gu_base) * m.per_row + at;
    if constexpr (N == 8) {
        reinterpret_cast<uint32_t*>(q)[out] = code == 255 ? 0u : mx_codes8(v, scale);
    } else {
        uint32_t w = 0;
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[0], v[1], scale, 0);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[2], v[3], scale, 1);
        reinterpret_cast<uint16_t*>(q)[out] = code == 255 ? 0 : (uint16_t)w;
    }
    if (threadIdx.x % kLanes == 0) s[out / kLanes] = (uint8_t)code;
}

// U units per thread, kThreads apart.
template <typename T, int U>
__global__ __launch_bounds__(kThreads) void dequantize_kernel(const uint8_t* __restrict__ q,
                                                              const uint8_t* __restrict__ s,
                                                              UnitMap m, T* __restrict__ x) {
    const int64_t u0 = (int64_t)blockIdx.x * (kThreads * U) + threadIdx.x;
    uint32_t w[U];
    int code[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
        const int64_t u = min(u0 + i * kThreads, m.units - 1);
        w[i] = reinterpret_cast<const uint32_t*>(q)[u];
        code[i] = s[u >> 2];
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
        const int64_t u = u0 + i * kThreads;
        if (u >= m.units) return;
        const float sc = mx_scale_value(code[i]);
        typedef float f32x2 __attribute__((ext_vector_type(2)));
        const f32x2 p0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[i], sc, 0);
        const f32x2 p1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[i], sc, 1);
        const f32x2 p2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[i], sc, 2);
        const f32x2 p3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[i], sc, 3);
        float v[kUnit] = {p0.x, p0.y, p1.x, p1.y, p2.x, p2.y, p3.x, p3.y};
        if (code[i] == 255) {
#pragma unroll
            for (int c = 0; c < kUnit; ++c) v[c] = __uint_as_float(0x7fc00000u);
        }
        int64_t row, at;
        locate(m, u, &row, &at);
        store_f32_once<T, kUnit>(x + row * m.ld + at * kUnit, v);
    }
}

UnitMap unit_map(int64_t rows, int64_t cols, int64_t ld, int32_t gu_base, int unit) {
    UnitMap m;
    m.units = rows * (cols / unit);
    m.per_row = (ld == cols && gu_base < 0) ? m.units : cols / unit;
    m.ld = ld;
    m.gu_base = gu_base;
    return m;
}

// A launch holds fewer than 2^32 threads.
constexpr int64_t kMaxGrid = (int64_t(1) << 32) / kThreads - 1;

}  // namespace

coli_status launch_quantize_mxfp4(const void* x, int32_t dtype, int64_t rows, int64_t cols,
                                  int64_t ld, uint8_t* q, uint8_t* s, int32_t gu_base,
                                  hipStream_t stream) {
    if (rows == 0) return COLI_OK;
    return with_elem(dtype, [&](auto e) -> coli_status {
        using T = decltype(e);
        const UnitMap m = unit_map(rows, cols, ld, gu_base, 16 / (int)sizeof(T));
        const int64_t grid = (m.units + kThreads - 1) / kThreads;
        if (grid > kMaxGrid) return fail(COLI_EUNSUPPORTED, "quantize_mxfp4: too many values for one launch");
        launch(quantize_kernel<T>, dim3((uint32_t)grid), dim3(kThreads), 0, stream, (const T*)x, m, q, s);
        COLI_CHECK_LAUNCH("quantize_mxfp4 kernel launch");
        return COLI_OK;
    });
}

coli_status launch_dequantize_mxfp4(const uint8_t* q, const uint8_t* s, int64_t rows, int64_t cols,
                                    void* x, int32_t dtype, int64_t ld, hipStream_t stream) {
    if (rows == 0) return COLI_OK;
    const UnitMap m = unit_map(rows, cols, ld, -1, kUnit);
    return with_elem(dtype, [&](auto e) -> coli_status {
        using T = decltype(e);
        constexpr int U = 2;                      // 1: 4% slower, 4: 1%, 8: 5%
        const int64_t grid = (m.units + kThreads * U - 1) / (kThreads * U);
        if (grid > kMaxGrid) return fail(COLI_EUNSUPPORTED, "dequantize_mxfp4: too many values for one launch");
        launch(dequantize_kernel<T, U>, dim3((uint32_t)grid), dim3(kThreads), 0, stream, q, s, m, (T*)x);
        COLI_CHECK_LAUNCH("dequantize_mxfp4 kernel launch");
        return COLI_OK;
    });
}

}  // namespace coli
