// MXFP4 rows: E2M1 codes with one E8M0 scale per 32 columns, and back.
//
// A lane takes 8 neighbouring columns, so a block is 4 lanes: the largest
// |x| of the block is the largest of 8 in the lane and of 4 lanes (two DPP
// exchanges inside the quad), and the codes are one 4-byte store per lane (256
// contiguous bytes a wave). The conversion itself is the hardware's scaled
// E2M1 convert (half to even, saturating).
//
// Both directions are bound by HBM: 4 (f32) or 2 bytes a value on one side,
// 17/32 byte on the other.
#include <algorithm>

#include "mxfp4.h"

namespace coli {
namespace {

constexpr int kThreads = 256;
constexpr int kUnit = 8;                          // columns per lane

// Position of unit `u` (8 columns): its row and the unit's number within it.
// Rows that follow each other without a gap are one long row (a block never
// crosses a row end: columns come in 32s), which needs no division.
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

// U units per thread, kThreads apart, all loaded before the first is converted.
template <typename T, int U>
__global__ __launch_bounds__(kThreads) void quantize_kernel(const T* __restrict__ x, UnitMap m,
                                                            uint8_t* __restrict__ q,
                                                            uint8_t* __restrict__ s) {
    const int64_t u0 = (int64_t)blockIdx.x * (kThreads * U) + threadIdx.x;
    float v[U][kUnit];
    int64_t out[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
        const int64_t u = u0 + i * kThreads;
        out[i] = -1;
        if (u < m.units) {
            int64_t row, at;
            locate(m, u, &row, &at);
            load_f32<T, kUnit>(x + row * m.ld + at * kUnit, v[i]);
            out[i] = (m.gu_base < 0 ? row : gu_row(row) + m.gu_base) * m.per_row + at;
        }
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
        if (out[i] < 0) continue;                 // whole quads: units come in 4s
        uint32_t top = 0;
#pragma unroll
        for (int c = 0; c < kUnit; ++c) top = max(top, abs_bits(v[i][c]));
        top = mx_quad_max(top);
        const int code = mx_scale_code(top);
        const uint32_t w = code == 255 ? 0u : mx_codes8(v[i], mx_scale_value(code));
        reinterpret_cast<uint32_t*>(q)[out[i]] = w;
        if ((threadIdx.x & 3) == 0) s[out[i] >> 2] = (uint8_t)code;
    }
}

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
        store_f32<T, kUnit>(x + row * m.ld + at * kUnit, v);
    }
}

UnitMap unit_map(int64_t rows, int64_t cols, int64_t ld, int32_t gu_base) {
    UnitMap m;
    m.units = rows * (cols / kUnit);
    m.per_row = (ld == cols && gu_base < 0) ? m.units : cols / kUnit;
    m.ld = ld;
    m.gu_base = gu_base;
    return m;
}

// One unit per thread until the launch has a workgroup for every CU four
// times over, then four, so that a thread has 64-128 bytes on the way.
constexpr int64_t kManyUnits = 4 * 256 * 4 * kThreads;
// A launch holds fewer than 2^32 threads.
constexpr int64_t kMaxGrid = (int64_t(1) << 32) / kThreads - 1;

}  // namespace

coli_status launch_quantize_mxfp4(const void* x, int32_t dtype, int64_t rows, int64_t cols,
                                  int64_t ld, uint8_t* q, uint8_t* s, int32_t gu_base,
                                  hipStream_t stream) {
    if (rows == 0) return COLI_OK;
    const UnitMap m = unit_map(rows, cols, ld, gu_base);
    return with_elem(dtype, [&](auto e) -> coli_status {
        using T = decltype(e);
        const int U = m.units >= kManyUnits ? 4 : 1;
        const int64_t grid = (m.units + kThreads * U - 1) / (kThreads * U);
        if (grid > kMaxGrid) return fail(COLI_EUNSUPPORTED, "quantize_mxfp4: 2^37 values or more");
        if (U == 4)
            launch(quantize_kernel<T, 4>, dim3((uint32_t)grid), dim3(kThreads), 0, stream, (const T*)x, m, q, s);
        else
            launch(quantize_kernel<T, 1>, dim3((uint32_t)grid), dim3(kThreads), 0, stream, (const T*)x, m, q, s);
        COLI_CHECK_LAUNCH("quantize_mxfp4 kernel launch");
        return COLI_OK;
    });
}

coli_status launch_dequantize_mxfp4(const uint8_t* q, const uint8_t* s, int64_t rows, int64_t cols,
                                    void* x, int32_t dtype, int64_t ld, hipStream_t stream) {
    if (rows == 0) return COLI_OK;
    const UnitMap m = unit_map(rows, cols, ld, -1);
    return with_elem(dtype, [&](auto e) -> coli_status {
        using T = decltype(e);
        const int U = m.units >= kManyUnits ? 4 : 1;
        const int64_t grid = (m.units + kThreads * U - 1) / (kThreads * U);
        if (grid > kMaxGrid) return fail(COLI_EUNSUPPORTED, "dequantize_mxfp4: 2^37 values or more");
        if (U == 4)
            launch(dequantize_kernel<T, 4>, dim3((uint32_t)grid), dim3(kThreads), 0, stream, q, s, m, (T*)x);
        else
            launch(dequantize_kernel<T, 1>, dim3((uint32_t)grid), dim3(kThreads), 0, stream, q, s, m, (T*)x);
        COLI_CHECK_LAUNCH("dequantize_mxfp4 kernel launch");
        return COLI_OK;
    });
}

}  // namespace coli
