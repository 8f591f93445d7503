// Internal: the MXFP4 format (E2M1 codes, one E8M0 scale per 32 columns), its
// row and element types, and the launchers of mxfp4_quant.hip, mxfp4_gemm.hip
// and permute.hip.
#pragma once

#include "common.h"
#include "row_groups.h"

namespace coli {

// ------------------------------------------------------------ element types
// Rows come and go as f32, bf16 or f16 (COLI_F32, COLI_BF16, COLI_F16).
template <int DT> struct ElemOf;
template <> struct ElemOf<COLI_F32> { using type = float; };
template <> struct ElemOf<COLI_BF16> { using type = __bf16; };
template <> struct ElemOf<COLI_F16> { using type = _Float16; };

inline bool elem_dtype(int32_t dt) { return dt == COLI_F32 || dt == COLI_BF16 || dt == COLI_F16; }
inline int elem_bytes(int32_t dt) { return dt == COLI_F32 ? 4 : 2; }

// N neighbouring elements. Aligned as one element: gfx950 takes 16-byte
// accesses at any element boundary, so rows of odd lengths and strides keep
// the wide loads and stores.
template <typename T, int N>
struct __attribute__((packed, aligned(sizeof(T)))) Pack {
    T v[N];
};

template <typename T, int N>
__device__ __forceinline__ void load_f32(const T* p, float (&out)[N]) {
    const Pack<T, N> r = *reinterpret_cast<const Pack<T, N>*>(p);
#pragma unroll
    for (int i = 0; i < N; ++i) out[i] = (float)r.v[i];
}

// One rounding (half to even) to T.
template <typename T, int N>
__device__ __forceinline__ void store_f32(T* p, const float (&in)[N]) {
    Pack<T, N> r;
#pragma unroll
    for (int i = 0; i < N; ++i) r.v[i] = (T)in[i];
    *reinterpret_cast<Pack<T, N>*>(p) = r;
}

// The same past the caches, for what is read once, and for results that are more
// than the caches hold.
template <typename T, int N>
__device__ __forceinline__ void load_f32_once(const T* p, float (&out)[N]) {
    typedef T V __attribute__((ext_vector_type(N), aligned(sizeof(T))));
    const V v = __builtin_nontemporal_load(reinterpret_cast<const V*>(p));
#pragma unroll
    for (int i = 0; i < N; ++i) out[i] = (float)v[i];
}

template <typename T, int N>
__device__ __forceinline__ void store_f32_once(T* p, const float (&in)[N]) {
    typedef T V __attribute__((ext_vector_type(N), aligned(sizeof(T))));
    V v;
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = (T)in[i];
    __builtin_nontemporal_store(v, reinterpret_cast<V*>(p));
}

// ------------------------------------------------------------ MXFP4 blocks
constexpr int kMxBlock = 32;

// Scale code of a block from the bits of its largest |x|: 2^(code - 127) is
// the power of two two binades below the largest value's (the largest E2M1
// value, 6, lies in [4, 8)), so the largest element lands in [4, 8) and
// saturates at 6. A block with an infinity or a NaN has the NaN code 255.
__device__ __forceinline__ int mx_scale_code(uint32_t top_bits) {
    if (top_bits >= 0x7f800000u) return 255;
    const int e = (int)(top_bits >> 23) - 2;
    return e < 0 ? 0 : e;
}

// 2^(code - 127) as a float (code 0 is subnormal); code 255 gives infinity's
// bits, which callers treat apart.
__device__ __forceinline__ float mx_scale_value(int code) {
    return __uint_as_float(code == 0 ? 1u << 22 : (uint32_t)code << 23);
}

__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }

// The largest of the four lanes of a quad (all four active).
__device__ __forceinline__ uint32_t mx_quad_max(uint32_t v) {
    v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xf, 0xf, true));   // lanes 1 0 3 2
    v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xf, 0xf, true));   // lanes 2 3 0 1
    return v;
}

// Codes of 8 elements (element 2i in bits 0-3 of byte i), rounded half to
// even, saturated at +-6, the sign kept for zeros too. Not for code 255.
__device__ __forceinline__ uint32_t mx_codes8(const float (&x)[8], float scale) {
    uint32_t q = 0;
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, x[0], x[1], scale, 0);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, x[2], x[3], scale, 1);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, x[4], x[5], scale, 2);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, x[6], x[7], scale, 3);
    return q;
}

// ------------------------------------------------------------ launchers
// Row r of the output (codes and scales) is row r of the input, or gu_row(r) +
// gu_base where a gate or up matrix goes into an interleaved blob (gu_base 0 or
// kGuBlock; -1: plain rows).
coli_status launch_quantize_mxfp4(const void* x, int32_t dtype, int64_t rows, int64_t cols,
                                  int64_t ld, uint8_t* q, uint8_t* s, int32_t gu_base,
                                  hipStream_t stream);
coli_status launch_dequantize_mxfp4(const uint8_t* q, const uint8_t* s, int64_t rows, int64_t cols,
                                    void* x, int32_t dtype, int64_t ld, hipStream_t stream);

// Grouped product of MXFP4 rows with MXFP4 matrices; see mxfp4_gemm.hip.
struct MxGemmArgs : RowGroups {
    const uint8_t* a;            // [rows][K/2] codes
    const uint8_t* as;           // [rows][K/32] scales
    size_t q_off, s_off;         // codes and scales of the matrix in its blob
    void* y;                     // [rows][ld] output, or codes [rows][n_out / 2]
    uint8_t* ys;                 // scales [rows][n_out / 32] of an MXFP4 output
    int64_t ld;
    int32_t K;
    int32_t N;                   // rows of the matrix (SwiGLU: 2 * inter)
};
// The kernel that a product runs: its rows, E, offsets, N, K, s_off and as decide.
enum MxKernel : int32_t {
    kMxFewRows2, kMxFewRows4,                    // by waves that share the columns
    kMxTilesShort, kMxTiles64, kMxTiles128,      // fewer than 512 columns; by rows a tile
    kMxLines128, kMxLines256,                    // by rows a tile
};
MxKernel choose_mxfp4_kernel(const MxGemmArgs& a);
coli_status launch_mxfp4_gemm(const MxGemmArgs& a, bool swiglu, int32_t dtype, hipStream_t stream);

// Token permutation (permute.hip).
coli_status launch_dispatch(const void* x, int32_t dtype, int32_t T, int32_t k, int32_t H,
                            int64_t ld_x, const int32_t* inv, void* rows, int64_t ld_rows,
                            hipStream_t stream);
coli_status launch_dispatch_mxfp4(const void* x, int32_t dtype, int32_t T, int32_t k, int32_t H,
                                  int64_t ld_x, const int32_t* inv, uint8_t* q, uint8_t* s,
                                  hipStream_t stream);
coli_status launch_dispatch_bwd(const void* g, int32_t g_dtype, int64_t ld_g, int32_t T, int32_t k,
                                int32_t H, const int32_t* inv, void* dx, int32_t dtype,
                                int64_t ld_dx, hipStream_t stream);
coli_status launch_combine_rows(const void* rows, int32_t rows_dtype, int64_t ld_rows, int32_t T,
                                int32_t k, int32_t H, const int32_t* inv, const float* w,
                                const void* shared, int64_t ld_shared, float scale, void* y,
                                int32_t dtype, int64_t ld_y, hipStream_t stream);
coli_status launch_combine_bwd(const void* dy, int32_t dy_dtype, int64_t ld_dy, const void* rows,
                               int32_t rows_dtype, int64_t ld_rows, int32_t T, int32_t k, int32_t H,
                               const int32_t* inv, const float* w, float scale, void* drows,
                               int64_t ld_drows, float* dw, hipStream_t stream);

// Runs fn with the element type of a checked dtype code.
template <typename F>
inline coli_status with_elem(int32_t dtype, F&& fn) {
    switch (dtype) {
        case COLI_F32: return fn(float{});
        case COLI_BF16: return fn(__bf16{});
        default: return fn(_Float16{});
    }
}

}  // namespace coli
