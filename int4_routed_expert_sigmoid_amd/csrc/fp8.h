// Internal: the FP8 format (e4m3 codes with one f32 scale per 128 columns of a row, or per
// block of 128 rows by 128 columns of a matrix), and the launchers of fp8_quant.hip,
// fp8_gemm.hip and fp8_wgrad.hip.
#pragma once

#include "mfma_tiles.h"

namespace coli {

constexpr int kFp8Block = 128;
constexpr int kFp8Unit = 16;                     // columns come in multiples of this

__host__ __device__ inline int64_t fp8_blocks(int64_t n) { return (n + kFp8Block - 1) / kFp8Block; }

// The exponent code of a block's scale from the bits of its largest |x|: 2^(code - 127) is
// the smallest power of two that brings it to 448, the largest e4m3 value, or below. A power
// of two makes every quotient exact, so that codes hang on no rounding but e4m3's own; e4m3
// has exponents of its own, so that the precision does not hang on where in its range a
// block lies (only values 2^-15 below the block's largest lose a bit to the subnormals).
// 255 for a block with an infinity or a NaN, as the E8M0 format has it.
__device__ __forceinline__ int fp8_scale_code(uint32_t top_bits) {
    if (top_bits >= 0x7f800000u) return 255;
    return max((int)(top_bits >> 23) - 8 + ((top_bits & 0x7fffffu) > 0x600000u ? 1 : 0), 1);
}

// The scale and its inverse: NaN, and 0 (for which fp8_codes4 gives codes 0, also of infinities and NaNs), for
// code 255.
__device__ __forceinline__ float fp8_scale_value(int code) {
    return __uint_as_float(code == 255 ? 0x7fc00000u : (uint32_t)code << 23);
}
__device__ __forceinline__ float fp8_scale_inverse(int code) {
    return __uint_as_float(code == 255 ? 0u : (uint32_t)(254 - code) << 23);
}

// Codes of 4 values times `inv`, rounded half to even; 0 where inv is 0.
__device__ __forceinline__ uint32_t fp8_codes4(float a, float b, float c, float d, float inv) {
    int q = 0;
    q = __builtin_amdgcn_cvt_pk_fp8_f32(a * inv, b * inv, q, false);
    q = __builtin_amdgcn_cvt_pk_fp8_f32(c * inv, d * inv, q, true);
    return inv == 0.f ? 0u : (uint32_t)q;
}

// The largest of v over LANES neighbouring lanes (all active; LANES 16 or 32, aligned).
template <int LANES>
__device__ __forceinline__ uint32_t lanes_umax(uint32_t v) {
    static_assert(LANES == 16 || LANES == 32, "the lanes of a block");
    v = umax_step<1>(v);
    v = umax_step<2>(v);
    v = umax_step<4>(v);
    v = umax_step<8>(v);
    if constexpr (LANES == 32) v = umax_step<16>(v);
    return v;
}

// ------------------------------------------------------------ operands
// 32 columns of a row and block: the 16-byte units g and g + 4, g = lane / 16.
struct Frag {
    u32x4 lo, hi;
};

__device__ __forceinline__ i32x8 words8(const Frag& f) {
    return i32x8{(int)f.lo.x, (int)f.lo.y, (int)f.lo.z, (int)f.lo.w, (int)f.hi.x, (int)f.hi.y, (int)f.hi.z, (int)f.hi.w};
}

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// The values of 8 codes times a power of two: exact in bf16 from 2^-124 on. Below, the two smallest scales that there are
// (values whose block has nothing above 1e-35) go past bf16's smallest step, 2^-133, to which they are rounded.
__device__ __forceinline__ bf16x8 bf16_of(uint32_t a, uint32_t b, float scale) {
    const bf16x2 x = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, scale, false);
    const bf16x2 y = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, scale, true);
    const bf16x2 z = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, scale, false);
    const bf16x2 w = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, scale, true);
    return bf16x8{x[0], x[1], y[0], y[1], z[0], z[1], w[0], w[1]};
}

// 32 codes of a row as bf16, and the product of two such in four instructions.
struct Wide {
    bf16x8 v[4];
};

__device__ __forceinline__ Wide widen(const Frag& f, float scale) {
    return Wide{{bf16_of(f.lo.x, f.lo.y, scale), bf16_of(f.lo.z, f.lo.w, scale), bf16_of(f.hi.x, f.hi.y, scale),
                 bf16_of(f.hi.z, f.hi.w, scale)}};
}

__device__ __forceinline__ f32x4 wide_mfma(const Wide& w, const Wide& a, f32x4 c) {
#pragma unroll
    for (int i = 0; i < 4; ++i) c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w.v[i], a.v[i], c, 0, 0, 0);
    return c;
}

// The FP8 instruction adds 8 products at a time, each cut off 2^-13 below the largest exponent among
// them, before they enter its f32 sums: 1.5e-5 of a sum of normal values (2-norm), at most 2^-15.7 of
// the sum of the terms' sizes. That is 1/100 of a 16-bit result's own rounding, but 30 times an f32
// sum's. Results of 32 bits, and few that become codes (EXACT), therefore take bf16 products, which are exact and
// summed in f32 (1e-8), at half the instruction's rate.

constexpr int kBlockUnits = kFp8Block / kFp8Unit;       // 16-byte units of a row's block

// What lanes behind the last column load into LDS.
__device__ const u32x4 kZeroUnit = {0, 0, 0, 0};

__device__ __forceinline__ void load4_to_lds(const uint8_t* p, uint32_t* dst) {
    __builtin_amdgcn_global_load_lds((global_void*)p, (lds_void*)dst, 4, 0, 0);
}

// ------------------------------------------------------------ launchers
// With offsets [E + 1] (device), of the rows in [offsets[0], offsets[E]) alone.
coli_status launch_quantize_fp8(const void* x, int32_t dtype, int64_t rows, int64_t cols, int64_t ld,
                                uint8_t* q, float* s, hipStream_t stream, const int32_t* offsets = nullptr,
                                int32_t E = 0);

// `count` matrices [rows][cols], x_stride elements apart, into codes and scales (of either way
// round, nullptr: not wanted) that lie q_stride, ... bytes apart.
struct Fp8MatrixArgs {
    const void* x;
    int64_t x_stride, ld;
    uint8_t *q, *qt;
    float *s, *st;
    int64_t q_stride, s_stride, qt_stride, st_stride;
    int32_t rows, cols;
};
coli_status launch_quantize_fp8_matrix(const Fp8MatrixArgs& a, int32_t dtype, int32_t count, hipStream_t stream);

// Rows sorted by expert into codes qt [blocks][cols][128] of 128 rows of an expert by one column
// (zeros behind its last row) with the scales' exponent codes st [blocks][cols]; q, s (nullptr:
// not wanted): the rows as launch_quantize_fp8 quantises them.
struct Fp8ColumnArgs {
    const void* x;
    int64_t ld;
    const int32_t* offsets;
    uint8_t *qt, *st, *q;
    float* s;
    int32_t rows, cols, E, blocks;
};
coli_status launch_quantize_fp8_columns(const Fp8ColumnArgs& a, int32_t dtype, hipStream_t stream);

// block_rows: rows that share a scale, 1 or 128. `count` matrices: codes and scales q_stride and s_stride bytes
// apart, outputs x_stride elements.
coli_status launch_dequantize_fp8(const uint8_t* q, const float* s, int64_t rows, int64_t cols,
                                  int32_t block_rows, void* x, int32_t dtype, int64_t ld,
                                  hipStream_t stream, int32_t count = 1, int64_t q_stride = 0, int64_t s_stride = 0,
                                  int64_t x_stride = 0);
coli_status launch_dispatch_fp8(const void* x, int32_t dtype, int32_t T, int32_t k, int32_t H, int64_t ld_x,
                                const int32_t* inv, uint8_t* q, float* s, hipStream_t stream);

// Grouped product of FP8 rows with FP8 matrices; see fp8_gemm.hip.
struct Fp8GemmArgs : RowGroups {
    const uint8_t* a;            // [rows][K] codes
    const float* as;             // [rows][ceil(K / 128)] scales
    size_t q_off, s_off;         // codes and scales of the matrix (SwiGLU: of gate) in its blob
    size_t up_q, up_s;           // SwiGLU: those of up
    void* y;                     // [rows][ld] output, or codes [rows][N]
    float* ys;                   // scales [rows][ceil(N / 128)] of an FP8 output
    void* ws;                    // plan_fp8_ws bytes, or nullptr
    int64_t ld;
    int32_t K, N;                // N: rows of the matrix, of gate and of up alone
    int32_t parts;               // of the columns, whose f32 sums the workspace holds, or 0
};
// The kernel that a product runs: its rows, E, offsets, N and K decide, and whether its results have 32 bits (wide).
enum Fp8Kernel : int32_t {
    kFp8FewRows16, kFp8FewRows32,                // by matrix rows a workgroup
    kFp8Lines128, kFp8Lines256,                  // by rows a tile
};
Fp8Kernel choose_fp8_kernel(const Fp8GemmArgs& a, bool swiglu, bool wide);
coli_status launch_fp8_gemm(const Fp8GemmArgs& a, bool swiglu, int32_t dtype, hipStream_t stream);
// The bytes of workspace that a product makes use of, with a.parts for it.
size_t plan_fp8_ws(Fp8GemmArgs& a, bool swiglu, int32_t dtype);

// dw[e][n][k] = sum over the expert's rows (+ dw[e][n][k]); see fp8_wgrad.hip.
struct Fp8WgradArgs {
    const uint8_t *g, *gs;       // [blocks][N][128], [blocks][N]
    const uint8_t *x, *xs;       // [blocks][K][128], [blocks][K]
    const int32_t* offsets;
    void* dw;                    // [E][N][ld]
    int64_t ld;
    int32_t blocks, rows, E, N, K;
    bool accumulate;
    void* ws;                    // fp8_wgrad_ws bytes, or nullptr
    int32_t splits;              // parts of an expert's rows, each into a gradient of its own (the launcher's)
};
coli_status launch_fp8_wgrad(const Fp8WgradArgs& a, int32_t dtype, hipStream_t stream);
// The workspace that the gradients make use of.
size_t fp8_wgrad_ws(const Fp8WgradArgs& a);

}  // namespace coli
