// Grouped products of MXFP4 rows with MXFP4 matrices on the scaled matrix
// instructions: y[r][n] = sum_k a[r][k] w_e(r)[n][k], rows sorted by expert.
//
// v_mfma_scale_f32_16x16x128_f8f6f4 multiplies 16 rows by 16 rows over 128
// columns: lane l holds row l % 16, columns 32 (l / 16) .. + 31, that is one
// 16-byte stretch of codes and one scale byte, exactly the stored format, so
// rows go from memory into the instruction without any unpacking. The matrix
// rows are the first operand: result lane l then holds outputs n = 4 (l / 16) ..
// + 3 of one row m = l % 16, which is one wide store. Products are exact and
// sums are f32.
#include <algorithm>

#include "mxfp4.h"

namespace coli {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kFrag = 16;                    // rows of one operand of the instruction
constexpr int kStep = 128;                   // columns of one instruction
constexpr int kStepBytes = kStep / 2;
constexpr int kXcds = 8;

// MXFP4 as an output type of the SwiGLU epilogue.
struct MxOut {};

// ------------------------------------------------------------ work units
// Unit `w` of the launch: an expert, a stretch of its rows and a stretch of the
// matrix' rows. Every wave finds its unit from the offsets by itself (a scan
// over at most 1024 counts, 16 a lane), so a product is one launch without a
// workspace. Consecutive workgroups run on different XCDs; each XCD is given
// one contiguous eighth of the units, ordered by expert, matrix rows, rows, so
// that units that read the same matrix rows follow each other behind one L2.
struct Unit {
    int e, m0, rows, nt;         // rows [m0, m0 + rows) (rows <= BM), n tile
};

__device__ __forceinline__ bool find_unit(const int32_t* offsets, int E, int R, int BM, int NT,
                                          Unit* out) {
    const int lane = threadIdx.x & 63;
    const uint32_t xcd = blockIdx.x % kXcds, at = blockIdx.x / kXcds;
    if (offsets == nullptr) {
        const uint32_t mt = (R + BM - 1) / BM, total = mt * NT, per = (total + kXcds - 1) / kXcds;
        const uint32_t w = xcd * per + at;
        if (at >= per || w >= total) return false;
        out->e = 0;
        out->nt = w / mt;
        out->m0 = (w % mt) * BM;
        out->rows = min(BM, R - out->m0);
        return true;
    }
    const int C = (E + 63) / 64;             // experts of a lane
    uint32_t tiles = 0;
    for (int c = 0; c < C; ++c) {
        const int e = lane * C + c;
        if (e >= E) break;
        const int lo = min(max(offsets[e], 0), R), hi = min(max(offsets[e + 1], lo), R);
        tiles += (hi - lo + BM - 1) / BM;
    }
    uint32_t incl = tiles;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const uint32_t v = __shfl_up(incl, o);
        if (lane >= o) incl += v;
    }
    const uint32_t total = __shfl(incl, 63) * NT, per = (total + kXcds - 1) / kXcds;
    const uint32_t w = xcd * per + at;
    if (at >= per || w >= total) return false;
    const uint32_t first = (incl - tiles) * NT;
    const unsigned long long has = __ballot(w >= first && w < incl * NT);
    if (has == 0) return false;              // offsets that are not ascending
    const int owner = __ffsll(has) - 1;
    Unit u = {0, 0, 0, 0};
    if (lane == owner) {
        uint32_t rest = w - first;
        for (int c = 0; c < C; ++c) {
            const int e = lane * C + c;
            if (e >= E) break;
            const int lo = min(max(offsets[e], 0), R), hi = min(max(offsets[e + 1], lo), R);
            const uint32_t mt = (hi - lo + BM - 1) / BM;
            if (rest < mt * NT) {
                u.e = e;
                u.nt = rest / mt;
                u.m0 = lo + (int)(rest % mt) * BM;
                u.rows = min(BM, hi - u.m0);
                break;
            }
            rest -= mt * NT;
        }
    }
    out->e = __builtin_amdgcn_readlane(u.e, owner);
    out->m0 = __builtin_amdgcn_readlane(u.m0, owner);
    out->rows = __builtin_amdgcn_readlane(u.rows, owner);
    out->nt = __builtin_amdgcn_readlane(u.nt, owner);
    return out->rows > 0;
}

// ------------------------------------------------------------ operands
struct __attribute__((packed, aligned(1))) Bytes16 {
    uint32_t w[4];
};

__device__ __forceinline__ f32x4 mx_mfma(const u32x4& w, uint32_t ws, const u32x4& a, uint32_t as,
                                         f32x4 c) {
    const i32x8 W = {(int)w.x, (int)w.y, (int)w.z, (int)w.w, 0, 0, 0, 0};
    const i32x8 A = {(int)a.x, (int)a.y, (int)a.z, (int)a.w, 0, 0, 0, 0};
    // 4: E2M1 operands; the scale is the low byte of its register
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(W, A, c, 4, 4, 0, (int)ws, 0, (int)as);
}

// ------------------------------------------------------------ epilogues
__device__ __forceinline__ float silu_mul(float g, float u) { return g / (1.f + expf(-g)) * u; }

// Outputs n0 .. n0 + 3 (those below N) of row `m`.
template <typename T>
__device__ __forceinline__ void store4(const MxGemmArgs& a, int m, int n0, int N, const f32x4& v) {
    T* p = (T*)a.y + (int64_t)m * a.ld + n0;
    const float r[4] = {v.x, v.y, v.z, v.w};
    if (n0 + 4 <= N) {
        store_f32<T, 4>(p, r);
    } else {
        for (int i = 0; i < 4 && n0 + i < N; ++i) p[i] = (T)r[i];
    }
}

// One block of 32 h of row `m`, starting at column n0: this lane holds columns
// 4 g .. + 3 (lo) and 16 + 4 g .. + 3 (hi), g = lane / 16; the four lanes of a row
// are 16 apart.
__device__ __forceinline__ void store_mx(const MxGemmArgs& a, int m, int n0, int n_out, bool live,
                                         const f32x4& lo, const f32x4& hi) {
    const int g = (threadIdx.x & 63) >> 4;
    const float v[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, abs_bits(v[i]));
    top = max(top, (uint32_t)__shfl_xor((int)top, 16));
    top = max(top, (uint32_t)__shfl_xor((int)top, 32));
    const int code = mx_scale_code(top);
    const uint32_t q = code == 255 ? 0u : mx_codes8(v, mx_scale_value(code));
    if (!live) return;
    uint16_t* p = (uint16_t*)((uint8_t*)a.y + (int64_t)m * (n_out / 2) + n0 / 2);
    p[g] = (uint16_t)q;
    p[4 + g] = (uint16_t)(q >> 16);
    if (g == 0) a.ys[(int64_t)m * (n_out / kMxBlock) + n0 / kMxBlock] = (uint8_t)code;
}

// ------------------------------------------------------------ few rows
// Workgroup: NF fragments of 16 matrix rows by up to 16 rows; the columns are
// split over its KS waves in stretches of whole steps, so that even one row of
// one expert has KS waves a fragment set on the way, and the partial sums meet
// in LDS in wave order.
template <typename Out, bool SWIGLU, int NF, int KS>
__global__ __launch_bounds__(64 * KS) void mx_few_rows_kernel(MxGemmArgs a, int NT) {
    __shared__ f32x4 part[KS][NF][64];
    Unit u;
    if (!find_unit(a.offsets, a.E, a.rows, kFrag, NT, &u)) return;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r = lane & 15, g = lane >> 4;
    const uint8_t* blob = (const uint8_t*)a.table[u.e];
    const int KB = a.K / kMxBlock, steps = (KB + 3) / 4;
    const int m = u.m0 + min(r, u.rows - 1);
    const uint8_t* ap = a.a + (int64_t)m * (a.K / 2);
    const uint8_t* asp = a.as + (int64_t)m * KB;
    const uint8_t *wp[NF], *wsp[NF];
#pragma unroll
    for (int f = 0; f < NF; ++f) {
        const int64_t n = min((u.nt * NF + f) * kFrag + r, a.N - 1);
        wp[f] = blob + a.q_off + n * (a.K / 2);
        wsp[f] = blob + a.s_off + n * KB;
    }
    f32x4 acc[NF];
#pragma unroll
    for (int f = 0; f < NF; ++f) acc[f] = f32x4{0.f, 0.f, 0.f, 0.f};
    const int s0 = (int)((int64_t)steps * wave / KS), s1 = (int)((int64_t)steps * (wave + 1) / KS);
    for (int s = s0; s < s1; ++s) {
        const int b = s * 4 + g;
        const bool in = b < KB;              // the last step may have fewer than 4 blocks
        const int bc = in ? b : KB - 1;
        u32x4 av = *(const u32x4*)(ap + bc * 16);
        const uint32_t as = asp[bc];
        if (!in) av = u32x4{0, 0, 0, 0};
#pragma unroll
        for (int f = 0; f < NF; ++f) {
            u32x4 wv = *(const u32x4*)(wp[f] + bc * 16);
            const uint32_t ws = wsp[f][bc];
            if (!in) wv = u32x4{0, 0, 0, 0};
            acc[f] = mx_mfma(wv, in ? ws : 0u, av, in ? as : 0u, acc[f]);
        }
    }
#pragma unroll
    for (int f = 0; f < NF; ++f) part[wave][f][lane] = acc[f];
    __syncthreads();
    constexpr int kOutputs = SWIGLU ? (std::is_same<Out, MxOut>::value ? NF / 4 : NF / 2) : NF;
    for (int o = wave; o < kOutputs; o += KS) {
        auto sum = [&](int f) {
            f32x4 v = part[0][f][lane];
#pragma unroll
            for (int w = 1; w < KS; ++w) v += part[w][f][lane];
            return v;
        };
        const bool live = r < u.rows;
        if constexpr (!SWIGLU) {
            const f32x4 v = sum(o);
            const int n0 = (u.nt * NF + o) * kFrag + 4 * g;
            if (live) store4<Out>(a, u.m0 + r, n0, a.N, v);
        } else {
            auto pair = [&](int f) {
                const f32x4 gv = sum(f), uv = sum(f + 1);
                f32x4 h;
#pragma unroll
                for (int i = 0; i < 4; ++i) h[i] = silu_mul(gv[i], uv[i]);
                return h;
            };
            if constexpr (std::is_same<Out, MxOut>::value) {
                const int n0 = (u.nt * (NF / 4) + o) * kMxBlock;
                const f32x4 lo = pair(4 * o), hi = pair(4 * o + 2);
                store_mx(a, u.m0 + r, n0, a.N / 2, live && n0 < a.N / 2, lo, hi);
            } else {
                const int n0 = (u.nt * (NF / 2) + o) * kFrag + 4 * g;
                const f32x4 h = pair(2 * o);
                if (live) store4<Out>(a, u.m0 + r, n0, a.N / 2, h);
            }
        }
    }
}

// Units of a launch at most: the rows fill rows / BM stretches, and each expert
// with rows may add one that is not full.
coli_status grid_of(const MxGemmArgs& a, int BM, int NT, int threads, uint32_t* grid) {
    const int64_t stretches = a.offsets ? (int64_t)a.rows / BM + std::min(a.E, a.rows)
                                        : ((int64_t)a.rows + BM - 1) / BM;
    const int64_t g = (stretches * NT + kXcds - 1) / kXcds * kXcds;
    if (g * threads > 0xffffffffll) return fail(COLI_EUNSUPPORTED, "mxfp4 product: more than 2^32 threads");
    *grid = (uint32_t)g;
    return COLI_OK;
}

template <typename Out, bool SWIGLU, int NF, int KS>
coli_status few_rows(const MxGemmArgs& a, hipStream_t stream) {
    const int NT = (a.N + NF * kFrag - 1) / (NF * kFrag);
    uint32_t grid;
    if (coli_status st = grid_of(a, kFrag, NT, 64 * KS, &grid)) return st;
    launch(mx_few_rows_kernel<Out, SWIGLU, NF, KS>, dim3(grid), dim3(64 * KS), 0, stream, a, NT);
    COLI_CHECK_LAUNCH("mxfp4 product kernel launch");
    return COLI_OK;
}

}  // namespace

coli_status launch_mxfp4_gemm(const MxGemmArgs& a, bool swiglu, int32_t dtype, hipStream_t stream) {
    if (swiglu && dtype == COLI_MXFP4) return few_rows<MxOut, true, 4, 4>(a, stream);
    return with_elem(dtype, [&](auto e) -> coli_status {
        using T = decltype(e);
        return swiglu ? few_rows<T, true, 2, 4>(a, stream) : few_rows<T, false, 1, 4>(a, stream);
    });
}

}  // namespace coli
