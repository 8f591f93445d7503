// Grouped products of MXFP4 rows with MXFP4 matrices on the scaled matrix
// instructions: y[r][n] = sum_k a[r][k] w_e(r)[n][k], rows sorted by expert.
//
// v_mfma_scale_f32_16x16x128_f8f6f4 multiplies 16 rows by 16 rows over 128
// columns: lane l holds row l % 16, columns 32 (l / 16) .. + 31, that is one
// 16-byte stretch of codes and one scale byte, exactly the stored format, so
// rows go from memory into the instruction without any unpacking. The matrix
// rows are the first operand: result lane l then holds outputs n = 4 (l / 16) ..
// + 3 of one row m = l % 16, which is one wide store. Products are exact and
// sums are f32. A step is one instruction's 128 columns; in registers alone the
// instruction runs at 8.1 PFLOP/s on this card.
//
// Up to about 100 rows an expert the products are bound by reading the matrices
// (17/32 byte a value): 256 experts' gate and up matrices of 2 x 2048 x 6144 are
// 3.4 GB. Three kernels, chosen by choose_mxfp4_kernel below:
//   few_rows  16 rows a tile, operands straight into registers: single tokens
//   lines     128 or 256 rows a tile, both operands over LDS, persistent
//   tiles     64 or 128 rows a tile, rows over LDS: any number of columns
#include <algorithm>
#include <cmath>

#include "mfma_tiles.h"

namespace coli {
namespace {

// MXFP4 as an output type of the SwiGLU epilogue.
struct MxOut {};

// ------------------------------------------------------------ operands
__device__ __forceinline__ f32x4 mx_mfma(const u32x4& w, uint32_t ws, const u32x4& a, uint32_t as,
                                         f32x4 c) {
    const i32x8 W = {(int)w.x, (int)w.y, (int)w.z, (int)w.w, 0, 0, 0, 0};
    const i32x8 A = {(int)a.x, (int)a.y, (int)a.z, (int)a.w, 0, 0, 0, 0};
    // 4: E2M1 operands; the scale is the low byte of its register
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(W, A, c, 4, 4, 0, (int)ws, 0, (int)as);
}

// Columns go through the kernels in chunks of 512: 4 steps, 16 blocks.
constexpr int kChunkSteps = 4;
constexpr int kChunkBlocks = 4 * kChunkSteps;          // 16 blocks: 512 columns

// Blocks b0 .. b0 + 15 of a row, all inside it.
__device__ __forceinline__ u32x4 load_scales16(const uint8_t* row, int b0) {
    global_bytes16* v = (global_bytes16*)(row + b0);
    return u32x4{v->w[0], v->w[1], v->w[2], v->w[3]};
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
// Workgroup: NF fragments of 16 matrix rows by up to 16 rows. Its KS waves take
// chunks of the columns in turn, so that even one row of one expert has KS
// waves a fragment set on the way, and the partial sums meet in LDS in wave
// order. Everything goes straight into the instruction's registers; those of two
// steps, 128 bytes or one cache line of every row, are refilled together for
// the wave's next chunk as soon as they are used. (Refilled step by step, the
// second half of a line came after the line had left the caches: 1.33 times the
// matrix' bytes from HBM, and 26-29 us in place of 22.6 for the SwiGLU of 8 rows
// of 8 experts, K 6144, inter 2048.) Whole chunks only (TAIL false) or any number
// of columns.
template <typename Out, bool SWIGLU, int NF, int KS, bool TAIL>
__global__ __launch_bounds__(64 * KS) void mx_few_rows_kernel(MxGemmArgs a, int NT) {
    __shared__ f32x4 part[KS][NF][64];
    Unit u;
    if (!find_unit<kFrag>(a, NT, &u)) return;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r = lane & 15, g = lane >> 4;
    const int KB = a.K / kMxBlock, chunks = (KB + kChunkBlocks - 1) / kChunkBlocks;
    const uint32_t row_bytes = KB * 16;
    const int n_tile = u.nt * NF * kFrag;
    const uint8_t* w_base = u.blob + a.q_off + (int64_t)n_tile * row_bytes;
    const uint8_t* ws_base = u.blob + a.s_off + (int64_t)n_tile * KB;
    const uint8_t* a_base = a.a + (int64_t)u.m0 * row_bytes;
    const uint8_t* as_base = a.as + (int64_t)u.m0 * KB;
    const int mr = min(r, u.rows - 1);
    int nr[NF];
#pragma unroll
    for (int f = 0; f < NF; ++f) nr[f] = min(f * kFrag + r, a.N - 1 - n_tile);

    u32x4 w[kChunkSteps][NF], av[kChunkSteps], ws[NF], as;
    auto load_pair = [&](int c, int s) {
        int b0 = c * kChunkBlocks + s * 4 + g, b1 = b0 + 4;
        if (TAIL) b0 = min(b0, KB - 1), b1 = min(b1, KB - 1);
#pragma unroll
        for (int f = 0; f < NF; ++f) {
            w[s][f] = load16(w_base + (nr[f] * row_bytes + b0 * 16));
            w[s + 1][f] = load16(w_base + (nr[f] * row_bytes + b1 * 16));
        }
        av[s] = load16(a_base + (mr * row_bytes + b0 * 16));
        av[s + 1] = load16(a_base + (mr * row_bytes + b1 * 16));
    };
    // a lane's scale byte of step s: byte g of word s
    auto load_scales = [&](int c) {
        if (!TAIL) {
            as = load_scales16(as_base + mr * (uint32_t)KB, c * kChunkBlocks);
#pragma unroll
            for (int f = 0; f < NF; ++f) ws[f] = load_scales16(ws_base + nr[f] * (uint32_t)KB, c * kChunkBlocks);
            return;
        }
#pragma unroll
        for (int s = 0; s < kChunkSteps; ++s) {
            const int b = min(c * kChunkBlocks + s * 4 + g, KB - 1);
            as[s] = load1(as_base + (mr * (uint32_t)KB + b));
#pragma unroll
            for (int f = 0; f < NF; ++f) ws[f][s] = load1(ws_base + (nr[f] * (uint32_t)KB + b));
        }
    };
    f32x4 acc[NF];
#pragma unroll
    for (int f = 0; f < NF; ++f) acc[f] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (wave < chunks) {
        load_scales(wave);
        load_pair(wave, 0);
        load_pair(wave, 2);
    }
    for (int c = wave; c < chunks; c += KS) {
        const bool more = c + KS < chunks;
        u32x4 as_c = as, ws_c[NF];
#pragma unroll
        for (int f = 0; f < NF; ++f) ws_c[f] = ws[f];
        if (more) load_scales(c + KS);
#pragma unroll
        for (int s = 0; s < kChunkSteps; ++s) {
            // a block from KB on has codes 0 on one side and the row's last scale on both
            u32x4 x = av[s];
            if (TAIL && c * kChunkBlocks + s * 4 + g >= KB) x = u32x4{0, 0, 0, 0};
            const int sh = TAIL ? 0 : 8 * g;
#pragma unroll
            for (int f = 0; f < NF; ++f) acc[f] = mx_mfma(w[s][f], ws_c[f][s] >> sh, x, as_c[s] >> sh, acc[f]);
            hold(acc);
            if (more && s % 2 == 1) load_pair(c + KS, s - 1);
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

// ------------------------------------------------------------ a tile's outputs
// A wave's outputs: L fragments of rows, STEP fragments apart (this lane's row of
// the first one: m_wave of the unit), by NF fragments of matrix rows from n_wave on.
template <typename Out, bool SWIGLU, int NF, int L, int STEP>
__device__ __forceinline__ void write_tile(const MxGemmArgs& a, int m0, int rows, int m_wave, int n_wave,
                                           const f32x4 (&acc)[L][NF]) {
    const int g = (threadIdx.x & 63) >> 4;
#pragma unroll
    for (int i = 0; i < L; ++i) {
        const int at = m_wave + i * STEP * kFrag, m = m0 + at;
        const bool live = at < rows;
        if constexpr (!SWIGLU) {
#pragma unroll
            for (int f = 0; f < NF; f += 2)
                store32<Out>(a, m, n_wave + f * kFrag, a.N, live, acc[i][f], acc[i][f + 1]);
        } else {
            f32x4 h[NF / 2];
#pragma unroll
            for (int p = 0; p < NF / 2; ++p)
#pragma unroll
                for (int x = 0; x < 4; ++x) h[p][x] = silu_mul(acc[i][2 * p][x], acc[i][2 * p + 1][x]);
            const int n0 = n_wave / 2;
            if constexpr (std::is_same<Out, MxOut>::value) {
                static_assert(NF == 4, "a wave holds one block of h");
                store_mx(a, m, n0, a.N / 2, live && n0 < a.N / 2, h[0], h[1]);
            } else {
#pragma unroll
                for (int p = 0; p < NF / 2; ++p)
                    if (live) store4<Out>(a, m, n0 + p * kFrag + 4 * g, a.N / 2, h[p]);
            }
        }
    }
}

// ------------------------------------------------------------ many rows, any columns
// Workgroup: WN waves, each NF fragments of matrix rows by MT fragments of rows.
// The matrix is the operand that has to come from HBM: each wave loads its own
// rows straight into the instruction's registers, a cache line of every row (two
// steps) refilled for the next chunk as soon as it is used, without a barrier. The
// rows are shared by the waves and come (from L2) over LDS, two chunks deep, and
// so do the scale bytes of both sides, which a wave then reads one per lane. Rows
// that are no whole chunks long end in blocks of zeros.

// BYTES (8 or 16) scale bytes.
template <int BYTES>
struct Scales {
    uint32_t w[BYTES / 4];
};

// The scale bytes of blocks b0 .. b0 + BYTES - 1 of a row in two steps, so that the
// load can be on the way while other work runs: the bytes from b0 on, or the row's
// last BYTES where fewer are left (no byte outside the row is touched: KB >= BYTES,
// or SHORT, a row of fewer, byte by byte), and then their shift into place, which
// leaves 0 (2^-127) for blocks from KB on; their codes are 0 on one side of the
// product.
template <int BYTES, bool SHORT>
__device__ __forceinline__ Scales<BYTES> load_scales(const uint8_t* row, int b0, int KB) {
    if (SHORT && KB < BYTES) {
        uint64_t v = 0;
        for (int i = 0; i < KB; ++i) v |= (uint64_t)load1(row + i) << (8 * i);
        return Scales<BYTES>{{(uint32_t)v, (uint32_t)(v >> 32)}};
    }
    typedef __attribute__((address_space(1))) const Pack<uint8_t, BYTES> G;
    G* p = (G*)(row + min(b0, KB - BYTES));
    Scales<BYTES> v;
    __builtin_memcpy(&v, p, BYTES);
    return v;
}

template <int BYTES, bool SHORT>
__device__ __forceinline__ Scales<BYTES> place_scales(const Scales<BYTES>& v, int b0, int KB) {
    const int sh = 8 * (b0 + BYTES - KB);            // uniform
    if (sh <= 0 || (SHORT && KB < BYTES)) return v;
    uint64_t lo = v.w[0] | (uint64_t)v.w[1] << 32, hi = 0;
    if constexpr (BYTES == 16) hi = v.w[2] | (uint64_t)v.w[3] << 32;
    const uint64_t l = sh < 64 ? lo >> sh | (hi << 1) << (63 - sh) : hi >> (sh - 64);
    const uint64_t h = sh < 64 ? hi >> sh : 0;
    Scales<BYTES> o;
    o.w[0] = (uint32_t)l;
    o.w[1] = (uint32_t)(l >> 32);
    if constexpr (BYTES == 16) o.w[2] = (uint32_t)h, o.w[3] = (uint32_t)(h >> 32);
    return o;
}

template <int BM, int BN, int CS>
struct TileLds {
    u32x4 code[2][BM * 4 * CS];
    Scales<4 * CS> scale[2][BM], w_scale[2][BN];
};

// Chunks of CS steps.
template <typename Out, bool SWIGLU, int MT, int NF, int WN, int CS, bool SHORT>
struct Tile {
    static constexpr int BM = MT * kFrag, BN = WN * NF * kFrag, kThreads = 64 * WN;
    static constexpr int U = 4 * CS;                          // 16-byte units of a row's chunk
    static_assert(BM <= kThreads && BN <= kThreads, "a thread stages one row's scales");
    static_assert(!SHORT || U == 8, "a short row's scales are gathered in 8 bytes");
    typedef TileLds<BM, BN, CS> Lds;

    // L: the fragments of a wave that hold rows.
    template <int L>
    static __device__ __forceinline__ void run(const MxGemmArgs& a, const Unit& u, Lds& lds) {
        constexpr int LM = L * kFrag;
        constexpr int kStage = LM * U / kThreads;             // 16-byte units a thread stages
        static_assert(LM * U % kThreads == 0, "whole units for every thread");
        const int tid = threadIdx.x, lane = tid & 63, r = lane & 15, g = lane >> 4;
        const int wn = tid >> 6;
        const int KB = a.K / kMxBlock, chunks = (KB + U - 1) / U;
        const uint32_t row_bytes = KB * 16;
        const int n_tile = u.nt * BN, n_wave = n_tile + wn * NF * kFrag;
        // bases are uniform, lanes add 32-bit offsets
        const uint8_t* w_base = u.blob + a.q_off + (int64_t)n_tile * row_bytes;
        const uint8_t* ws_row = u.blob + a.s_off + (int64_t)min(n_tile + tid, a.N - 1) * KB;
        const uint8_t* a_base = a.a + (int64_t)u.m0 * row_bytes;
        const uint8_t* as_row = a.as + (int64_t)(u.m0 + min(tid, u.rows - 1)) * KB;
        uint32_t w_off[NF], s_off[kStage];
#pragma unroll
        for (int f = 0; f < NF; ++f)
            w_off[f] = (uint32_t)(min(n_wave + f * kFrag + r, a.N - 1) - n_tile) * row_bytes;
#pragma unroll
        for (int i = 0; i < kStage; ++i)
            s_off[i] = (uint32_t)min((tid + i * kThreads) / U, u.rows - 1) * row_bytes;

        u32x4 stage[kStage];
        Scales<U> stage_s, stage_ws;
        auto stage_load = [&](int c) {
            const uint32_t b = min(c * U + tid % U, KB - 1) * 16;
#pragma unroll
            for (int i = 0; i < kStage; ++i) stage[i] = load16(a_base + (s_off[i] + b));
            stage_ws = load_scales<U, SHORT>(ws_row, c * U, KB);
            stage_s = load_scales<U, SHORT>(as_row, c * U, KB);
        };
        auto stage_store = [&](int c, int buf) {
            const bool in = c * U + tid % U < KB;
#pragma unroll
            for (int i = 0; i < kStage; ++i) {
                const int x = tid + i * kThreads;
                lds.code[buf][lds_unit<U>(x / U, x % U)] = in ? stage[i] : u32x4{0, 0, 0, 0};
            }
            if (tid < BN) lds.w_scale[buf][tid] = place_scales<U, SHORT>(stage_ws, c * U, KB);
            if (tid < LM) lds.scale[buf][tid] = place_scales<U, SHORT>(stage_s, c * U, KB);
        };

        u32x4 w[CS][NF];
        auto w_pair = [&](int c, int s) {                     // steps s and s + 1: a cache line of every row
            const int b = c * U + s * 4 + g;
            const uint32_t b0 = min(b, KB - 1) * 16, b1 = min(b + 4, KB - 1) * 16;
#pragma unroll
            for (int f = 0; f < NF; ++f) {
                w[s][f] = load16(w_base + (w_off[f] + b0));
                w[s + 1][f] = load16(w_base + (w_off[f] + b1));
            }
        };

        f32x4 acc[L][NF];
#pragma unroll
        for (int i = 0; i < L; ++i)
#pragma unroll
            for (int f = 0; f < NF; ++f) acc[i][f] = f32x4{0.f, 0.f, 0.f, 0.f};

        stage_load(0);
#pragma unroll
        for (int s = 0; s < CS; s += 2) w_pair(0, s);
        stage_store(0, 0);
        __syncthreads();
        for (int c = 0; c < chunks; ++c) {
            const int buf = c & 1, next = min(c + 1, chunks - 1);
            const uint8_t* as_b = (const uint8_t*)lds.scale[buf] + r * U + g;
            const uint8_t* ws_b = (const uint8_t*)lds.w_scale[buf] + (wn * NF * kFrag + r) * U + g;
            stage_load(next);
#pragma unroll
            for (int s = 0; s < CS; ++s) {
                u32x4 av[L];
                uint32_t as[L], ws[NF];
#pragma unroll
                for (int f = 0; f < NF; ++f) ws[f] = ws_b[f * kFrag * U + s * 4];
#pragma unroll
                for (int i = 0; i < L; ++i) {
                    as[i] = as_b[i * kFrag * U + s * 4];
                    av[i] = lds.code[buf][lds_unit<U>(i * kFrag + r, s * 4 + g)];
                }
#pragma unroll
                for (int f = 0; f < NF; ++f)
#pragma unroll
                    for (int i = 0; i < L; ++i) acc[i][f] = mx_mfma(w[s][f], ws[f], av[i], as[i], acc[i][f]);
#pragma unroll
                for (int i = 0; i < L; ++i) hold(acc[i]);
                if (s % 2 == 1) w_pair(next, s - 1);
                sched_fence();
            }
            stage_store(next, buf ^ 1);
            __syncthreads();
        }
        write_tile<Out, SWIGLU, NF, L, 1>(a, u.m0, u.rows, r, n_wave, acc);
    }
};

template <typename Out, bool SWIGLU, int MT, int NF, int WN, int CS, bool SHORT>
__global__ __launch_bounds__(64 * WN, 2) void mx_tile_kernel(MxGemmArgs a, int NT) {
    typedef Tile<Out, SWIGLU, MT, NF, WN, CS, SHORT> T;
    __shared__ typename T::Lds lds;
    Unit u;
    if (!find_unit<T::BM>(a, NT, &u)) return;
    if constexpr (MT >= 8) {
        if (u.rows <= T::BM / 2) return T::template run<MT / 2>(a, u, lds);
    }
    T::template run<MT>(a, u, lds);
}

// ------------------------------------------------------------ both sides over LDS
// Persistent workgroups of WM x WN waves, each MT fragments of rows (those with
// number i * WM + wm, so that a short stretch of rows is shared evenly) by NF
// fragments of matrix rows. Codes and scales of both operands go from memory
// straight into LDS (no registers on the way), in chunks of two steps, one cache
// line of every row. The loads run STAGES chunks ahead and straight on into the
// workgroup's next unit, so that its first chunks arrive while the unit before is
// multiplied and written. A wave waits for its own loads of a chunk by count and
// meets the others at one barrier a chunk, in its middle: by then all have the
// second step in registers, so the slot can be filled again and the next chunk's
// first step be read while the second step is multiplied. Scales come 16 bytes a
// row, for two chunks at once (4 bytes a row and chunk took more of the cache's
// cycles than the codes: 800 in place of 694 us below). An even number of whole
// chunks, at least STAGES, and scale rows on 16-byte boundaries.
//
// SwiGLU of 16384 rows over 256 experts, K 6144, inter 2048: 674 us, 5.3 TB/s; of
// 4072 rows 620 us, 5.6 TB/s, what HBM gives. Dense 8191 x 8192 x 8192: 274 us, 4.0
// PFLOP/s (the matrix instructions alone 136). There a chunk's 64 KB are on the way
// for as long as one chunk is multiplied, which does not cover their latency (LDS
// has no room for a third slot, and chunks of one step with four slots gave 331 us
// where this gave 306), and the loads behind a tile's stores wait for those (255 us
// without stores).
constexpr int kLineBlocks = 8;               // 16-byte units of a row's chunk

template <typename Out, bool SWIGLU, int MT, int NF, int WM, int WN, int STAGES>
struct LineTile {
    static constexpr int BM = WM * MT * kFrag, BN = WN * NF * kFrag, kWaves = WM * WN, kThreads = 64 * kWaves;
    static constexpr int U = kLineBlocks;
    static constexpr int kLoads = (BM + BN) * U / kThreads;   // code loads of a wave and chunk
    static constexpr int kARows = BM * U / kThreads;          // of them for the rows
    static constexpr int kScaleLoads = (BM + BN) / 64;        // 64 rows each, one per wave
    static_assert(BM * U % kThreads == 0 && BN * U % kThreads == 0, "whole loads for every wave");
    static_assert(kScaleLoads <= kWaves && BM % 64 == 0, "one scale load a wave, of rows or matrix rows");
    // The scales of chunks t and t + 1 are loaded in chunk t - STAGES behind its
    // barrier, into the slot whose last bytes, of chunk t - 3, are read before the
    // barrier of that chunk.
    static_assert(STAGES == 2 || STAGES == 3, "a scale slot is read before it is filled again");
    struct Lds {
        u32x4 code[STAGES][(BM + BN) * U];                    // rows, then matrix rows
        u32x4 scale[2][BM + BN];                              // the same order, a row's 16 bytes
        uint32_t first[kMaxExperts];                          // first unit of every expert
    };
};

template <typename Out, bool SWIGLU, int MT, int NF, int WM, int WN, int STAGES>
__global__ __launch_bounds__(64 * WM * WN, 2) void mx_line_kernel(MxGemmArgs a, int NT) {
    typedef LineTile<Out, SWIGLU, MT, NF, WM, WN, STAGES> T;
    constexpr int U = T::U;
    __shared__ typename T::Lds lds;
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wn = wave % WN, wm = wave / WN;
    const int KB = a.K / kMxBlock, chunks = KB / U;
    const uint32_t row_bytes = KB * 16;

    const uint32_t total = scan_units<T::BM, T::kThreads>(a, NT, lds.first, (uint32_t*)lds.scale[0]);
    const uint32_t per = (total + kXcds - 1) / kXcds, xcd = blockIdx.x % kXcds, step = gridDim.x / kXcds;
    uint32_t at = blockIdx.x / kXcds;        // this workgroup's units: at, at + step, ... of its XCD's `per`
    auto unit_at = [&](uint32_t x) {
        const uint32_t w = xcd * per + x;
        return line_unit<T::BM>(a, NT, lds.first, w, x < per && w < total);
    };
    LineUnit u = unit_at(at);
    if (u.rows <= 0) return;

    // the unit that is being loaded
    const uint8_t *w_base, *ws_base, *a_base, *as_base;
    int m_last, n_last;                      // its last row and matrix row
    int lc = 0;                              // its next chunk
    bool loading = true;
    auto set_unit = [&](const LineUnit& v) {
        const int n_tile = v.nt * T::BN;
        m_last = v.rows - 1, n_last = a.N - 1 - n_tile;
        w_base = v.blob + a.q_off + (int64_t)n_tile * row_bytes;
        ws_base = v.blob + a.s_off + (int64_t)n_tile * KB;
        a_base = a.a + (int64_t)v.m0 * row_bytes;
        as_base = a.as + (int64_t)v.m0 * KB;
        lc = 0;
    };
    // Load i of this wave for the next chunk: 8 rows into a slot, lane l row l / 8,
    // position l % 8. Behind the last unit the same number of loads goes out, so that
    // the counts hold, each of one place and into a slot that is not read again.
    const uint32_t unit16 = ((lane & 7) ^ (lane >> 3)) * 16;
    auto load_codes = [&](int slot, int i) {
        const bool rows = i < T::kARows;
        const int x = (rows ? i : i - T::kARows) * T::kWaves + wave;
        const uint32_t row = min(x * 8 + (lane >> 3), rows ? m_last : n_last);
        load_to_lds((rows ? a_base : w_base) + (loading ? __umul24(row, row_bytes) + lc * U * 16 + unit16 : 0u),
                    lds.code[slot] + (rows ? x : T::BM / 8 + x) * 64);
    };
    // With the first of two chunks, their scales: 64 rows a wave (two waves the same
    // ones where there are fewer).
    int scale_fill = 0;                      // the scale slot that is filled next
    auto load_scales = [&]() {
        const int x = min(wave, T::kScaleLoads - 1);
        const bool rows = x * 64 < T::BM;
        const uint32_t row = min(x * 64 - (rows ? 0 : T::BM) + lane, rows ? m_last : n_last);
        load_to_lds((rows ? as_base : ws_base) + (loading ? __umul24(row, KB) + lc * U : 0u),
                    lds.scale[scale_fill] + x * 64);
        scale_fill ^= 1;
    };

    set_unit(u);
    __syncthreads();                         // the scan's scratch is a scale slot
#pragma unroll
    for (int c = 0; c < STAGES; ++c, ++lc) {
        if (c % 2 == 0) load_scales();
#pragma unroll
        for (int i = 0; i < T::kLoads; ++i) load_codes(c, i);
    }

    const int m_lds = wm * kFrag + r, n_lds = T::BM + wn * NF * kFrag + r;
    auto code = [&](int slot, int row, int s) { return lds.code[slot][lds_unit<U>(row, s * 4 + g)]; };
    // the scale byte of step s of the even (0) or odd (1) chunk of a scale slot
    auto scale = [&](int from, int row, int odd, int s) {
        return (uint32_t)((const uint8_t*)lds.scale[from])[row * 16 + odd * U + s * 4 + g];
    };
    u32x4 av[MT], w[NF], w_next[NF];
    uint32_t as[MT], ws[NF], ws_next[NF];
    f32x4 acc[MT][NF];
    int slot = 0, scales = 0;                // of the chunk that is multiplied
    wait_loads<(STAGES - 1) * T::kLoads>();
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
#pragma unroll
    for (int f = 0; f < NF; ++f) w[f] = code(0, n_lds + f * kFrag, 0), ws[f] = scale(0, n_lds + f * kFrag, 0, 0);
#pragma unroll
    for (int i = 0; i < MT; ++i) av[i] = code(0, m_lds + i * WM * kFrag, 0), as[i] = scale(0, m_lds + i * WM * kFrag, 0, 0);
    while (true) {
        const int live = (u.rows - wm * kFrag + WM * kFrag - 1) / (WM * kFrag);   // fragments with rows
        at += step;
        const LineUnit next = unit_at(at);
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int f = 0; f < NF; ++f) acc[i][f] = f32x4{0.f, 0.f, 0.f, 0.f};
        // Multiplies the step in the registers and reads step s of a chunk into those it
        // leaves; between the products, a share of the loads into slot `fill` (-1: none).
        auto multiply = [&](int from, int from_scales, int odd, int s, int fill) {
#pragma unroll
            for (int f = 0; f < NF; ++f) {
                w_next[f] = code(from, n_lds + f * kFrag, s);
                ws_next[f] = scale(from_scales, n_lds + f * kFrag, odd, s);
            }
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                if (MT > 4 || i < live) {
#pragma unroll
                    for (int f = 0; f < NF; ++f) acc[i][f] = mx_mfma(w[f], ws[f], av[i], as[i], acc[i][f]);
                    hold(acc[i]);
                }
                av[i] = code(from, m_lds + i * WM * kFrag, s);
                as[i] = scale(from_scales, m_lds + i * WM * kFrag, odd, s);
                if (fill >= 0) {
#pragma unroll
                    for (int x = i * T::kLoads / MT; x < (i + 1) * T::kLoads / MT; ++x) load_codes(fill, x);
                }
            }
#pragma unroll
            for (int f = 0; f < NF; ++f) w[f] = w_next[f], ws[f] = ws_next[f];
        };
#pragma unroll 1
        for (int c = 0; c < chunks; ++c) {
            const int odd = c & 1;
            multiply(slot, scales, odd, 1, -1);
            // The next chunk and its scales (issued before its codes) have arrived, the
            // codes of the STAGES - 2 behind it may not have, and this one is read.
            wait_loads<(STAGES - 2) * T::kLoads>();
            __builtin_amdgcn_s_barrier();
            asm volatile("" ::: "memory");
            if (lc == chunks) {
                loading = next.rows > 0;
                set_unit(loading ? next : u);
            }
            if (lc % 2 == 0) load_scales();
            const int fill = slot;
            slot = slot == STAGES - 1 ? 0 : slot + 1;
            scales ^= odd;
            multiply(slot, scales, odd ^ 1, 0, fill);
            ++lc;
        }
        write_tile<Out, SWIGLU, NF, MT, WM>(a, u.m0, u.rows, m_lds, u.nt * T::BN + wn * NF * kFrag, acc);
        if (next.rows <= 0) break;
        u = next;
    }
    wait_loads<0>();                         // nothing lands in LDS after the workgroup
}

template <typename Out, bool SWIGLU, int NF, int KS>
coli_status few_rows(const MxGemmArgs& a, hipStream_t stream) {
    const int NT = (a.N + NF * kFrag - 1) / (NF * kFrag);
    uint32_t grid;
    if (coli_status st = grid_of(a, kFrag, NT, 64 * KS, "mxfp4 product", &grid)) return st;
    if (a.K % (kChunkBlocks * kMxBlock) == 0)
        launch(mx_few_rows_kernel<Out, SWIGLU, NF, KS, false>, dim3(grid), dim3(64 * KS), 0, stream, a, NT);
    else
        launch(mx_few_rows_kernel<Out, SWIGLU, NF, KS, true>, dim3(grid), dim3(64 * KS), 0, stream, a, NT);
    COLI_CHECK_LAUNCH("mxfp4 product kernel launch");
    return COLI_OK;
}

template <typename Out, bool SWIGLU, int MT, int NF, int WN, int CS, bool SHORT>
coli_status tiles(const MxGemmArgs& a, hipStream_t stream) {
    typedef Tile<Out, SWIGLU, MT, NF, WN, CS, SHORT> T;
    const int NT = (a.N + T::BN - 1) / T::BN;
    uint32_t grid;
    if (coli_status st = grid_of(a, T::BM, NT, T::kThreads, "mxfp4 product", &grid)) return st;
    launch(mx_tile_kernel<Out, SWIGLU, MT, NF, WN, CS, SHORT>, dim3(grid), dim3(T::kThreads), 0, stream, a, NT);
    COLI_CHECK_LAUNCH("mxfp4 product kernel launch");
    return COLI_OK;
}

template <typename Out, bool SWIGLU, int MT, int NF, int WM, int WN, int STAGES>
coli_status lines(const MxGemmArgs& a, hipStream_t stream) {
    typedef LineTile<Out, SWIGLU, MT, NF, WM, WN, STAGES> T;
    const int NT = (a.N + T::BN - 1) / T::BN;
    uint32_t grid;
    if (coli_status st = grid_of(a, T::BM, NT, 1, "mxfp4 product", &grid)) return st;
    grid = std::min(grid, kCus);             // LDS holds one workgroup a CU
    launch(mx_line_kernel<Out, SWIGLU, MT, NF, WM, WN, STAGES>, dim3(grid), dim3(T::kThreads), 0, stream, a, NT);
    COLI_CHECK_LAUNCH("mxfp4 product kernel launch");
    return COLI_OK;
}

template <typename Out, bool SWIGLU>
coli_status product(const MxGemmArgs& a, hipStream_t stream) {
    constexpr int kFew = std::is_same<Out, MxOut>::value ? 4 : 2;   // a block of h is four fragments
    switch (choose_mxfp4_kernel(a)) {
        case kMxFewRows2: return few_rows<Out, SWIGLU, kFew, 2>(a, stream);
        case kMxFewRows4: return few_rows<Out, SWIGLU, kFew, 4>(a, stream);
        case kMxTilesShort: return tiles<Out, SWIGLU, 8, 4, 4, 2, true>(a, stream);
        case kMxTiles64: return tiles<Out, SWIGLU, 4, 4, 4, 4, false>(a, stream);
        case kMxTiles128: return tiles<Out, SWIGLU, 8, 4, 4, 2, false>(a, stream);
        case kMxLines128: return lines<Out, SWIGLU, 4, 4, 2, 4, 3>(a, stream);
        default: return lines<Out, SWIGLU, 8, 4, 2, 4, 2>(a, stream);
    }
}

}  // namespace

// Which kernel, from the average rows of an expert (`per`) and the workgroups the
// kernel would have. Times on one MI355X, us: SwiGLU K 6144, inter 2048 / product
// K 2048, N 6144, over 256 experts unless noted.
//  - few_rows keeps 16 rows a tile and reads the matrix once per tile. 2 rows an
//    expert: 497 / 262 against 498 / 265 for lines; 4: 598 / 321 against 587 / 312.
//    Where lines would not fill the CUs it wins for longer, until its reads, at 5.2
//    TB/s, and 3 us of its own take longer than lines' chunks, 1.1 us each, and
//    their 7.8: one product of N 8192, K 8192 and 64 rows 30.5 against 40.1, 96 rows
//    44.1 against 42.9; N 6144, K 2048 and 128 rows 12.2 against 16.4, 192 rows 17.8
//    against 16.3; eight of N 2048, K 2048 and 48 rows 14.2 against 15.6, 64 rows
//    16.7 against 16.2. Against tiles it is given a little more: N 6144, K 2080 and
//    128 rows 13.9 against 19.8, 192 rows 20.0 against 18.1.
//  - lines of 256 rows halve the traffic into LDS of lines of 128, once they fill
//    the CUs: N 8192, K 8192, 2048 rows 78 against 99, 1024 rows 68 against 52.
//  - tiles take what lines cannot (columns not in 512s, fewer than 1024, scales off
//    16 bytes): 16384 rows over 256 experts 877 / 449 against 698 / 394 for lines.
//    Against few_rows they win from more rows: 128 experts, K 2880, inter 2048, 8
//    rows an expert 186 against 217; K 2080, N 2880, 109 against 120.
MxKernel choose_mxfp4_kernel(const MxGemmArgs& a) {
    const int64_t experts = a.offsets ? std::min(a.E, a.rows) : 1;
    const double per = (double)a.rows / experts;
    auto units = [&](int bm, int bn) { return experts * (int64_t)std::ceil(per / bm) * ((a.N + bn - 1) / bn); };
    const bool fits = a.K % 512 == 0 && a.K >= 1024 && a.s_off % 16 == 0 && (uintptr_t)a.as % 16 == 0;
    const double reads_us = std::ceil(per / kFrag) * experts * a.N * (a.K * (17 / 32.0)) / 5.2e6;
    const double chunks_us = fits ? 1.1 * a.K / 256 + 4.8 : 1.2 * a.K / 256 + 5;   // less few_rows' own
    const bool few = per <= (fits ? 2 : 4) || (units(fits ? 128 : 64, 256) < kCus && reads_us < chunks_us);
    // a wave takes at least two chunks where there are that many: 12.5 us with 2
    // waves against 14.2 with 4 for 8 rows of 8 experts at K 2048, N 6144 (4
    // chunks), 23.8 with 4 against 24.9 with 2 at K 6144, inter 2048 (12)
    if (few) return a.K >= 8 * kChunkBlocks * kMxBlock ? kMxFewRows4 : kMxFewRows2;
    if (fits) return per >= 1024 && units(256, 256) >= kCus ? kMxLines256 : kMxLines128;
    // the other two load 8 and 16 scales of a row at once (short rows: 8000 x 8000 x
    // 224 56 us against 184 for few_rows, 4000 x 5000 x 96 24 against 60)
    if (a.K < 512) return kMxTilesShort;
    // 64-row tiles leave two workgroups a CU: 681 against 755 us for 4072 rows over
    // 256 experts (K 6144, inter 2048), 908 against 865 for 16384
    return per <= 32 ? kMxTiles64 : kMxTiles128;
}

coli_status launch_mxfp4_gemm(const MxGemmArgs& a, bool swiglu, int32_t dtype, hipStream_t stream) {
    if (swiglu && dtype == COLI_MXFP4) return product<MxOut, true>(a, stream);
    return with_elem(dtype, [&](auto e) -> coli_status {
        using T = decltype(e);
        return swiglu ? product<T, true>(a, stream) : product<T, false>(a, stream);
    });
}

}  // namespace coli
