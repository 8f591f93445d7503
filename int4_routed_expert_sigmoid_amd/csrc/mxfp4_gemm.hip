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
// over at most 1024 counts), so a product is one launch without a workspace. Up
// to 256 experts a lane's four offsets and blob pointers are loaded together:
// the search costs one memory latency. Consecutive workgroups run on different
// XCDs; each XCD is given one contiguous eighth of the units, ordered by
// expert, matrix rows, rows, so that units that read the same matrix rows
// follow each other behind one L2.
struct Unit {
    const uint8_t* blob;
    int m0, rows, nt;            // rows [m0, m0 + rows) (rows <= BM), n tile
};

constexpr int kLaneExperts = 4;

// First row and row count of experts e0 .. e0 + 3, clamped to the R rows; 0 rows
// from expert E on.
__device__ __forceinline__ void expert_rows(const int32_t* offsets, int e0, int E, int R,
                                            int (&lo)[kLaneExperts], int (&n)[kLaneExperts]) {
    int o[kLaneExperts + 1];
#pragma unroll
    for (int c = 0; c <= kLaneExperts; ++c) o[c] = offsets[min(e0 + c, E)];
#pragma unroll
    for (int c = 0; c < kLaneExperts; ++c) {
        lo[c] = min(max(o[c], 0), R);
        n[c] = min(max(o[c + 1], lo[c]), R) - lo[c];
    }
}

template <int BM>
__device__ __forceinline__ bool find_unit(const MxGemmArgs& a, int NT, Unit* out) {
    const int lane = threadIdx.x & 63, E = a.E, R = a.rows;
    const uint32_t xcd = blockIdx.x % kXcds, at = blockIdx.x / kXcds;
    if (a.offsets == nullptr) {
        const uint32_t mt = (R + BM - 1) / BM, total = mt * NT, per = (total + kXcds - 1) / kXcds;
        const uint32_t w = xcd * per + at;
        if (at >= per || w >= total) return false;
        out->blob = (const uint8_t*)a.table[0];
        out->nt = w / mt;
        out->m0 = (w % mt) * BM;
        out->rows = min(BM, R - out->m0);
        return true;
    }
    const int groups = (E + 64 * kLaneExperts - 1) / (64 * kLaneExperts);   // of 4 experts a lane
    const int e0 = lane * groups * kLaneExperts;
    int lo[kLaneExperts], n[kLaneExperts];
    uint32_t tiles = 0;
    for (int c = groups - 1; c >= 0; --c) {                  // ends with the lane's first group loaded
        expert_rows(a.offsets, e0 + c * kLaneExperts, E, R, lo, n);
#pragma unroll
        for (int i = 0; i < kLaneExperts; ++i) tiles += (n[i] + BM - 1) / BM;
    }
    const uint8_t* ptr[kLaneExperts];
#pragma unroll
    for (int i = 0; i < kLaneExperts; ++i) ptr[i] = (const uint8_t*)a.table[min(e0 + i, E - 1)];
    uint32_t incl = tiles;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const uint32_t v = __shfl_up(incl, o);
        if (lane >= o) incl += v;
    }
    const uint32_t total = __builtin_amdgcn_readlane(incl, 63) * NT, per = (total + kXcds - 1) / kXcds;
    const uint32_t w = xcd * per + at;
    if (at >= per || w >= total) return false;
    const uint32_t first = (incl - tiles) * NT;
    const unsigned long long has = __ballot(w >= first && w < incl * NT);
    if (has == 0) return false;                              // offsets that are not ascending
    const int owner = __ffsll(has) - 1;
    Unit u = {nullptr, 0, 0, 0};
    if (lane == owner) {
        uint32_t rest = w - first;
        for (int c = 0; c < groups; ++c) {
            if (c > 0) {
                expert_rows(a.offsets, e0 + c * kLaneExperts, E, R, lo, n);
#pragma unroll
                for (int i = 0; i < kLaneExperts; ++i)
                    ptr[i] = (const uint8_t*)a.table[min(e0 + c * kLaneExperts + i, E - 1)];
            }
#pragma unroll
            for (int i = 0; i < kLaneExperts; ++i) {
                const uint32_t mt = (n[i] + BM - 1) / BM;
                if (u.rows == 0 && rest < mt * NT) {
                    u.blob = ptr[i];
                    u.nt = rest / mt;
                    u.m0 = (int)(rest % mt) * BM;
                    u.rows = min(BM, n[i] - u.m0);
                    u.m0 += lo[i];
                }
                rest -= u.rows == 0 ? mt * NT : 0;
            }
        }
    }
    const uint64_t b = (uint64_t)u.blob;
    const uint32_t b_lo = __builtin_amdgcn_readlane((uint32_t)b, owner);
    const uint32_t b_hi = __builtin_amdgcn_readlane((uint32_t)(b >> 32), owner);
    out->blob = (const uint8_t*)((uint64_t)b_hi << 32 | b_lo);
    out->m0 = __builtin_amdgcn_readlane(u.m0, owner);
    out->rows = __builtin_amdgcn_readlane(u.rows, owner);
    out->nt = __builtin_amdgcn_readlane(u.nt, owner);
    return out->rows > 0;
}

// ------------------------------------------------------------ operands
struct __attribute__((packed, aligned(1))) Bytes16 {
    uint32_t w[4];
};
// Blob pointers come from a table in memory: without the address space their
// loads would be generic ones, which also count as LDS accesses.
typedef __attribute__((address_space(1))) const uint8_t global_u8;
typedef __attribute__((address_space(1))) const Bytes16 global_bytes16;

__device__ __forceinline__ u32x4 load16(const uint8_t* p) { return *(global_u32x4*)(p); }
// Matrix rows that one workgroup alone reads: kept out of the caches.
__device__ __forceinline__ u32x4 load16_once(const uint8_t* p) { return __builtin_nontemporal_load((global_u32x4*)(p)); }
__device__ __forceinline__ uint32_t load1(const uint8_t* p) { return *(global_u8*)(p); }

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

// The scale bytes of blocks b0 .. b0 + 15 of a row in two steps, so that the
// load can be on the way while other work runs: the 16 bytes from b0 on, or the
// row's last 16 where fewer are left (no byte outside the row is touched; KB >=
// 16), and then their shift into place, which leaves 0 (2^-127) for blocks from KB
// on; their codes are 0 on one side of the product.
__device__ __forceinline__ u32x4 load_scales16(const uint8_t* row, int b0, int KB) {
    global_bytes16* v = (global_bytes16*)(row + min(b0, KB - 16));
    return u32x4{v->w[0], v->w[1], v->w[2], v->w[3]};
}

__device__ __forceinline__ u32x4 place_scales16(const u32x4& v, int b0, int KB) {
    const int sh = 8 * (b0 + 16 - KB);               // uniform
    if (sh <= 0) return v;
    const uint64_t lo = v.x | (uint64_t)v.y << 32, hi = v.z | (uint64_t)v.w << 32;
    const uint64_t l = sh < 64 ? lo >> sh | hi << (64 - sh) : hi >> (sh - 64);
    const uint64_t h = sh < 64 ? hi >> sh : 0;
    return u32x4{(uint32_t)l, (uint32_t)(l >> 32), (uint32_t)h, (uint32_t)(h >> 32)};
}

// Everything above this point happens before everything below it: memory
// accesses by the clobber, the instructions that feed `acc` (which the compiler
// would otherwise collect at the end of the loop, with all their operands
// live) by the operands. No instruction of its own.
template <int N>
__device__ __forceinline__ void hold(f32x4 (&acc)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) asm volatile("" : "+v"(acc[i])::"memory");
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
// Workgroup: NF fragments of 16 matrix rows by up to 16 rows. Its KS waves take
// chunks of the columns in turn, so that even one row of one expert has KS
// waves a fragment set on the way, and the partial sums meet in LDS in wave
// order. Everything goes straight into the instruction's registers; a step's
// registers are refilled for the wave's next chunk as soon as the step has
// used them. Whole chunks only (TAIL false) or any number of columns.
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
    auto load_step = [&](int c, int s) {
        int b = c * kChunkBlocks + s * 4 + g;
        if (TAIL) b = min(b, KB - 1);
        av[s] = load16(a_base + (mr * row_bytes + b * 16));
#pragma unroll
        for (int f = 0; f < NF; ++f) w[s][f] = load16_once(w_base + (nr[f] * row_bytes + b * 16));
    };
    // a lane's scale byte of step s: byte g of word s
    auto load_scales = [&](int c) {
        if (!TAIL) {
            as = load_scales16(as_base + mr * (uint32_t)KB, c * kChunkBlocks, KB);
#pragma unroll
            for (int f = 0; f < NF; ++f) ws[f] = load_scales16(ws_base + nr[f] * (uint32_t)KB, c * kChunkBlocks, KB);
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
#pragma unroll
        for (int s = 0; s < kChunkSteps; ++s) load_step(wave, s);
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
            if (more) load_step(c + KS, s);
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

// ------------------------------------------------------------ many rows
// Workgroup: 4 waves, each 64 matrix rows (4 fragments) by MT fragments of 16
// rows. The matrix is the operand that has to come from HBM: each wave loads
// its own rows straight into the instruction's registers, one step's registers
// refilled for the next chunk as soon as the step has used them, so that nearly
// a chunk (16 KB a wave) is on the way all the time without a barrier. The rows
// are shared by the waves and come (from L2) over LDS, two chunks deep, and so
// do the scale bytes of both sides, which a wave then reads one per lane.
constexpr int kWaveFrags = 4;
constexpr int kTileWaves = 4;
constexpr int kTileRows = kTileWaves * kWaveFrags * kFrag;   // 256 matrix rows

// Position of 16-byte unit b of row r in the LDS chunk: the units of a row
// are permuted by its number, so that the 16 rows that a load reads at one
// column fall into different banks.
__device__ __forceinline__ int lds_unit(int r, int b) { return r * kChunkBlocks + (b ^ (r & 15)); }

template <int MT>
struct TileLds {
    u32x4 code[2][MT * kFrag * kChunkBlocks];
    u32x4 scale[2][MT * kFrag];                // a row's 16 scale bytes
    u32x4 w_scale[2][kTileRows];
};

template <typename Out, bool SWIGLU, int MT>
__global__ __launch_bounds__(64 * kTileWaves, MT <= 4 ? 2 : 1) void mx_tile_kernel(MxGemmArgs a, int NT) {
    constexpr int BM = MT * kFrag;
    constexpr int kThreads = 64 * kTileWaves;
    constexpr int kStage = BM * kChunkBlocks / kThreads;      // 16-byte units a thread stages
    __shared__ TileLds<MT> lds;
    Unit u;
    if (!find_unit<BM>(a, NT, &u)) return;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, r = lane & 15, g = lane >> 4;
    const int KB = a.K / kMxBlock, chunks = (KB + kChunkBlocks - 1) / kChunkBlocks;
    const uint32_t row_bytes = KB * 16;
    const int n_tile = u.nt * kTileRows, n_wave = n_tile + wave * kWaveFrags * kFrag;
    // bases are uniform, lanes add 32-bit offsets
    const uint8_t* w_base = u.blob + a.q_off + (int64_t)n_tile * row_bytes;
    const uint8_t* ws_row = u.blob + a.s_off + (int64_t)min(n_tile + tid, a.N - 1) * KB;
    const uint8_t* a_base = a.a + (int64_t)u.m0 * row_bytes;
    const uint8_t* as_row = a.as + (int64_t)(u.m0 + min(tid, u.rows - 1)) * KB;
    uint32_t w_off[kWaveFrags], s_off[kStage];
#pragma unroll
    for (int f = 0; f < kWaveFrags; ++f)
        w_off[f] = (uint32_t)(min(n_wave + f * kFrag + r, a.N - 1) - n_tile) * row_bytes;
#pragma unroll
    for (int i = 0; i < kStage; ++i)
        s_off[i] = (uint32_t)min((tid + i * kThreads) / kChunkBlocks, u.rows - 1) * row_bytes;

    u32x4 stage[kStage], stage_s, stage_ws;
    auto stage_load = [&](int c) {
        const int b = c * kChunkBlocks + tid % kChunkBlocks, bc = min(b, KB - 1) * 16;
#pragma unroll
        for (int i = 0; i < kStage; ++i) stage[i] = load16(a_base + (s_off[i] + bc));
        stage_ws = load_scales16(ws_row, c * kChunkBlocks, KB);
        stage_s = load_scales16(as_row, c * kChunkBlocks, KB);
    };
    auto stage_store = [&](int c, int buf) {
        const bool in = c * kChunkBlocks + tid % kChunkBlocks < KB;
#pragma unroll
        for (int i = 0; i < kStage; ++i) {
            const int x = tid + i * kThreads;
            lds.code[buf][lds_unit(x / kChunkBlocks, x % kChunkBlocks)] = in ? stage[i] : u32x4{0, 0, 0, 0};
        }
        lds.w_scale[buf][tid] = place_scales16(stage_ws, c * kChunkBlocks, KB);
        if (tid < BM) lds.scale[buf][tid] = place_scales16(stage_s, c * kChunkBlocks, KB);
    };

    u32x4 w[kChunkSteps][kWaveFrags];
    auto w_load = [&](int c, int s) {
        const uint32_t b = min(c * kChunkBlocks + s * 4 + g, KB - 1) * 16;
#pragma unroll
        for (int f = 0; f < kWaveFrags; ++f) w[s][f] = load16(w_base + (w_off[f] + b));
    };

    f32x4 acc[kWaveFrags][MT];
#pragma unroll
    for (int f = 0; f < kWaveFrags; ++f)
#pragma unroll
        for (int i = 0; i < MT; ++i) acc[f][i] = f32x4{0.f, 0.f, 0.f, 0.f};

    stage_load(0);
#pragma unroll
    for (int s = 0; s < kChunkSteps; ++s) w_load(0, s);
    stage_store(0, 0);
    __syncthreads();
    for (int c = 0; c < chunks; ++c) {
        const int buf = c & 1, next = min(c + 1, chunks - 1);
        const uint8_t* as_b = (const uint8_t*)lds.scale[buf] + r * 16 + g;
        const uint8_t* ws_b = (const uint8_t*)lds.w_scale[buf] + (wave * kWaveFrags * kFrag + r) * 16 + g;
        stage_load(next);
#pragma unroll
        for (int s = 0; s < kChunkSteps; ++s) {
            u32x4 av[MT];
            uint32_t as[MT], ws[kWaveFrags];
#pragma unroll
            for (int f = 0; f < kWaveFrags; ++f) ws[f] = ws_b[f * kFrag * 16 + s * 4];
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                as[i] = as_b[i * kFrag * 16 + s * 4];
                av[i] = lds.code[buf][lds_unit(i * kFrag + r, s * 4 + g)];
            }
#pragma unroll
            for (int f = 0; f < kWaveFrags; ++f)
#pragma unroll
                for (int i = 0; i < MT; ++i) acc[f][i] = mx_mfma(w[s][f], ws[f], av[i], as[i], acc[f][i]);
#pragma unroll
            for (int f = 0; f < kWaveFrags; ++f) hold(acc[f]);
            w_load(next, s);
            sched_fence();
        }
        stage_store(next, buf ^ 1);
        __syncthreads();
    }
    // outputs
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        const bool live = i * kFrag + r < u.rows;
        const int m = u.m0 + i * kFrag + r;
        if constexpr (!SWIGLU) {
#pragma unroll
            for (int f = 0; f < kWaveFrags; ++f)
                if (live) store4<Out>(a, m, n_wave + f * kFrag + 4 * g, a.N, acc[f][i]);
        } else {
            f32x4 h[2];
#pragma unroll
            for (int p = 0; p < 2; ++p)
#pragma unroll
                for (int x = 0; x < 4; ++x) h[p][x] = silu_mul(acc[2 * p][i][x], acc[2 * p + 1][i][x]);
            const int n0 = n_wave / 2;
            if constexpr (std::is_same<Out, MxOut>::value) {
                store_mx(a, m, n0, a.N / 2, live && n0 < a.N / 2, h[0], h[1]);
            } else {
#pragma unroll
                for (int p = 0; p < 2; ++p)
                    if (live) store4<Out>(a, m, n0 + p * kFrag + 4 * g, a.N / 2, h[p]);
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
    if (a.K % (kChunkBlocks * kMxBlock) == 0)
        launch(mx_few_rows_kernel<Out, SWIGLU, NF, KS, false>, dim3(grid), dim3(64 * KS), 0, stream, a, NT);
    else
        launch(mx_few_rows_kernel<Out, SWIGLU, NF, KS, true>, dim3(grid), dim3(64 * KS), 0, stream, a, NT);
    COLI_CHECK_LAUNCH("mxfp4 product kernel launch");
    return COLI_OK;
}

template <typename Out, bool SWIGLU, int MT>
coli_status tiles(const MxGemmArgs& a, hipStream_t stream) {
    const int NT = (a.N + kTileRows - 1) / kTileRows;
    uint32_t grid;
    if (coli_status st = grid_of(a, MT * kFrag, NT, 64 * kTileWaves, &grid)) return st;
    launch(mx_tile_kernel<Out, SWIGLU, MT>, dim3(grid), dim3(64 * kTileWaves), 0, stream, a, NT);
    COLI_CHECK_LAUNCH("mxfp4 product kernel launch");
    return COLI_OK;
}

template <typename Out, bool SWIGLU>
coli_status product(const MxGemmArgs& a, hipStream_t stream) {
    constexpr bool mx = std::is_same<Out, MxOut>::value;
    const double per = (double)a.rows / (a.offsets ? std::min(a.E, a.rows) : 1);
    if (per <= 8 || a.K < kChunkBlocks * kMxBlock) return few_rows<Out, SWIGLU, mx ? 4 : 2, 4>(a, stream);
    if (per <= 128) return tiles<Out, SWIGLU, 4>(a, stream);
    return tiles<Out, SWIGLU, 8>(a, stream);
}

}  // namespace

coli_status launch_mxfp4_gemm(const MxGemmArgs& a, bool swiglu, int32_t dtype, hipStream_t stream) {
    if (swiglu && dtype == COLI_MXFP4) return product<MxOut, true>(a, stream);
    return with_elem(dtype, [&](auto e) -> coli_status {
        using T = decltype(e);
        return swiglu ? product<T, true>(a, stream) : product<T, false>(a, stream);
    });
}

}  // namespace coli
