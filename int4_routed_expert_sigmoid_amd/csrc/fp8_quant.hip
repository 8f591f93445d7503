// FP8 rows and matrices: e4m3 codes with a scale for each block of 128 columns (of one row, or of 128 rows of a
// matrix), the same by columns for a product over rows, and back.
//
// A lane takes 16 bytes of values (4 or 8 columns), so that a block of a row is 32 or 16 lanes and its largest |x|
// is theirs by DPP exchanges. Scales are powers of two (fp8.h): x / scale is exact and e4m3's rounding (the
// hardware convert, half to even) is the only one. All of these are bound by HBM. On one MI355X (a copy: 4.7 TB/s):
// 16383 rows of 2048 bf16, 102 MB, 21 us, and back 15 (out of the caches, in part); 16 matrices of 6144 x 2048 f32
// both ways round, 1.2 GB, 190 us (6.4 TB/s), and back from either, 103; the columns of 16384 rows of 2048 bf16 by
// 64 experts, with the rows, 134 MB, 37, of 6144 without, 302 MB, 71 (48 and 98 with the tile in f32, which leaves
// room for three workgroups a CU in place of six).
#include "fp8.h"

namespace coli {
namespace {

constexpr int kThreads = 256;
// A launch holds fewer than 2^32 threads.
constexpr int64_t kMaxGrid = (int64_t(1) << 32) / kThreads - 1;

template <typename T>
constexpr int kVec = 16 / (int)sizeof(T);           // columns of a lane
template <typename T>
constexpr int kLanes = kFp8Block / kVec<T>;         // lanes of a block

// Codes of a lane's columns.
template <int N>
__device__ __forceinline__ void store_codes(uint8_t* p, const float (&v)[N], float inv) {
    if constexpr (N == 4) {
        *(uint32_t*)p = fp8_codes4(v[0], v[1], v[2], v[3], inv);
    } else {
        typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
        *(u32x2*)p = u32x2{fp8_codes4(v[0], v[1], v[2], v[3], inv), fp8_codes4(v[4], v[5], v[6], v[7], inv)};
    }
}

template <int N>
__device__ __forceinline__ uint32_t top_bits(const float (&v)[N]) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) top = max(top, abs_bits(v[i]));
    return top;
}

// Units of kVec columns; a row has whole blocks of them, of which the last one's may lie behind
// its columns.
struct UnitMap {
    int64_t units, per_row;
    int64_t ld;
    int32_t cols;
};

__device__ __forceinline__ void locate(const UnitMap& m, int64_t u, int64_t* row, int64_t* at) {
    if (m.units <= 0xffffffffll) {
        const uint32_t r = (uint32_t)u / (uint32_t)m.per_row;
        *row = r;
        *at = (uint32_t)u - r * (uint32_t)m.per_row;
    } else {
        *row = u / m.per_row;
        *at = u - *row * m.per_row;
    }
}

// ------------------------------------------------------------ rows
template <typename T, bool BOUNDED>
__global__ __launch_bounds__(kThreads) void quantize_rows_kernel(const T* __restrict__ x, UnitMap m,
                                                                 uint8_t* __restrict__ q,
                                                                 float* __restrict__ s,
                                                                 const int32_t* __restrict__ offsets, int E) {
    constexpr int N = kVec<T>;
    const int64_t u = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (u >= m.units) return;                     // whole blocks: their lanes come together
    int64_t row, at;
    locate(m, u, &row, &at);
    const int64_t c = at * N;
    const bool mine = !BOUNDED || (row >= offsets[0] && row < offsets[E]);      // alike in a block's lanes
    const bool in = c < m.cols && mine;
    float v[N] = {};
    if (in) load_f32_once<T, N>(x + row * m.ld + c, v);
    const int code = fp8_scale_code(lanes_umax<kLanes<T>>(top_bits(v)));
    if (in) store_codes(q + row * m.cols + c, v, fp8_scale_inverse(code));
    if (threadIdx.x % kLanes<T> == 0 && mine) s[u / kLanes<T>] = fp8_scale_value(code);
}

// The same into the experts' order: a token is read and converted once, its codes and scales go to
// all of its rows.
template <typename T>
__global__ __launch_bounds__(kThreads) void dispatch_fp8_kernel(
    const T* __restrict__ x, int64_t ld_x, int k, int H, int64_t n, int tiles,
    const int32_t* __restrict__ inv, uint8_t* __restrict__ q, float* __restrict__ s) {
    constexpr int N = kVec<T>, L = kLanes<T>;
    const int64_t t = blockIdx.x / (uint32_t)tiles;
    const int u = (blockIdx.x % (uint32_t)tiles) * kThreads + threadIdx.x, c = u * N;
    const int SB = (int)fp8_blocks(H);
    if (u >= SB * L) return;                      // whole blocks
    const bool in = c < H;
    float v[N] = {};
    if (in) load_f32<T, N>(x + t * ld_x + c, v);
    const int code = fp8_scale_code(lanes_umax<L>(top_bits(v)));
    const float inverse = fp8_scale_inverse(code), scale = fp8_scale_value(code);
    for (int j = 0; j < k; ++j) {
        const int32_t p = inv[t * k + j];
        if (p < 0 || p >= n) continue;
        if (in) store_codes(q + (int64_t)p * H + c, v, inverse);
        if (threadIdx.x % L == 0) s[(int64_t)p * SB + u / L] = scale;
    }
}

// A thread takes U units of kVec columns, kThreads apart; `per` workgroups a matrix.
template <typename T, int U>
__global__ __launch_bounds__(kThreads) void dequantize_kernel(const uint8_t* __restrict__ q,
                                                              const float* __restrict__ s, UnitMap m,
                                                              int block_rows, T* __restrict__ x, uint32_t per,
                                                              int64_t q_stride, int64_t s_stride, int64_t x_stride) {
    constexpr int N = kVec<T>, W = N / 4;
    const uint32_t mat = blockIdx.x / per;
    q += mat * q_stride;
    s = (const float*)((const uint8_t*)s + mat * s_stride);
    x += mat * x_stride;
    const int64_t u0 = (int64_t)(blockIdx.x - mat * per) * (kThreads * U) + threadIdx.x;
    const int64_t SB = fp8_blocks(m.cols);
    Pack<uint32_t, W> w[U];
    float sc[U];
    int64_t out[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
        const int64_t u = min(u0 + i * kThreads, m.units - 1);
        int64_t row, at;
        locate(m, u, &row, &at);
        w[i] = *reinterpret_cast<const Pack<uint32_t, W>*>(q + u * N);
        sc[i] = s[(block_rows == 1 ? row : row / kFp8Block) * SB + at * N / kFp8Block];
        out[i] = row * m.ld + at * N;
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
        if (u0 + i * kThreads >= m.units) return;
        float v[N];
#pragma unroll
        for (int j = 0; j < W; ++j) {
            typedef float f32x2 __attribute__((ext_vector_type(2)));
            const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[i].v[j], false);
            const f32x2 hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[i].v[j], true);
            v[4 * j] = lo.x * sc[i], v[4 * j + 1] = lo.y * sc[i];
            v[4 * j + 2] = hi.x * sc[i], v[4 * j + 3] = hi.y * sc[i];
        }
        store_f32_once<T, N>(x + out[i], v);
    }
}

// ------------------------------------------------------------ tiles of 128 x 128
// A workgroup holds a tile in registers, in its own type: pass p of a thread is row p * kRows + tid / kLanes, columns
// kVec (tid % kLanes) on; what lies outside the matrix is 0.
template <typename T>
struct TileIn {
    static constexpr int N = kVec<T>, L = kLanes<T>, kRows = kThreads / L, kPasses = kFp8Block / kRows;
    typedef T V __attribute__((ext_vector_type(N), aligned(sizeof(T))));
    u32x4 raw[kPasses];
    int c, r;

    __device__ __forceinline__ void load(const T* x, int64_t ld, int rows, int cols) {
        c = threadIdx.x % L * N, r = threadIdx.x / L;
#pragma unroll
        for (int p = 0; p < kPasses; ++p) {
            raw[p] = u32x4{0, 0, 0, 0};
            if (p * kRows + r < rows && c < cols)
                raw[p] = __builtin_bit_cast(u32x4, __builtin_nontemporal_load(reinterpret_cast<const V*>(x + (p * kRows + r) * ld + c)));
        }
    }
    __device__ __forceinline__ void get(int p, float (&v)[N]) const {
        const Pack<T, N> t = __builtin_bit_cast(Pack<T, N>, raw[p]);
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = (float)t.v[i];
    }
    // Nothing formed from the values is kept from here on (the compiler would keep them all as f32).
    __device__ __forceinline__ void forget() {
#pragma unroll
        for (int p = 0; p < kPasses; ++p) asm volatile("" : "+v"(raw[p]));
    }
};

// The codes of a tile in LDS, rows of 128 bytes and a bank's gap, and from there the columns.
constexpr int kTileWords = kFp8Block / 4 + 1;
struct TileLds {
    uint32_t code[kFp8Block * kTileWords];
    uint32_t top[4][kFp8Block];
};

// 4 x 4 bytes: byte i of word j to byte j of word i.
__device__ __forceinline__ void transpose4(uint32_t (&w)[4]) {
    const uint32_t a = __builtin_amdgcn_perm(w[1], w[0], 0x05010400), b = __builtin_amdgcn_perm(w[1], w[0], 0x07030602);
    const uint32_t c = __builtin_amdgcn_perm(w[3], w[2], 0x05010400), d = __builtin_amdgcn_perm(w[3], w[2], 0x07030602);
    w[0] = __builtin_amdgcn_perm(c, a, 0x05040100), w[1] = __builtin_amdgcn_perm(c, a, 0x07060302);
    w[2] = __builtin_amdgcn_perm(d, b, 0x05040100), w[3] = __builtin_amdgcn_perm(d, b, 0x07060302);
}

// Column c of the tile to qt + c * ld, `rows` (a multiple of 16) bytes: a thread takes 4 columns by
// 16 rows, 8 neighbouring threads write a column's 128 bytes.
__device__ __forceinline__ void store_columns(const TileLds& lds, uint8_t* qt, int64_t ld, int rows, int cols) {
    const int r0 = threadIdx.x % 8 * 16, c0 = threadIdx.x / 8 * 4;
    if (r0 >= rows || c0 >= cols) return;
    u32x4 out[4];
#pragma unroll
    for (int b = 0; b < 4; ++b) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = lds.code[(r0 + 4 * b + i) * kTileWords + c0 / 4];
        transpose4(w);
#pragma unroll
        for (int i = 0; i < 4; ++i) out[i][b] = w[i];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (c0 + i < cols) *reinterpret_cast<u32x4*>(qt + (c0 + i) * ld + r0) = out[i];
}

template <typename T>
__global__ __launch_bounds__(kThreads) void quantize_matrix_kernel(Fp8MatrixArgs a, int tiles_r, int tiles_c) {
    __shared__ TileLds lds;
    typedef TileIn<T> In;
    const int tid = threadIdx.x;
    const uint32_t per = (uint32_t)tiles_r * tiles_c, mat = blockIdx.x / per, at = blockIdx.x % per;
    const int tr = at / tiles_c, tc = at % tiles_c;
    const int rows = min(kFp8Block, a.rows - tr * kFp8Block), cols = min(kFp8Block, a.cols - tc * kFp8Block);
    In in;
    in.load((const T*)a.x + mat * a.x_stride + (int64_t)tr * kFp8Block * a.ld + tc * kFp8Block, a.ld, rows, cols);
    uint32_t top = 0;
#pragma unroll
    for (int p = 0; p < In::kPasses; ++p) {
        float v[In::N];
        in.get(p, v);
        top = max(top, top_bits(v));
    }
    in.forget();
    top = wave_umax(top);
    if (tid % 64 == 0) lds.top[0][tid / 64] = top;
    __syncthreads();
    top = max(max(lds.top[0][0], lds.top[0][1]), max(lds.top[0][2], lds.top[0][3]));
    const int code = fp8_scale_code(top);
    const float inv = fp8_scale_inverse(code);
    uint8_t* q = a.q ? a.q + mat * a.q_stride + (int64_t)tr * kFp8Block * a.cols + tc * kFp8Block : nullptr;
#pragma unroll
    for (int p = 0; p < In::kPasses; ++p) {
        const int r = p * In::kRows + in.r;
        uint32_t w[In::N / 4];
        float v[In::N];
        in.get(p, v);
#pragma unroll
        for (int i = 0; i < In::N / 4; ++i) w[i] = fp8_codes4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3], inv);
        if (q && r < rows && in.c < cols) {
            Pack<uint32_t, In::N / 4> o;
#pragma unroll
            for (int i = 0; i < In::N / 4; ++i) o.v[i] = w[i];
            *reinterpret_cast<Pack<uint32_t, In::N / 4>*>(q + (int64_t)r * a.cols + in.c) = o;
        }
        if (a.qt) {
#pragma unroll
            for (int i = 0; i < In::N / 4; ++i) lds.code[r * kTileWords + in.c / 4 + i] = w[i];
        }
    }
    if (tid == 0 && a.q) *(float*)((uint8_t*)a.s + mat * a.s_stride + 4 * ((int64_t)tr * tiles_c + tc)) = fp8_scale_value(code);
    if (!a.qt) return;
    if (tid == 0) *(float*)((uint8_t*)a.st + mat * a.st_stride + 4 * ((int64_t)tc * tiles_r + tr)) = fp8_scale_value(code);
    __syncthreads();
    store_columns(lds, a.qt + mat * a.qt_stride + (int64_t)tc * kFp8Block * a.rows + tr * kFp8Block, a.rows, rows, cols);
}

// ------------------------------------------------------------ columns, by expert
// Block b of 128 rows of an expert, in the experts' order: its first row and how many rows it has
// (0: there is no such block). A wave finds it by itself.
__device__ __forceinline__ void rows_block(const int32_t* offsets, int E, int R, uint32_t b, int* m0, int* rows) {
    *rows = 0;
    *m0 = 0;
    if (offsets == nullptr) {
        if ((int64_t)b * kFp8Block < R) *m0 = b * kFp8Block, *rows = min(kFp8Block, R - *m0);
        return;
    }
    const int lane = threadIdx.x & 63, per = (E + 63) / 64;
    uint32_t mine = 0;
    for (int i = 0; i < per; ++i) {
        const int e = min(lane * per + i, E);
        const int lo = min(max(offsets[e], 0), R), hi = min(max(offsets[min(e + 1, E)], lo), R);
        mine += (uint32_t)fp8_blocks(hi - lo);
    }
    uint32_t incl = mine;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const uint32_t v = __shfl_up(incl, o);
        if (lane >= o) incl += v;
    }
    const unsigned long long has = __ballot(b >= incl - mine && b < incl);
    if (has == 0) return;
    const int owner = __ffsll(has) - 1;
    int at = 0, n = 0;
    if (lane == owner) {
        uint32_t rest = b - (incl - mine);
        for (int i = 0; i < per && n == 0; ++i) {
            const int e = min(lane * per + i, E);
            const int lo = min(max(offsets[e], 0), R), hi = min(max(offsets[min(e + 1, E)], lo), R);
            const uint32_t nb = (uint32_t)fp8_blocks(hi - lo);
            if (rest < nb) at = lo + (int)rest * kFp8Block, n = min(kFp8Block, hi - at);
            else rest -= nb;
        }
    }
    *m0 = __builtin_amdgcn_readlane(at, owner);
    *rows = __builtin_amdgcn_readlane(n, owner);
}

template <typename T>
__global__ __launch_bounds__(kThreads) void quantize_columns_kernel(Fp8ColumnArgs a, int tiles_c) {
    __shared__ TileLds lds;
    typedef TileIn<T> In;
    constexpr int N = In::N, W = N / 4;
    const int tid = threadIdx.x;
    const uint32_t b = blockIdx.x / (uint32_t)tiles_c;
    const int tc = blockIdx.x % (uint32_t)tiles_c, cols = min(kFp8Block, a.cols - tc * kFp8Block);
    int m0, rows;
    rows_block(a.offsets, a.E, a.rows, b, &m0, &rows);
    if (rows == 0) return;
    In in;
    in.load((const T*)a.x + (int64_t)m0 * a.ld + tc * kFp8Block, a.ld, rows, cols);
    // a column's largest: over the thread's rows, over the lanes of its columns, over the waves
    uint32_t top[N];
#pragma unroll
    for (int i = 0; i < N; ++i) top[i] = 0;
#pragma unroll
    for (int p = 0; p < In::kPasses; ++p) {
        float v[N];
        in.get(p, v);
#pragma unroll
        for (int i = 0; i < N; ++i) top[i] = max(top[i], abs_bits(v[i]));
    }
    in.forget();
#pragma unroll
    for (int i = 0; i < N; ++i) {
        if constexpr (In::L == 16) top[i] = umax_step<16>(top[i]);
        top[i] = umax_step<32>(top[i]);
    }
    if ((tid & 63) < In::L) {
#pragma unroll
        for (int i = 0; i < N; ++i) lds.top[tid >> 6][in.c + i] = top[i];
    }
    __syncthreads();
    float inv[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int c = in.c + i;
        const int code = fp8_scale_code(max(max(lds.top[0][c], lds.top[1][c]), max(lds.top[2][c], lds.top[3][c])));
        inv[i] = fp8_scale_inverse(code);
        if (in.r == 0 && c < cols) a.st[(int64_t)b * a.cols + tc * kFp8Block + c] = (uint8_t)code;
    }
    const int SB = (int)fp8_blocks(a.cols);
#pragma unroll
    for (int p = 0; p < In::kPasses; ++p) {
        const int r = p * In::kRows + in.r;
        float x[N];
        in.get(p, x);
#pragma unroll
        for (int i = 0; i < W; ++i) {
            float v[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)                  // (0: a column with an infinity or a NaN)
                v[j] = inv[4 * i + j] == 0.f ? 0.f : x[4 * i + j] * inv[4 * i + j];
            lds.code[r * kTileWords + in.c / 4 + i] = fp8_codes4(v[0], v[1], v[2], v[3], 1.f);
        }
        if (a.q) {
            const int code = fp8_scale_code(lanes_umax<In::L>(top_bits(x)));
            if (r < rows && in.c < cols)
                store_codes(a.q + (int64_t)(m0 + r) * a.cols + tc * kFp8Block + in.c, x, fp8_scale_inverse(code));
            if (r < rows && tid % In::L == 0) a.s[(int64_t)(m0 + r) * SB + tc] = fp8_scale_value(code);
        }
    }
    __syncthreads();
    store_columns(lds, a.qt + ((int64_t)b * a.cols + tc * kFp8Block) * kFp8Block, kFp8Block, kFp8Block, cols);
}

coli_status check_grid(int64_t grid, const char* what) {
    if (grid > kMaxGrid) return fail(COLI_EUNSUPPORTED, std::string(what) + ": too many values for one launch");
    return COLI_OK;
}

}  // namespace

coli_status launch_quantize_fp8(const void* x, int32_t dtype, int64_t rows, int64_t cols, int64_t ld,
                                uint8_t* q, float* s, hipStream_t stream, const int32_t* offsets, int32_t E) {
    if (rows == 0) return COLI_OK;
    return with_elem(dtype, [&](auto e) -> coli_status {
        using T = decltype(e);
        UnitMap m;
        m.per_row = fp8_blocks(cols) * kLanes<T>;
        m.units = rows * m.per_row;
        m.ld = ld;
        m.cols = (int32_t)cols;
        const int64_t grid = (m.units + kThreads - 1) / kThreads;
        if (coli_status st = check_grid(grid, "quantize_fp8")) return st;
        if (offsets) launch(quantize_rows_kernel<T, true>, dim3((uint32_t)grid), dim3(kThreads), 0, stream, (const T*)x, m, q, s, offsets, E);
        else launch(quantize_rows_kernel<T, false>, dim3((uint32_t)grid), dim3(kThreads), 0, stream, (const T*)x, m, q, s, offsets, E);
        COLI_CHECK_LAUNCH("quantize_fp8 kernel launch");
        return COLI_OK;
    });
}

coli_status launch_dispatch_fp8(const void* x, int32_t dtype, int32_t T, int32_t k, int32_t H, int64_t ld_x,
                                const int32_t* inv, uint8_t* q, float* s, hipStream_t stream) {
    if (T == 0) return COLI_OK;
    return with_elem(dtype, [&](auto e) -> coli_status {
        using V = decltype(e);
        const int64_t units = fp8_blocks(H) * kLanes<V>, tiles = (units + kThreads - 1) / kThreads;
        if (coli_status st = check_grid(T * tiles, "dispatch_fp8")) return st;
        launch(dispatch_fp8_kernel<V>, dim3((uint32_t)(T * tiles)), dim3(kThreads), 0, stream, (const V*)x, ld_x, k, H,
               (int64_t)T * k, (int)tiles, inv, q, s);
        COLI_CHECK_LAUNCH("dispatch_fp8 kernel launch");
        return COLI_OK;
    });
}

coli_status launch_dequantize_fp8(const uint8_t* q, const float* s, int64_t rows, int64_t cols,
                                  int32_t block_rows, void* x, int32_t dtype, int64_t ld,
                                  hipStream_t stream, int32_t count, int64_t q_stride, int64_t s_stride, int64_t x_stride) {
    if (rows == 0 || count == 0) return COLI_OK;
    return with_elem(dtype, [&](auto e) -> coli_status {
        using T = decltype(e);
        constexpr int U = 2;
        UnitMap m;
        m.per_row = cols / kVec<T>;
        m.units = rows * m.per_row;
        m.ld = ld;
        m.cols = (int32_t)cols;
        const int64_t per = (m.units + kThreads * U - 1) / (kThreads * U);
        if (coli_status st = check_grid(per > kMaxGrid ? per : per * count, "dequantize_fp8")) return st;
        launch(dequantize_kernel<T, U>, dim3((uint32_t)(per * count)), dim3(kThreads), 0, stream, q, s, m, (int)block_rows, (T*)x,
               (uint32_t)per, q_stride, s_stride, x_stride);
        COLI_CHECK_LAUNCH("dequantize_fp8 kernel launch");
        return COLI_OK;
    });
}

coli_status launch_quantize_fp8_matrix(const Fp8MatrixArgs& a, int32_t dtype, int32_t count, hipStream_t stream) {
    if (count == 0 || a.rows == 0) return COLI_OK;
    const int64_t tr = fp8_blocks(a.rows), tc = fp8_blocks(a.cols);
    if (tr * tc > kMaxGrid / count) return fail(COLI_EUNSUPPORTED, "quantize_fp8_matrix: too many values for one launch");
    return with_elem(dtype, [&](auto e) -> coli_status {
        using T = decltype(e);
        launch(quantize_matrix_kernel<T>, dim3((uint32_t)(tr * tc * count)), dim3(kThreads), 0, stream, a, (int)tr, (int)tc);
        COLI_CHECK_LAUNCH("quantize_fp8_matrix kernel launch");
        return COLI_OK;
    });
}

coli_status launch_quantize_fp8_columns(const Fp8ColumnArgs& a, int32_t dtype, hipStream_t stream) {
    if (a.rows == 0) return COLI_OK;
    const int64_t tc = fp8_blocks(a.cols);
    const int64_t most = a.offsets ? (a.rows + (int64_t)(kFp8Block - 1) * std::min(a.E, a.rows)) / kFp8Block : fp8_blocks(a.rows);
    const int64_t grid = tc * std::min<int64_t>(a.blocks, most);
    if (coli_status st = check_grid(grid, "quantize_fp8_columns")) return st;
    return with_elem(dtype, [&](auto e) -> coli_status {
        using T = decltype(e);
        launch(quantize_columns_kernel<T>, dim3((uint32_t)grid), dim3(kThreads), 0, stream, a, (int)tc);
        COLI_CHECK_LAUNCH("quantize_fp8_columns kernel launch");
        return COLI_OK;
    });
}

}  // namespace coli
