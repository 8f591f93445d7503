// Tokens to the experts' order and back.
//
// inv [T][k] holds each assignment's row in the experts' order (the inverse of
// the union's perm; anything outside [0, T*k) marks a slot without a row).
//   dispatch        rows[inv[t][j]] = x[t]
//   its gradient    dx[t] = sum_j g[inv[t][j]]
//   combine         y[t] = shared[t] + scale * sum_j w[t][j] rows[inv[t][j]]
//   its gradients   drows[inv[t][j]] = scale * w[t][j] * dy[t]
//                   dw[t][j] = scale * <dy[t], rows[inv[t][j]]>
// Every kernel works by token: x[t], dx[t], y[t] and dy[t] are touched once
// however many experts the token has, sums run in slot order in f32, and
// nothing is added atomically, so results do not depend on scheduling. All are
// bound by HBM (the k rows of every token, read or written once).
#include <algorithm>

#include "mxfp4.h"

namespace coli {
namespace {

constexpr int kThreads = 256;
// A launch holds fewer than 2^32 threads.
constexpr int64_t kMaxGrid = (int64_t(1) << 32) / kThreads - 1;

// 16 bytes of a row per thread.
template <typename T>
constexpr int kVec = 16 / (int)sizeof(T);

// The row of slot j, or -1.
__device__ __forceinline__ int64_t slot_row(const int32_t* inv, int64_t at, int64_t n) {
    const int32_t p = inv[at];
    return p >= 0 && p < n ? p : -1;
}

// The V columns from c on. FULL: all are below H, one access (wherever the row
// starts: see Pack); otherwise one by one, columns from H on as 0, loaded from
// the last column so that the loads need no branch and stay in flight together.
template <int V, bool FULL, typename T>
__device__ __forceinline__ void load_cols(const T* row, int c, int H, float (&v)[V]) {
    if constexpr (FULL) {
        load_f32<T, V>(row + c, v);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float f = (float)row[min(c + i, H - 1)];
            v[i] = c + i < H ? f : 0.f;
        }
    }
}

template <int V, bool FULL, typename T>
__device__ __forceinline__ void store_cols(T* row, int c, int H, const float (&v)[V]) {
    if constexpr (FULL) {
        store_f32<T, V>(row + c, v);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (c + i < H) row[c + i] = (T)v[i];
    }
}

// ------------------------------------------------------------ dispatch
// Workgroup (token, stretch of kThreads * kVec columns). T is any type of the
// element's size: the copy keeps every bit. The rows are stored past the caches:
// 16384 rows of 6144 bf16 43.7 us, 36.5 with it (5.8 TB/s and 6.2 with the tokens).
template <typename T>
__global__ __launch_bounds__(kThreads) void dispatch_kernel(const T* __restrict__ x, int64_t ld_x,
                                                            int k, int H, int64_t n, int tiles,
                                                            const int32_t* __restrict__ inv,
                                                            T* __restrict__ rows, int64_t ld_rows) {
    constexpr int V = kVec<T>;
    const int64_t t = blockIdx.x / (uint32_t)tiles;
    const int c = ((blockIdx.x % (uint32_t)tiles) * kThreads + threadIdx.x) * V;
    const T* src = x + t * ld_x;
    if (c + V <= H) {
        typedef T Vec __attribute__((ext_vector_type(V), aligned(sizeof(T))));
        const Vec v = *reinterpret_cast<const Vec*>(src + c);
        for (int j = 0; j < k; ++j) {
            const int64_t p = slot_row(inv, t * k + j, n);
            if (p >= 0) __builtin_nontemporal_store(v, reinterpret_cast<Vec*>(rows + p * ld_rows + c));
        }
    } else if (c < H) {
        T v[V];
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = src[min(c + i, H - 1)];
        for (int j = 0; j < k; ++j) {
            const int64_t p = slot_row(inv, t * k + j, n);
            if (p < 0) continue;
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (c + i < H) rows[p * ld_rows + c + i] = v[i];
        }
    }
}

// The same, quantised on the way: a token is read and converted once, its codes
// and scales go to all of its rows. A lane takes 8 columns, as in the
// quantiser.
template <typename T>
__global__ __launch_bounds__(kThreads) void dispatch_mxfp4_kernel(
    const T* __restrict__ x, int64_t ld_x, int k, int H, int64_t n, int tiles,
    const int32_t* __restrict__ inv, uint8_t* __restrict__ q, uint8_t* __restrict__ s) {
    const int64_t t = blockIdx.x / (uint32_t)tiles;
    const int unit = (blockIdx.x % (uint32_t)tiles) * kThreads + threadIdx.x;
    if (unit * 8 >= H) return;                    // whole quads: H is a multiple of 32
    float v[8];
    load_f32<T, 8>(x + t * ld_x + unit * 8, v);
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, abs_bits(v[i]));
    top = mx_quad_max(top);
    const int code = mx_scale_code(top);
    const uint32_t w = code == 255 ? 0u : mx_codes8(v, mx_scale_value(code));
    for (int j = 0; j < k; ++j) {
        const int64_t p = slot_row(inv, t * k + j, n);
        if (p < 0) continue;
        reinterpret_cast<uint32_t*>(q + p * (H / 2))[unit] = w;
        if ((threadIdx.x & 3) == 0) s[p * (H / kMxBlock) + (unit >> 2)] = (uint8_t)code;
    }
}

// ------------------------------------------------------------ sums over slots
// dx (w == nullptr: every weight 1, no scale) and combine. Slots are taken in
// groups of G whose rows are all loaded before the first is added; a slot
// without a row re-reads the token's first row (in cache by then) and adds
// nothing, so that the loads need no branch.
template <typename Tin, typename Tout, int G>
__global__ __launch_bounds__(kThreads) void gather_sum_kernel(
    const Tin* __restrict__ rows, int64_t ld_rows, int k, int H, int64_t n, int tiles,
    const int32_t* __restrict__ inv, const float* __restrict__ w, const Tout* shared,
    int64_t ld_shared, float scale, Tout* y, int64_t ld_y) {
    constexpr int V = kVec<Tin>;
    const int64_t t = blockIdx.x / (uint32_t)tiles;
    const int c = ((blockIdx.x % (uint32_t)tiles) * kThreads + threadIdx.x) * V;
    if (c >= H) return;
    int64_t first = -1;
    for (int j = 0; j < k && first < 0; ++j) first = slot_row(inv, t * k + j, n);
    auto sum = [&](auto full) {
        constexpr bool FULL = decltype(full)::value;
        float acc[V], sh[V];
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] = sh[i] = 0.f;
        if (shared) load_cols<V, FULL>(shared + t * ld_shared, c, H, sh);
        if (first >= 0) {
            for (int j0 = 0; j0 < k; j0 += G) {
                float v[G][V], wj[G];
                bool on[G];
#pragma unroll
                for (int j = 0; j < G; ++j) {
                    const int64_t p = j0 + j < k ? slot_row(inv, t * k + j0 + j, n) : -1;
                    on[j] = p >= 0;
                    wj[j] = on[j] && w ? w[t * k + j0 + j] : 1.f;
                    const Tin* src = rows + (on[j] ? p : first) * ld_rows;
                    if constexpr (FULL) load_f32_once<Tin, V>(src + c, v[j]);
                    else load_cols<V, FULL>(src, c, H, v[j]);
                }
#pragma unroll
                for (int j = 0; j < G; ++j)
#pragma unroll
                    for (int i = 0; i < V; ++i) acc[i] = on[j] ? fmaf(wj[j], v[j][i], acc[i]) : acc[i];
            }
        }
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] = fmaf(scale, acc[i], sh[i]);
        store_cols<V, FULL>(y + t * ld_y, c, H, acc);
    };
    if (c + V <= H) sum(std::true_type{});
    else sum(std::false_type{});
}

// ------------------------------------------------------------ combine backward
// Workgroup (token, group of up to G of its slots): one pass over H with the
// group's dot products in registers, then one reduction over the workgroup
// (lanes, then waves in order). Rows and their gradient go past the caches:
// forward and backward of 4096 tokens of 8 rows of 6144 bf16 278 us, 260 with it.
template <typename Td, typename Tr, int G>
__global__ __launch_bounds__(kThreads) void combine_bwd_kernel(
    const Td* __restrict__ dy, int64_t ld_dy, const Tr* __restrict__ rows, int64_t ld_rows, int k,
    int H, int64_t n, int groups, const int32_t* __restrict__ inv, const float* __restrict__ w,
    float scale, Tr* __restrict__ drows, int64_t ld_drows, float* __restrict__ dw) {
    constexpr int V = kVec<Tr>;
    __shared__ float part[kThreads / 64][G];
    const int64_t t = blockIdx.x / (uint32_t)groups;
    const int j0 = (blockIdx.x % (uint32_t)groups) * G;
    int64_t p[G];
    float wj[G], dot[G];
#pragma unroll
    for (int j = 0; j < G; ++j) {
        p[j] = j0 + j < k ? slot_row(inv, t * k + j0 + j, n) : -1;
        wj[j] = p[j] >= 0 ? scale * w[t * k + j0 + j] : 0.f;
        dot[j] = 0.f;
    }
    auto columns = [&](auto full, int c) {
        constexpr bool FULL = decltype(full)::value;
        float g[V];
        load_cols<V, FULL>(dy + t * ld_dy, c, H, g);
#pragma unroll
        for (int j = 0; j < G; ++j) {
            if (p[j] < 0) continue;               // uniform
            float v[V], out[V];
            if constexpr (FULL) load_f32_once<Tr, V>(rows + p[j] * ld_rows + c, v);
            else load_cols<V, FULL>(rows + p[j] * ld_rows, c, H, v);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                dot[j] = fmaf(g[i], v[i], dot[j]);
                out[i] = wj[j] * g[i];
            }
            if constexpr (FULL) store_f32_once<Tr, V>(drows + p[j] * ld_drows + c, out);
            else store_cols<V, FULL>(drows + p[j] * ld_drows, c, H, out);
        }
    };
    for (int c = threadIdx.x * V; c < H; c += kThreads * V) {
        if (c + V <= H) columns(std::true_type{}, c);
        else columns(std::false_type{}, c);
    }
#pragma unroll
    for (int j = 0; j < G; ++j) {
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) dot[j] += __shfl_xor(dot[j], o);
        if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6][j] = dot[j];
    }
    __syncthreads();
    const int j = threadIdx.x;
    if (j < G && j0 + j < k) {
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < kThreads / 64; ++i) sum += part[i][j];
        dw[t * k + j0 + j] = slot_row(inv, t * k + j0 + j, n) >= 0 ? scale * sum : 0.f;
    }
}

// Workgroups of `per` for every token, or an error where a launch cannot hold
// them.
coli_status grid_of(int64_t T, int64_t per, uint32_t* grid) {
    if (T * per > kMaxGrid) return fail(COLI_EUNSUPPORTED, "permute: more than 2^32 threads");
    *grid = (uint32_t)(T * per);
    return COLI_OK;
}

int tiles_of(int H, int vec) { return (H + kThreads * vec - 1) / (kThreads * vec); }

}  // namespace

coli_status launch_dispatch(const void* x, int32_t dtype, int32_t T, int32_t k, int32_t H,
                            int64_t ld_x, const int32_t* inv, void* rows, int64_t ld_rows,
                            hipStream_t stream) {
    const int64_t n = (int64_t)T * k;
    const int tiles = tiles_of(H, 16 / elem_bytes(dtype));
    uint32_t grid;
    if (coli_status st = grid_of(T, tiles, &grid)) return st;
    if (elem_bytes(dtype) == 4)
        launch(dispatch_kernel<uint32_t>, dim3(grid), dim3(kThreads), 0, stream, (const uint32_t*)x,
               ld_x, k, H, n, tiles, inv, (uint32_t*)rows, ld_rows);
    else
        launch(dispatch_kernel<uint16_t>, dim3(grid), dim3(kThreads), 0, stream, (const uint16_t*)x,
               ld_x, k, H, n, tiles, inv, (uint16_t*)rows, ld_rows);
    COLI_CHECK_LAUNCH("dispatch kernel launch");
    return COLI_OK;
}

coli_status launch_dispatch_mxfp4(const void* x, int32_t dtype, int32_t T, int32_t k, int32_t H,
                                  int64_t ld_x, const int32_t* inv, uint8_t* q, uint8_t* s,
                                  hipStream_t stream) {
    const int64_t n = (int64_t)T * k;
    const int tiles = tiles_of(H, 8);
    uint32_t grid;
    if (coli_status st = grid_of(T, tiles, &grid)) return st;
    return with_elem(dtype, [&](auto e) -> coli_status {
        using Tx = decltype(e);
        launch(dispatch_mxfp4_kernel<Tx>, dim3(grid), dim3(kThreads), 0, stream, (const Tx*)x, ld_x,
               k, H, n, tiles, inv, q, s);
        COLI_CHECK_LAUNCH("dispatch_mxfp4 kernel launch");
        return COLI_OK;
    });
}

static coli_status gather_sum(const void* rows, int32_t rows_dtype, int64_t ld_rows, int32_t T,
                              int32_t k, int32_t H, const int32_t* inv, const float* w,
                              const void* shared, int64_t ld_shared, float scale, void* y,
                              int32_t dtype, int64_t ld_y, hipStream_t stream) {
    const int64_t n = (int64_t)T * k;
    const int tiles = tiles_of(H, 16 / elem_bytes(rows_dtype));
    uint32_t grid;
    if (coli_status st = grid_of(T, tiles, &grid)) return st;
    return with_elem(rows_dtype, [&](auto e) -> coli_status {
        using Tin = decltype(e);
        return with_elem(dtype, [&](auto f) -> coli_status {
            using Tout = decltype(f);
            auto go = [&](auto kernel) {
                launch(kernel, dim3(grid), dim3(kThreads), 0, stream, (const Tin*)rows, ld_rows, k, H,
                       n, tiles, inv, w, (const Tout*)shared, ld_shared, scale, (Tout*)y, ld_y);
            };
            k > 4 ? go(gather_sum_kernel<Tin, Tout, 8>) : go(gather_sum_kernel<Tin, Tout, 4>);
            COLI_CHECK_LAUNCH("gather_sum kernel launch");
            return COLI_OK;
        });
    });
}

coli_status launch_dispatch_bwd(const void* g, int32_t g_dtype, int64_t ld_g, int32_t T, int32_t k,
                                int32_t H, const int32_t* inv, void* dx, int32_t dtype,
                                int64_t ld_dx, hipStream_t stream) {
    return gather_sum(g, g_dtype, ld_g, T, k, H, inv, nullptr, nullptr, 0, 1.f, dx, dtype, ld_dx, stream);
}

coli_status launch_combine_rows(const void* rows, int32_t rows_dtype, int64_t ld_rows, int32_t T,
                                int32_t k, int32_t H, const int32_t* inv, const float* w,
                                const void* shared, int64_t ld_shared, float scale, void* y,
                                int32_t dtype, int64_t ld_y, hipStream_t stream) {
    return gather_sum(rows, rows_dtype, ld_rows, T, k, H, inv, w, shared, ld_shared, scale, y, dtype,
                      ld_y, stream);
}

coli_status launch_combine_bwd(const void* dy, int32_t dy_dtype, int64_t ld_dy, const void* rows,
                               int32_t rows_dtype, int64_t ld_rows, int32_t T, int32_t k, int32_t H,
                               const int32_t* inv, const float* w, float scale, void* drows,
                               int64_t ld_drows, float* dw, hipStream_t stream) {
    const int64_t n = (int64_t)T * k;
    constexpr int G = 4;
    const int groups = (k + G - 1) / G;
    uint32_t grid;
    if (coli_status st = grid_of(T, groups, &grid)) return st;
    return with_elem(dy_dtype, [&](auto e) -> coli_status {
        using Td = decltype(e);
        return with_elem(rows_dtype, [&](auto f) -> coli_status {
            using Tr = decltype(f);
            launch(combine_bwd_kernel<Td, Tr, G>, dim3(grid), dim3(kThreads), 0, stream,
                   (const Td*)dy, ld_dy, (const Tr*)rows, ld_rows, k, H, n, groups, inv, w, scale,
                   (Tr*)drows, ld_drows, dw);
            COLI_CHECK_LAUNCH("combine_bwd kernel launch");
            return COLI_OK;
        });
    });
}

}  // namespace coli
