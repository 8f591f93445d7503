// Internal: what the grouped products on the matrix instructions share: operand loads, loads
// straight into LDS, and the results' stores.
#pragma once

#include "mxfp4.h"

namespace coli {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kFrag = 16;                    // rows of one operand of the instruction

constexpr uint32_t kCus = 256;

struct __attribute__((packed, aligned(1))) Bytes16 {
    uint32_t w[4];
};
// Blob pointers come from a table in memory: without the address space their
// loads would be generic ones, which also count as LDS accesses.
typedef __attribute__((address_space(1))) const uint8_t global_u8;
typedef __attribute__((address_space(1))) const Bytes16 global_bytes16;

__device__ __forceinline__ u32x4 load16(const uint8_t* p) { return *(global_u32x4*)(p); }
__device__ __forceinline__ uint32_t load1(const uint8_t* p) { return *(global_u8*)(p); }

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
template <typename T, typename Args>
__device__ __forceinline__ void store4(const Args& a, int m, int n0, int N, const f32x4& v) {
    T* p = (T*)a.y + (int64_t)m * a.ld + n0;
    const float r[4] = {v.x, v.y, v.z, v.w};
    if (n0 + 4 <= N) {
        store_f32<T, 4>(p, r);
    } else {
        for (int i = 0; i < 4 && n0 + i < N; ++i) p[i] = (T)r[i];
    }
}

// The four lanes of a row, g = lane / 16, hold quarter g of two 16-byte halves (x:
// the first): afterwards lane 0 holds quarters 0 and 1 of the first half, lane 1
// its quarters 2 and 3, lanes 2 and 3 the same of the second.
__device__ __forceinline__ void swap_quarters(uint32_t& x, uint32_t& y) {
    const auto a = __builtin_amdgcn_permlane32_swap(x, y, false, false);   // x of lanes 2, 3 with y of 0, 1
    const auto b = __builtin_amdgcn_permlane16_swap(a[0], a[1], false, false);   // x of 1, 3 with y of 0, 2
    x = b[0], y = b[1];
}

__device__ __forceinline__ void swap_quarters_back(uint32_t& x, uint32_t& y) {
    const auto a = __builtin_amdgcn_permlane16_swap(x, y, false, false);
    const auto b = __builtin_amdgcn_permlane32_swap(a[0], a[1], false, false);
    x = b[0], y = b[1];
}

// Outputs n0 .. n0 + 31 (those below N) of row `m`, of which this lane holds n0 + 4 g
// .. + 3 (lo) and n0 + 16 + 4 g .. + 3 (hi): for a 16-bit type one store of 16 bytes a
// lane, 64 neighbouring bytes a row. Stores hold up the loads behind them, all of
// which a wave counts in one order: half as many take the dense product of 8191 x
// 8192 x 8192 from 302 to 283 us, 16384 rows of 256 experts (K 2048, N 6144) from
// 398 to 391. (For SwiGLU, whose stores the activations space out, it is no gain:
// 648 with store4, 667 with this; its MXFP4 codes 696 and 707.)
template <typename T, typename Args>
__device__ __forceinline__ void store32(const Args& a, int m, int n0, int N, bool live,
                                        const f32x4& lo, const f32x4& hi) {
    const int g = (threadIdx.x & 63) >> 4;
    if (sizeof(T) == 2 && n0 + 32 <= N) {         // uniform
        union {
            T v[4];
            uint32_t w[2];
        } x, y;
#pragma unroll
        for (int i = 0; i < 4; ++i) x.v[i] = (T)lo[i], y.v[i] = (T)hi[i];
        swap_quarters(x.w[0], y.w[0]);
        swap_quarters(x.w[1], y.w[1]);
        if (!live) return;
        Pack<T, 8> r;
#pragma unroll
        for (int i = 0; i < 4; ++i) r.v[i] = x.v[i], r.v[4 + i] = y.v[i];
        *reinterpret_cast<Pack<T, 8>*>((T*)a.y + (int64_t)m * a.ld + n0 + 8 * g) = r;
    } else if (live) {
        store4<T>(a, m, n0 + 4 * g, N, lo);
        store4<T>(a, m, n0 + kFrag + 4 * g, N, hi);
    }
}

// x where a lane's number within 16 is below 8, y of the lane 8 further down where it is not (EVEN); or x of the
// lane 8 further up where it is below, y where it is not.
template <bool EVEN>
__device__ __forceinline__ uint32_t merge_halves(uint32_t x, uint32_t y) {
    // row_ror:8 into the upper, or the lower, two banks of four lanes
    if constexpr (EVEN) return (uint32_t)__builtin_amdgcn_update_dpp((int)x, (int)y, 0x128, 0xf, 0xc, false);
    else return (uint32_t)__builtin_amdgcn_update_dpp((int)y, (int)x, 0x128, 0xf, 0x3, false);
}

// Four fragments of results, columns 0 .. 63 of a row behind `out` (its row 0 and first column), in whole cache
// lines: of a fragment's 16 rows, a store takes 8 rows by 128 bytes, so that no line is written in parts. A lane
// holds row lane % 16; rows from `rows` on are left out. (3.2 GB of f32 by 16 rows of 64 bytes a store took 696 us,
// by whole lines 624.) They go past the caches, which hold the operands (gradients of 64 experts' 2048 x 6144
// matrices, 256 rows each: 1136 us through them, 828 past them; in bf16 646 and 417). Two stores for a 16-bit type,
// four for f32.
template <typename T>
__device__ __forceinline__ void store64(T* out, int64_t ld, int rows, const f32x4& v0, const f32x4& v1, const f32x4& v2,
                                        const f32x4& v3) {
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4, row = r & 7;
    if constexpr (sizeof(T) == 2) {
        union Words {
            T v[4];
            uint32_t w[2];
        } x[4];
        const f32x4* v[4] = {&v0, &v1, &v2, &v3};
#pragma unroll
        for (int f = 0; f < 4; ++f)
#pragma unroll
            for (int i = 0; i < 4; ++i) x[f].v[i] = (T)(*v[f])[i];
#pragma unroll
        for (int f = 0; f < 4; f += 2)
#pragma unroll
            for (int i = 0; i < 2; ++i) swap_quarters(x[f].w[i], x[f + 1].w[i]);
        Pack<uint32_t, 4> lo, hi;            // columns 8 g of the first 32, of the second
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t a = x[i / 2].w[i % 2], b = x[2 + i / 2].w[i % 2];
            lo.v[i] = merge_halves<true>(a, b);
            hi.v[i] = merge_halves<false>(a, b);
        }
        typedef Pack<T, 8> P;
        T* p = out + row * ld + (r >= 8 ? 32 : 0) + 8 * g;
        typedef uint32_t V __attribute__((ext_vector_type(4), aligned(2)));
        if (row < rows) __builtin_nontemporal_store(__builtin_bit_cast(V, lo), reinterpret_cast<V*>(p));
        if (row + 8 < rows) __builtin_nontemporal_store(__builtin_bit_cast(V, hi), reinterpret_cast<V*>(p + 8 * ld));
    } else {
        const f32x4* v[4] = {&v0, &v1, &v2, &v3};
        T* p = out + row * ld + (r >= 8 ? 16 : 0) + 4 * g;
#pragma unroll
        for (int f = 0; f < 4; f += 2) {
            float lo[4], hi[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t a = __float_as_uint((*v[f])[i]), b = __float_as_uint((*v[f + 1])[i]);
                lo[i] = __uint_as_float(merge_halves<true>(a, b));
                hi[i] = __uint_as_float(merge_halves<false>(a, b));
            }
            if (row < rows) store_f32_once<T, 4>(p + 16 * f, lo);
            if (row + 8 < rows) store_f32_once<T, 4>(p + 16 * f + 8 * ld, hi);
        }
    }
}

// What store64 would replace: loaded the same way, and added to the fragments (merge_halves is its own inverse).
template <typename T>
struct Old64 {
    typedef uint32_t V __attribute__((ext_vector_type(4), aligned(2)));
    V v[sizeof(T)];

    __device__ __forceinline__ void load(const T* out, int64_t ld, int rows) {
        constexpr int kStep = 16 / sizeof(T);        // of a lane, and columns of a store's half / 4
        const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4, row = r & 7;
        const T* p = out + row * ld + (r >= 8 ? 4 * kStep : 0) + kStep * g;
#pragma unroll
        for (int x = 0; x < (int)sizeof(T); x += 2) {
            v[x] = V{0, 0, 0, 0};
            v[x + 1] = V{0, 0, 0, 0};
            if (row < rows) v[x] = __builtin_nontemporal_load(reinterpret_cast<const V*>(p + 16 * x));
            if (row + 8 < rows) v[x + 1] = __builtin_nontemporal_load(reinterpret_cast<const V*>(p + 16 * x + 8 * ld));
        }
    }

    __device__ __forceinline__ void add_to(f32x4 (&acc)[4]) const {
        if constexpr (sizeof(T) == 2) {
            union Words {
                T v[4];
                uint32_t w[2];
            } x[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[i / 2].w[i % 2] = merge_halves<true>(v[0][i], v[1][i]);
                x[2 + i / 2].w[i % 2] = merge_halves<false>(v[0][i], v[1][i]);
            }
#pragma unroll
            for (int f = 0; f < 4; f += 2)
#pragma unroll
                for (int i = 0; i < 2; ++i) swap_quarters_back(x[f].w[i], x[f + 1].w[i]);
#pragma unroll
            for (int f = 0; f < 4; ++f)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[f][i] += (float)x[f].v[i];
        } else {
#pragma unroll
            for (int f = 0; f < 4; f += 2)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    acc[f][i] += __uint_as_float(merge_halves<true>(v[f][i], v[f + 1][i]));
                    acc[f + 1][i] += __uint_as_float(merge_halves<false>(v[f][i], v[f + 1][i]));
                }
        }
    }
};

// Position of 16-byte unit b of row r in an LDS chunk of U units a row: the units
// of a row are permuted by its number, so that the rows that a load reads at one
// column fall into different banks.
template <int U>
__device__ __forceinline__ int lds_unit(int r, int b) { return r * U + (b ^ (r & (U - 1))); }

typedef __attribute__((address_space(1))) const void global_void;
typedef __attribute__((address_space(3))) void lds_void;

// 16 bytes a lane, from p (per lane) to 64 consecutive units at dst (uniform).
__device__ __forceinline__ void load_to_lds(const uint8_t* p, u32x4* dst) {
    __builtin_amdgcn_global_load_lds((global_void*)p, (lds_void*)dst, 16, 0, 0);
}

// Waits until at most N of this wave's vector memory operations are in flight,
// and for all of its LDS operations. One instruction that no memory access
// crosses in either direction: the count says which loads are done only if they
// were issued in program order. (Stores of results count too: with them in
// flight the wait is longer than it has to be, never shorter.)
template <int N>
__device__ __forceinline__ void wait_loads() {
    static_assert(N < 64, "vmcnt has 6 bits");
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(N) : "memory");
}

// The same with the stores of up to `tiles` (0, 1 or 2) tiles, STORES each, allowed to be in flight besides: they
// were issued behind the loads that are waited for. (Fewer than were issued only make the wait longer.)
template <int N, int STORES>
__device__ __forceinline__ void wait_behind_stores(int tiles) {
    static_assert(N + STORES < 64, "vmcnt has 6 bits");
    if (tiles == 0) wait_loads<N>();
    else if (tiles == 1) wait_loads<N + STORES>();
    else wait_loads<(N + 2 * STORES < 64 ? N + 2 * STORES : N + STORES)>();
}

}  // namespace coli
