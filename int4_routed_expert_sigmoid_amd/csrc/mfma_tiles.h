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

}  // namespace coli
