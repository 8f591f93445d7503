// Internal: the work units of a grouped product (rows sorted by expert, a matrix per
// expert), shared by the MXFP4 and FP8 products.
#pragma once

#include <algorithm>

#include "common.h"

namespace coli {

constexpr int kXcds = 8;
constexpr int kMaxExperts = 1024;
constexpr uint32_t kBlockM = 8;

struct RowGroups {
    const int32_t* offsets;      // [E + 1], or nullptr: every row belongs to matrix 0
    const void* const* table;    // [E] blobs
    int32_t rows, E;
};

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
__device__ __forceinline__ bool find_unit(const RowGroups& a, int NT, Unit* out) {
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

// The first unit of every expert into first[0 .. E - 1], and the number of units,
// for a workgroup of THREADS.
template <int BM, int THREADS>
__device__ __forceinline__ uint32_t scan_units(const RowGroups& a, int NT, uint32_t* first, uint32_t* scratch) {
    constexpr int kPer = kMaxExperts / THREADS;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    uint32_t n[kPer], sum = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int e = tid * kPer + i;
        n[i] = 0;
        if (a.offsets == nullptr) {
            n[i] = e == 0 ? (uint32_t)(a.rows + BM - 1) / BM * NT : 0;
        } else if (e < a.E) {
            const int lo = min(max(a.offsets[e], 0), a.rows), hi = min(max(a.offsets[e + 1], lo), a.rows);
            n[i] = (uint32_t)(hi - lo + BM - 1) / BM * NT;
        }
        sum += n[i];
    }
    uint32_t incl = sum;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const uint32_t v = __shfl_up(incl, o);
        if (lane >= o) incl += v;
    }
    if (lane == 63) scratch[wave] = incl;
    __syncthreads();
    uint32_t at = incl - sum, total = 0;
    for (int w = 0; w < THREADS / 64; ++w) {
        at += w < wave ? scratch[w] : 0;
        total += scratch[w];
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        if (tid * kPer + i < a.E) first[tid * kPer + i] = at;
        at += n[i];
    }
    __syncthreads();
    return __builtin_amdgcn_readfirstlane(total);
}

struct LineUnit {
    const uint8_t* blob;
    int m0, rows, nt;                        // rows 0: no unit
};

typedef __attribute__((address_space(4))) const int32_t const_i32;
typedef __attribute__((address_space(4))) const uint64_t const_u64;

// Unit w from the table of first units: a search in LDS, and scalar loads of the
// expert's offsets and blob, which leave the vector loads in flight alone.
template <int BM>
__device__ __forceinline__ LineUnit line_unit(const RowGroups& a, int NT, const uint32_t* first, uint32_t w, bool live) {
    LineUnit u = {(const uint8_t*)((const_u64*)a.table)[0], 0, 0, 0};
    const int lane = threadIdx.x & 63;
    int e = -1;
    for (int b = 0; b < a.E; b += 64) e += __popcll(__ballot(b + lane < a.E && first[min(b + lane, a.E - 1)] <= w));
    if (!live || e < 0) return u;
    int lo = 0, hi = a.rows;
    if (a.offsets) {
        lo = min(max(((const_i32*)a.offsets)[e], 0), a.rows);
        hi = min(max(((const_i32*)a.offsets)[e + 1], lo), a.rows);
    }
    const uint32_t mt = (uint32_t)(hi - lo + BM - 1) / BM;
    if (mt == 0) return u;                   // offsets that are not ascending
    const uint32_t rest = w - __builtin_amdgcn_readfirstlane(first[e]);
    u.blob = (const uint8_t*)((const_u64*)a.table)[e];
    // blocks of kBlockM row tiles by all matrix tiles, row tiles first: the units that
    // an XCD's workgroups are at together share rows and matrix rows evenly
    const uint32_t block = min(rest / (kBlockM * NT), (mt - 1) / kBlockM), in = rest - block * kBlockM * NT;
    const uint32_t wide = min(kBlockM, mt - block * kBlockM);
    u.nt = min(in / wide, (uint32_t)NT - 1);
    u.m0 = lo + (int)(block * kBlockM + in % wide) * BM;
    u.rows = min(BM, hi - u.m0);
    return u;
}

// Units of a launch at most: the rows fill rows / BM stretches, and each expert
// with rows may add one that is not full.
inline coli_status grid_of(const RowGroups& a, int BM, int NT, int threads, const char* what, uint32_t* grid) {
    const int64_t stretches = a.offsets ? (int64_t)a.rows / BM + std::min(a.E, a.rows)
                                        : ((int64_t)a.rows + BM - 1) / BM;
    const int64_t g = (stretches * NT + kXcds - 1) / kXcds * kXcds;
    if (g * threads > 0xffffffffll) return fail(COLI_EUNSUPPORTED, std::string(what) + ": more than 2^32 threads");
    *grid = (uint32_t)g;
    return COLI_OK;
}

}  // namespace coli
