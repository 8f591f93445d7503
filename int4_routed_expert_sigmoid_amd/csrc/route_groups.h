// Internal: launchers of route_groups.hip.
#pragma once

#include "common.h"

namespace coli {

constexpr int kRouteMaxExperts = 1024;           // 16 a lane
constexpr int kRouteMaxSlots = 32;
constexpr int kRouteMaxGroups = 64;              // one a lane, a bit each in a 64-bit word

struct RouteArgs {
    const void* logits;          // [T][E]
    const float* bias;           // [E] or nullptr
    int32_t T, E, k;
    bool softmax, norm;
    int32_t groups, kept, group_top;
    float scale;
    int32_t* idx;                // [T][k]
    float* w;                    // [T][k]
    float* scores;               // [T][E] or nullptr
};
coli_status launch_route_groups(const RouteArgs& a, int32_t dtype, hipStream_t stream);

struct RouteBwdArgs {
    const float* dw;             // [T][k]
    const void* logits;          // [T][E]
    const int32_t* idx;          // [T][k]
    int32_t T, E, k;
    bool softmax, norm;
    float scale;
    const float* dscores;        // [T][E] or nullptr
    void* dlogits;               // [T][E]
};
coli_status launch_route_groups_bwd(const RouteBwdArgs& a, int32_t dtype, int32_t grad_dtype, hipStream_t stream);

}  // namespace coli
