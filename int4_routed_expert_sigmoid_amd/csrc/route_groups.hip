// Routing with softmax or sigmoid scores, a selection bias and groups of experts, and the
// gradient of its weights (and of the scores) to the logits.
//
//   s_e = 1 / (1 + exp(-l_e)), or exp(l_e - max l) / sum_f exp(l_f - max l)
//   key_e = s_e + b_e; a group's value is its largest key or the sum of its two largest; the
//   best groups' experts with the k largest keys; w_j = scale * s_j / sum_i s_i, or scale * s_j
//   h_j = scale * (s_j / S) (g_j - sum_i g_i s_i / S), S = sum_i s_i, or scale * s_j g_j: s times the
//   gradient of the picked score; d: the gradient of the scores themselves
//   dl_e = (d_e s_e + h_e) (1 - s_e), or s_e d_e + h_e - s_e sum_f (s_f d_f + h_f)
//
// Scores are formed in double and rounded once to f32, so that the order of two experts, and with it
// the whole choice, does not hang on how an exponential was computed; gradients are f32. A wave has one
// token; lane l holds experts l * EPL .. + EPL - 1.
//
// What bounds them: the forward, instructions: 16384 tokens of 256 experts, softmax, 4 of 8 groups, k 8 take 25 us
// (the bytes alone 8), of which the k rounds of a maximum over the wave are about 8, the groups 3, the exponentials in
// 64 bits 2.5. (28 with keys and experts in one 64-bit code; four tokens a wave, 16 lanes each, are slower: 34.) The
// backward, HBM: 12. One token takes a launch, 4.
#include "mxfp4.h"
#include "route_groups.h"

namespace coli {
namespace {

constexpr int kThreads = 256, kTokens = kThreads / 64;

template <int S>
__device__ __forceinline__ float fmax_step(float v) { return fmaxf(v, __int_as_float(lane_xchg<S>(__float_as_int(v)))); }

__device__ __forceinline__ float wave_fmax(float v) {
    return fmax_step<32>(fmax_step<16>(fmax_step<8>(fmax_step<4>(fmax_step<2>(fmax_step<1>(v))))));
}

__device__ __forceinline__ float wave_fsum(float v) {
    return plain_stage<1>(plain_stage<2>(plain_stage<4>(plain_stage<8>(plain_stage<16>(plain_stage<32>(v))))));
}

// What a softmax subtracts from its logits: their largest, 0 where all are -inf (which has no difference to itself). A
// finite one is taken as it is, so that logits which all have the type's lowest value are equal ones.
__device__ __forceinline__ float softmax_top(float top) { return top == -__builtin_inff() ? 0.f : top; }

// The logits of a lane's experts, -inf behind the last.
template <typename T, int EPL>
__device__ __forceinline__ void load_logits(const T* row, int E, int e0, float (&l)[EPL]) {
    if (e0 + EPL <= E) {
        load_f32<T, EPL>(row + e0, l);
    } else {
#pragma unroll
        for (int i = 0; i < EPL; ++i) l[i] = e0 + i < E ? (float)row[e0 + i] : -__builtin_inff();
    }
}

// The wave's largest, uniform: rows of 16 by shifts, then from row to row; lane 63 ends with it. Lanes without a
// source take 0.
__device__ __forceinline__ uint32_t wave_top(uint32_t v) {
    auto step = [&](auto ctrl, auto rows) {
        v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, decltype(ctrl)::value, decltype(rows)::value, 0xf, false));
    };
    typedef std::integral_constant<int, 0xf> all;
    step(std::integral_constant<int, 0x111>{}, all{});                               // row_shr:1
    step(std::integral_constant<int, 0x112>{}, all{});
    step(std::integral_constant<int, 0x114>{}, all{});
    step(std::integral_constant<int, 0x118>{}, all{});
    step(std::integral_constant<int, 0x142>{}, std::integral_constant<int, 0xa>{});  // row_bcast:15
    step(std::integral_constant<int, 0x143>{}, std::integral_constant<int, 0xc>{});  // row_bcast:31
    return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

// The code by which a key is chosen, above 0; a NaN key comes first, so that it shows in the weights.
__device__ __forceinline__ uint32_t key_code(float key) {
    return (uint32_t)(selection_code(key != key ? __uint_as_float(0x7fc00000u) : key, 0) >> 32);
}

// The two largest of four, each pair in order.
__device__ __forceinline__ void merge2(float& a0, float& a1, float b0, float b1) {
    const float hi = fmaxf(a0, b0), lo = fminf(a0, b0);
    a1 = fmaxf(lo, fmaxf(a1, b1));
    a0 = hi;
}

// A group's value from its two largest keys (-inf: it has none, or only one). A sum that passes the lowest f32 value
// (biases that switch whole groups off do) stays there, so that the group comes before those without any expert.
__device__ __forceinline__ float group_value(float first, float second, bool nan, int top) {
    if (nan) return __uint_as_float(0x7fc00000u);
    return top == 2 && second != -__builtin_inff() ? fmaxf(first + second, -__FLT_MAX__) : first;
}

// How many of the groups, whose codes the lanes 0, step, 2 step, .. hold, come before group `mine`.
__device__ __forceinline__ int group_rank(uint32_t code, uint32_t mine, int groups, uint32_t step) {
    const uint64_t self = (uint64_t)code << 32 | ~mine;
    int rank = 0;
    for (uint32_t j = 0; j < (uint32_t)groups; ++j)
        rank += ((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)code, j * step) << 32 | ~j) > self;
    return rank;
}

template <typename T, int EPL>
__global__ __launch_bounds__(kThreads) void route_groups_kernel(RouteArgs a) {
    __shared__ float lds[kTokens][64 * EPL];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, E = a.E, e0 = lane * EPL;
    const int64_t t = (int64_t)blockIdx.x * kTokens + wave;
    if (t >= a.T) return;
    float l[EPL], s[EPL], key[EPL];
    load_logits<T, EPL>((const T*)a.logits + t * E, E, e0, l);
    float b[EPL] = {};
    if (a.bias) {
#pragma unroll
        for (int i = 0; i < EPL; ++i) b[i] = a.bias[min(e0 + i, E - 1)];
    }
    if (a.softmax) {
        float top = l[0];
#pragma unroll
        for (int i = 1; i < EPL; ++i) top = fmaxf(top, l[i]);
        const double m = softmax_top(wave_fmax(top));
        double x[EPL], sum = 0;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            x[i] = exp((double)l[i] - m);
            sum += x[i];
        }
        sum = wave_sum_f64(sum);
        const double inv = sum == 0 ? 0.0 : 1.0 / sum;
#pragma unroll
        for (int i = 0; i < EPL; ++i) s[i] = (float)(x[i] * inv);
    } else {
#pragma unroll
        for (int i = 0; i < EPL; ++i) s[i] = sigmoid_score(l[i]);
    }
    if (a.scores) {
        float* row = a.scores + t * E;
        if (e0 + EPL <= E) {
            store_f32<float, EPL>(row + e0, s);
        } else {
#pragma unroll
            for (int i = 0; i < EPL; ++i)
                if (e0 + i < E) row[e0 + i] = s[i];
        }
    }
    const float none = -__builtin_inff();
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        key[i] = l[i] == none || b[i] == none || e0 + i >= E ? none : s[i] + b[i];
        s[i] = key[i] != key[i] ? key[i] : s[i];      // a NaN bias shows in the weight, as a NaN score does
    }

    // the groups whose experts can be chosen
    uint32_t c[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) c[i] = key[i] != none ? key_code(key[i]) : 0;
    if (a.kept < a.groups) {
        const uint32_t size = E / a.groups, wide = size / EPL;
        if (size % EPL == 0 && (wide & (wide - 1)) == 0) {
            // a group is 1, 2, 4, .. 64 whole lanes: its two largest by exchanges among them
            float first = none, second = none;
            uint32_t nan = 0;
#pragma unroll
            for (int i = 0; i < EPL; ++i) {
                nan |= key[i] != key[i];
                second = fmaxf(second, fminf(first, key[i]));
                first = fmaxf(first, key[i]);
            }
            auto join = [&](auto s) {
                constexpr int S = decltype(s)::value;
                if (wide <= S) return;                // uniform
                merge2(first, second, __int_as_float(lane_xchg<S>(__float_as_int(first))),
                       __int_as_float(lane_xchg<S>(__float_as_int(second))));
                nan |= (uint32_t)lane_xchg<S>((int)nan);
            };
            join(std::integral_constant<int, 1>{});
            join(std::integral_constant<int, 2>{});
            join(std::integral_constant<int, 4>{});
            join(std::integral_constant<int, 8>{});
            join(std::integral_constant<int, 16>{});
            join(std::integral_constant<int, 32>{});
            const float value = group_value(first, second, nan != 0, a.group_top);
            const uint32_t code = value != none ? key_code(value) : 0;
            const int rank = group_rank(code, lane / wide, a.groups, wide);
#pragma unroll
            for (int i = 0; i < EPL; ++i) c[i] = rank < a.kept ? c[i] : 0;
        } else {
            const uint32_t div = ((1u << 21) + size - 1) / size;                     // e / size = e div >> 21, e < 1024
#pragma unroll
            for (int i = 0; i < EPL; ++i) lds[wave][e0 + i] = key[i];
            __builtin_amdgcn_wave_barrier();
            float first = none, second = none;
            bool nan = false;
            if (lane < a.groups) {
                for (uint32_t i = 0; i < size; ++i) {
                    const float v = lds[wave][lane * size + i];
                    nan |= v != v;
                    second = fmaxf(second, fminf(first, v));
                    first = fmaxf(first, v);
                }
            }
            const float value = group_value(first, second, nan, a.group_top);
            const uint32_t code = lane < a.groups && value != none ? key_code(value) : 0;
            const int rank = group_rank(code, lane, a.groups, 1);
            const uint64_t open = __ballot(code != 0 && rank < a.kept);
#pragma unroll
            for (int i = 0; i < EPL; ++i) c[i] = open >> (((uint32_t)(e0 + i) * div) >> 21 & 63) & 1 ? c[i] : 0;
            __builtin_amdgcn_wave_barrier();
        }
    }
    // The scores where a slot finds them by its expert. Each lane's codes in descending order (equal ones as they
    // are), with their places among its experts, 4 bits each; then k times the largest of the lanes' first codes, which
    // that lane drops; of equal ones the lowest lane's, whose experts come first.
    uint32_t place[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        lds[wave][e0 + i] = s[i];
        place[i] = i;
    }
#pragma unroll
    for (int pass = 0; pass < EPL; ++pass)
#pragma unroll
        for (int i = pass & 1; i + 1 < EPL; i += 2) {
            const bool sw = c[i + 1] > c[i];
            const uint32_t x = c[i], y = c[i + 1], p = place[i], q = place[i + 1];
            c[i] = sw ? y : x;
            c[i + 1] = sw ? x : y;
            place[i] = sw ? q : p;
            place[i + 1] = sw ? p : q;
        }
    typedef std::conditional_t<EPL == 16, uint64_t, uint32_t> Places;
    Places places = 0;
#pragma unroll
    for (int i = 0; i < EPL; ++i) places |= (Places)place[i] << (4 * i);
    int my_idx = -1, found = 0;
    for (; found < a.k; ++found) {
        const uint32_t top = wave_top(c[0]);
        if (top == 0) break;                          // no expert is left
        const int src = (int)__builtin_ctzll(__ballot(c[0] == top));
        const int e = src * EPL + (__builtin_amdgcn_readlane((int)(uint32_t)places, src) & 15);
        my_idx = lane == found ? e : my_idx;
        const bool taken = lane == src;
#pragma unroll
        for (int i = 0; i + 1 < EPL; ++i) c[i] = taken ? c[i + 1] : c[i];
        c[EPL - 1] = taken ? 0 : c[EPL - 1];
        places = taken ? places >> 4 : places;
    }
    __builtin_amdgcn_wave_barrier();
    const float mine = my_idx < 0 ? 0.f : lds[wave][my_idx];
    double sum = 0.0;
    for (int j = 0; j < found; ++j) sum += (double)__int_as_float(__builtin_amdgcn_readlane(__float_as_int(mine), j));
    if (lane < a.k) {
        double w = mine;
        if (a.norm && my_idx >= 0) w = sum == 0.0 ? 1.0 / found : w / sum;
        a.idx[t * a.k + lane] = my_idx;
        a.w[t * a.k + lane] = my_idx < 0 ? 0.f : (float)((double)a.scale * w);
    }
}

// s and 1 - s of a logit, without an overflow on either side.
__device__ __forceinline__ void sigmoid_pair(float l, float& s, float& rest) {
    const float e = expf(-fabsf(l)), r = 1.f / (1.f + e);
    s = l >= 0.f ? r : e * r;
    rest = l >= 0.f ? e * r : r;
    if (l != l) s = rest = l;
}

template <typename T, typename G, int EPL>
__global__ __launch_bounds__(kThreads) void route_groups_bwd_kernel(RouteBwdArgs a) {
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, E = a.E, e0 = lane * EPL;
    const int64_t t = (int64_t)blockIdx.x * kTokens + wave;
    if (t >= a.T) return;
    const T* row = (const T*)a.logits + t * E;
    // lane j < k: slot j
    int idx = -1;
    float g = 0.f;
    if (lane < a.k) {
        idx = a.idx[t * a.k + lane];
        g = a.dw[t * a.k + lane];
    }
    const bool used = idx >= 0 && idx < E;
    const float picked = used ? (float)row[idx] : 0.f;
    float l[EPL], d[EPL] = {};
    load_logits<T, EPL>(row, E, e0, l);
    if (a.dscores) {
        const float* p = a.dscores + t * E;
        if (e0 + EPL <= E) {
            load_f32<float, EPL>(p + e0, d);
        } else {
#pragma unroll
            for (int i = 0; i < EPL; ++i) d[i] = e0 + i < E ? p[e0 + i] : 0.f;
        }
    }
    float s[EPL], rest[EPL], sel;                // rest: 1 - s (sigmoid)
    if (a.softmax) {
        float top = l[0];
#pragma unroll
        for (int i = 1; i < EPL; ++i) top = fmaxf(top, l[i]);
        const float m = softmax_top(wave_fmax(top));
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            s[i] = expf(l[i] - m);
            sum += s[i];
        }
        sum = wave_fsum(sum);
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
        for (int i = 0; i < EPL; ++i) s[i] *= inv;
        sel = expf(picked - m) * inv;
    } else {
#pragma unroll
        for (int i = 0; i < EPL; ++i) sigmoid_pair(l[i], s[i], rest[i]);
        float unused;
        sigmoid_pair(picked, sel, unused);
    }
    sel = used ? sel : 0.f;
    g = used ? a.scale * g : 0.f;
    float h = sel * g;
    if (a.norm) {
        const float total = wave_fsum(sel), share = total == 0.f ? 0.f : sel / total;
        h = share * (g - wave_fsum(g * share));
    }
    if (!used) h = 0.f;
    float x[EPL];                                // s_e d_e + h_e
#pragma unroll
    for (int i = 0; i < EPL; ++i) x[i] = s[i] * d[i];
    for (int j = 0; j < a.k; ++j) {
        const int e = __builtin_amdgcn_readlane(used ? idx : -1, j);
        const float v = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(h), j));
#pragma unroll
        for (int i = 0; i < EPL; ++i) x[i] += e == e0 + i ? v : 0.f;
    }
    if (a.softmax) {
        float all = 0.f;
#pragma unroll
        for (int i = 0; i < EPL; ++i) all += x[i];
        all = wave_fsum(all);
#pragma unroll
        for (int i = 0; i < EPL; ++i) x[i] -= s[i] * all;
    } else {
#pragma unroll
        for (int i = 0; i < EPL; ++i) x[i] *= rest[i];
    }
    G* o = (G*)a.dlogits + t * E;
    if (e0 + EPL <= E) {
        store_f32<G, EPL>(o + e0, x);
    } else {
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            if (e0 + i < E) o[e0 + i] = (G)x[i];
    }
}

// Runs fn with the number of experts a lane holds.
template <typename F>
coli_status with_epl(int E, F&& fn) {
    if (E <= 64) return fn(std::integral_constant<int, 1>{});
    if (E <= 128) return fn(std::integral_constant<int, 2>{});
    if (E <= 256) return fn(std::integral_constant<int, 4>{});
    if (E <= 512) return fn(std::integral_constant<int, 8>{});
    return fn(std::integral_constant<int, 16>{});
}

}  // namespace

coli_status launch_route_groups(const RouteArgs& a, int32_t dtype, hipStream_t stream) {
    if (a.T == 0) return COLI_OK;
    const uint32_t grid = ((uint32_t)a.T + kTokens - 1) / kTokens;
    return with_elem(dtype, [&](auto e) -> coli_status {
        using T = decltype(e);
        return with_epl(a.E, [&](auto n) -> coli_status {
            launch(route_groups_kernel<T, decltype(n)::value>, dim3(grid), dim3(kThreads), 0, stream, a);
            COLI_CHECK_LAUNCH("route_groups kernel launch");
            return COLI_OK;
        });
    });
}

coli_status launch_route_groups_bwd(const RouteBwdArgs& a, int32_t dtype, int32_t grad_dtype, hipStream_t stream) {
    if (a.T == 0) return COLI_OK;
    const uint32_t grid = ((uint32_t)a.T + kTokens - 1) / kTokens;
    return with_elem(dtype, [&](auto e) -> coli_status {
        using T = decltype(e);
        return with_elem(grad_dtype, [&](auto ge) -> coli_status {
            using G = decltype(ge);
            return with_epl(a.E, [&](auto n) -> coli_status {
                launch(route_groups_bwd_kernel<T, G, decltype(n)::value>, dim3(grid), dim3(kThreads), 0, stream, a);
                COLI_CHECK_LAUNCH("route_groups_bwd kernel launch");
                return COLI_OK;
            });
        });
    });
}

}  // namespace coli
