// The router of a mixture-of-experts block and its gradient.
//
// Mathematics, per token with logits l[e] (see include/libmxmoe_block.h):
//   s = softmax(l) or sigmoid(l), c = s + bias; the k largest c among the
//   groups of the largest group scores; weights from s at those experts.
//
// Layout: a team of W neighbouring lanes has a token, W a power of two, and
// lane a of it ITEMS experts in registers.  With G groups padded to the next
// power of two P, lanes [a LG, (a + 1) LG), LG = W / P, have group a, and lane p of
// them the group's experts [p ITEMS, (p + 1) ITEMS): lower lanes have lower
// indices, so that "the lowest index" is the lowest lane of a ballot, and
// group scores are reductions over aligned lanes.
#include "mx_bf16.h"
#include "mx_block.h"
#include "mx_lanes.h"

namespace mx {
namespace {

constexpr int kThreads = 256;

// Keys: unsigned numbers in the order of the floats they stand for, NaN on
// top, 0 for what cannot be chosen (no float has it).
__device__ __forceinline__ uint64_t key_of(double v) {
    if (v != v) return ~0ull;
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    return u >> 63 ? ~u : u | (1ull << 63);
}
__device__ __forceinline__ double value_of(uint64_t key) {
    if (key == ~0ull) return __builtin_nan("");
    return __builtin_bit_cast(double, key >> 63 ? key & ~(1ull << 63) : ~key);
}

__device__ __forceinline__ float load_logit(const float* p) { return *p; }
__device__ __forceinline__ float load_logit(const uint16_t* p) { return __builtin_bit_cast(float, (uint32_t)*p << 16); }

// The two largest keys of a set.
struct Top2 {
    uint64_t a, b;
};

// L: float or uint16_t (bf16).
template <class L, int W, int ITEMS>
__global__ __launch_bounds__(kThreads) void router_kernel(RouterArgs g, int32_t lanes_per_group) {
    const int lane = threadIdx.x & 63;
    const int a = lane & (W - 1);
    const int64_t token = (int64_t)blockIdx.x * (kThreads / W) + threadIdx.x / W;
    const bool live = token < g.T;
    const L* const row = (const L*)g.logits + (live ? token : 0) * g.ldl;
    const int size = g.E / g.groups;
    const int group = a / lanes_per_group;
    const int first = a % lanes_per_group * ITEMS;  // in the group
    const int here = !live || group >= g.groups ? 0 : size - first < 0 ? 0 : size - first < ITEMS ? size - first : ITEMS;
    const int base = group * size + first;
    const float lowest = -__builtin_inff();
    const bool sigmoid = g.flags & MX_ROUTER_SIGMOID, renorm = g.flags & MX_ROUTER_RENORM;

    // without a bias, and with one choice per group score, the logits have the order of the choices
    const bool by_logit = g.bias == nullptr && (g.groups == 1 || g.top == 1);

    float l[ITEMS];
    float top = lowest;
#pragma unroll
    for (int j = 0; j < ITEMS; ++j) {
        l[j] = j < here ? load_logit(row + base + j) : lowest;
        top = fmaxf(top, l[j]);
    }
    top = team_reduce<W>(top, [](float p, float q) { return fmaxf(p, q); });

    // scores in binary64
    double sum = 0.0;
    if (!sigmoid) {
#pragma unroll
        for (int j = 0; j < ITEMS; ++j)
            if (l[j] != lowest) sum += exp((double)l[j] - (double)top);
        sum = team_reduce<W>(sum, [](double p, double q) { return p + q; });
    }
    const auto score = [&](float v) {
        if (v == lowest) return 0.0;
        return sigmoid ? 1.0 / (1.0 + exp(-(double)v)) : exp((double)v - (double)top) / sum;
    };
    uint64_t key[ITEMS];
#pragma unroll
    for (int j = 0; j < ITEMS; ++j) {
        key[j] = 0;
        if (j >= here) continue;
        const double s = score(l[j]);
        if (g.scores != nullptr) g.scores[token * g.E + base + j] = (float)s;
        if (l[j] == lowest) continue;
        const double c = by_logit ? (double)l[j] : g.bias != nullptr ? s + (double)g.bias[base + j] : s;
        if (c != -__builtin_inf()) key[j] = key_of(c);
    }

    if (g.groups > 1) {
        Top2 t{0, 0};
#pragma unroll
        for (int j = 0; j < ITEMS; ++j) {
            const uint64_t lower = key[j] < t.a ? key[j] : t.a;
            t.a = key[j] > t.a ? key[j] : t.a;
            t.b = lower > t.b ? lower : t.b;
        }
        for (int d = 1; d < lanes_per_group; d *= 2) {
            const uint64_t oa = __shfl_xor((unsigned long long)t.a, d), ob = __shfl_xor((unsigned long long)t.b, d);
            const uint64_t lower = oa < t.a ? oa : t.a;
            t.b = t.b > ob ? t.b : ob;
            t.b = t.b > lower ? t.b : lower;
            t.a = oa > t.a ? oa : t.a;
        }
        const uint64_t mine = g.top > 1 && t.b != 0 ? key_of(value_of(t.a) + value_of(t.b)) : t.a;
        int ahead = 0;
        for (int h = 0; h < g.groups; ++h) {
            const uint64_t other = __shfl((unsigned long long)mine, h * lanes_per_group, W);
            ahead += other > mine || (other == mine && h < group);
        }
        if (ahead >= g.kept)
#pragma unroll
            for (int j = 0; j < ITEMS; ++j) key[j] = 0;
    }

    // k rounds: the largest key, the lowest lane that has it, its lowest item
    int32_t chosen = -1;  // of round a
    for (int i = 0; i < g.k; ++i) {
        uint64_t best = 0;
        int at = 0;
#pragma unroll
        for (int j = 0; j < ITEMS; ++j)
            if (key[j] > best) {
                best = key[j];
                at = j;
            }
        const uint64_t most = team_reduce<W>(best, [](uint64_t p, uint64_t q) { return p > q ? p : q; });
        uint64_t have = __ballot(best == most && most != 0);
        if constexpr (W < 64) have = have >> (lane & ~(W - 1)) & ((1ull << W) - 1);
        const int winner = have != 0 ? __builtin_ctzll(have) : 0;
        const int32_t expert = __shfl(base + at, winner, W);
        if (have != 0 && a == i) chosen = expert;
        if (have != 0 && a == winner) {
#pragma unroll
            for (int j = 0; j < ITEMS; ++j)
                if (j == at) key[j] = 0;
        }
    }

    // lane i < k has choice i
    double s = 0.0;
    if (live && a < g.k && chosen >= 0) {
        const float v = load_logit(row + chosen);
        // the softmax's sum cancels (unless a NaN is in it that is not chosen)
        s = !sigmoid && renorm && by_logit ? exp((double)v - (double)top) : score(v);
    }
    if (renorm) {
        const double all = team_reduce<W>(s, [](double p, double q) { return p + q; });
        s = chosen < 0 || all == 0.0 ? 0.0 : s / all;
    }
    if (live && a < g.k) {
        g.experts[token * g.k + a] = chosen;
        g.weights[token * g.k + a] = (float)((double)g.scale * s);
    }
}

template <class L, int W, int ITEMS>
hipError_t run_router(const RouterArgs& g, int lanes_per_group, hipStream_t stream) {
    const int64_t blocks = (g.T + kThreads / W - 1) / (kThreads / W);
    hipLaunchKernelGGL((router_kernel<L, W, ITEMS>), dim3((unsigned)blocks), dim3(kThreads), 0, stream, g,
                       lanes_per_group);
    return hipGetLastError();
}

template <class L, int W>
hipError_t pick_items(const RouterArgs& g, int items, int lanes_per_group, hipStream_t stream) {
    if (items <= 1) return run_router<L, W, 1>(g, lanes_per_group, stream);
    if (items <= 2) return run_router<L, W, 2>(g, lanes_per_group, stream);
    if (items <= 4) return run_router<L, W, 4>(g, lanes_per_group, stream);
    if constexpr (W == 64) {
        if (items <= 8) return run_router<L, W, 8>(g, lanes_per_group, stream);
        if (items <= 16) return run_router<L, W, 16>(g, lanes_per_group, stream);
        if (items <= 32) return run_router<L, W, 32>(g, lanes_per_group, stream);
        return run_router<L, W, 64>(g, lanes_per_group, stream);
    }
    return hipErrorInvalidValue;  // (the team is widened before it gets here)
}

template <class L>
hipError_t pick_team(const RouterArgs& g, hipStream_t stream) {
    int padded = 1;
    while (padded < g.groups) padded *= 2;
    const int size = g.E / g.groups;
    // the narrowest team that has a lane for each choice and group and at most 4 experts per lane
    int W = 8;
    while (W < 64 && (W < g.k || W < padded || size > 4 * (W / padded))) W *= 2;
    const int lanes = W / padded;
    const int items = (size + lanes - 1) / lanes;
    if (W == 8) return pick_items<L, 8>(g, items, lanes, stream);
    if (W == 16) return pick_items<L, 16>(g, items, lanes, stream);
    if (W == 32) return pick_items<L, 32>(g, items, lanes, stream);
    return pick_items<L, 64>(g, items, lanes, stream);
}

// ---------------------------------------------------------------------------
// Gradient.  A team of W lanes has a token; lane i < k its choice i, and each
// lane every W-th expert of the row.
// ---------------------------------------------------------------------------

__device__ __forceinline__ float wide_exp(float v) { return expf(v); }
__device__ __forceinline__ float sigmoid_of(float v) { return 1.0f / (1.0f + expf(-v)); }
__device__ __forceinline__ void store_grad(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_grad(uint16_t* p, float v) { *p = __builtin_bit_cast(uint16_t, (__bf16)v); }

template <class L, int W>
__global__ __launch_bounds__(kThreads) void router_backward_kernel(RouterBackwardArgs g) {
    const int a = threadIdx.x & (W - 1);
    const int64_t token = (int64_t)blockIdx.x * (kThreads / W) + threadIdx.x / W;
    const bool live = token < g.T;
    const int64_t t = live ? token : 0;
    const L* const row = (const L*)g.logits + t * g.ldl;
    const float lowest = -__builtin_inff();
    const bool sigmoid = g.flags & MX_ROUTER_SIGMOID, renorm = g.flags & MX_ROUTER_RENORM;

    // softmax: the row's largest logit, and the sum
    float top = 0.0f, over = 1.0f;
    if (!sigmoid) {
        top = lowest;
        for (int e = a; e < g.E; e += W) top = fmaxf(top, load_logit(row + e));
        top = team_reduce<W>(top, [](float p, float q) { return fmaxf(p, q); });
        float sum = 0.0f;
        for (int e = a; e < g.E; e += W) {
            const float v = load_logit(row + e);
            if (v != lowest) sum += expf(v - top);
        }
        over = 1.0f / team_sum<W>(sum);
    }
    const auto score = [&](float v) {
        if (v == lowest) return 0.0f;
        return sigmoid ? sigmoid_of(v) : expf(v - top) * over;
    };

    int32_t expert = -1;
    float d = 0.0f, s = 0.0f;
    if (live && a < g.k) {
        expert = g.experts[t * g.k + a];
        if (expert < 0 || expert >= g.E) expert = -1;
        if (expert >= 0) {
            d = g.dweights[t * g.k + a];
            const float v = load_logit(row + expert);
            s = !sigmoid && renorm ? (v == lowest ? 0.0f : expf(v - top)) : score(v);
        }
    }
    if (renorm) {
        const float all = team_sum<W>(s);
        const float part = all == 0.0f ? 0.0f : s / all;  // s_i / S
        const float mean = team_sum<W>(part == 0.0f ? 0.0f : part * d);
        // softmax: S is taken over e^(l - top), and s_i = e^(l_i - top) over: d s_i / S is the same
        const float under = sigmoid ? all : all * over;
        d = expert < 0 || all == 0.0f ? 0.0f : (d - mean) / under;
    }
    d *= g.scale;

    // sum_f s_f ds_f
    float mean = 0.0f;
    if (!sigmoid) {
        float sum = 0.0f;
        if (expert >= 0) {
            const float p = score(load_logit(row + expert));
            if (p != 0.0f) sum = p * d;
        }
        if (g.dscores != nullptr)
            for (int e = a; e < g.E; e += W) {
                const float p = score(load_logit(row + e));
                if (p != 0.0f) sum += p * g.dscores[t * g.E + e];
            }
        mean = team_sum<W>(sum);
    }
    L* const out = (L*)g.dlogits + t * g.ldd;
    for (int e0 = 0; e0 < g.E; e0 += W) {
        const int e = e0 + a;
        const bool in = live && e < g.E;
        float ds = in && g.dscores != nullptr ? g.dscores[t * g.E + e] : 0.0f;
        for (int i = 0; i < g.k; ++i) {
            const int32_t at = __shfl(expert, i, W);
            const float more = __shfl(d, i, W);
            if (at == e) ds += more;
        }
        if (!in) continue;
        const float v = load_logit(row + e);
        const float p = score(v);
        const float grad = v == lowest ? 0.0f : sigmoid ? p * (1.0f - p) * ds : p * (ds - mean);
        store_grad(out + e, grad);
    }
}

template <class L>
hipError_t run_backward(const RouterBackwardArgs& g, hipStream_t stream) {
    constexpr int W = 64;
    const int64_t blocks = (g.T + kThreads / W - 1) / (kThreads / W);
    hipLaunchKernelGGL((router_backward_kernel<L, W>), dim3((unsigned)blocks), dim3(kThreads), 0, stream, g);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_router(const RouterArgs& a, hipStream_t stream) {
    return a.flags & MX_ROUTER_LOGITS_BF16 ? pick_team<uint16_t>(a, stream) : pick_team<float>(a, stream);
}

hipError_t launch_router_backward(const RouterBackwardArgs& a, hipStream_t stream) {
    return a.flags & MX_ROUTER_LOGITS_BF16 ? run_backward<uint16_t>(a, stream) : run_backward<float>(a, stream);
}

}  // namespace mx
