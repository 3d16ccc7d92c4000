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
//
// Choices are compared in binary64, but only few are computed in it: choices
// in binary32, within a bound tau of the true ones, give a threshold that at
// least k + 1 experts reach (the (k + 1)-th largest of the maxima of small
// blocks of experts); whoever comes within 2 tau of it, usually k + 1 to 2 k
// experts, is collected in LDS, computed in binary64 one expert a lane, and
// ranked against the others.  A list that is full (rows of ties) is ranked as
// far as it goes, and its k best stay in it for the next ones.  Group scores
// that binary32 cannot tell apart are formed again from the few largest
// choices of each group in binary64.
//
// What bounds it: vector instructions, about 250 per token at 256 experts and
// k = 8 (HBM would take 7 us for what follows).  Measured: 32768 tokens to 8 of
// 256 experts in 8 groups, sigmoid, bias, float32 logits 21 us (the same in bf16);
// 8191 tokens to 6 of 165 in 3 groups, softmax, all scores written, bf16 10; 16
// tokens 6.4, the chain of reductions.  k rounds of "the largest that is left" in
// binary64 took 59, 18 and 7.6.
//
// Six waves a vector unit: the bf16 instances of 16 experts a lane spill 4 to 7
// registers for it (with five, 32768 tokens to 8 of 256 in 8 groups take as
// long, to 4 of 128 9.9 us instead of 10.5; float32 spills none).
#include <type_traits>

#include "mx_bf16.h"
#include "mx_block.h"
#include "mx_lanes.h"

namespace mx {
namespace {

constexpr int kThreads = 256;
constexpr float kLowest = -__builtin_inff();

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
__device__ __forceinline__ uint32_t key_of(float v) {
    if (v != v) return ~0u;
    const uint32_t u = __builtin_bit_cast(uint32_t, v);
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t key) {
    if (key == ~0u) return __builtin_nanf("");
    return __builtin_bit_cast(float, key >> 31 ? key & 0x7FFFFFFFu : ~key);
}

__device__ __forceinline__ float load_logit(const float* p) { return *p; }
__device__ __forceinline__ float load_logit(const uint16_t* p) { return __builtin_bit_cast(float, (uint32_t)*p << 16); }

// Pieces of a row as they lie, of any alignment (global loads and stores of
// 16 bytes need none).
typedef float f32x4u __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u32x4u __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x2u __attribute__((ext_vector_type(2), aligned(2)));

// n consecutive logits, of which `here` exist; the others read as -infinity.
template <int n>
__device__ __forceinline__ void load_logits(const float* p, int here, float (&v)[n]) {
    if constexpr (n >= 4) {
        if (here == n) {
#pragma unroll
            for (int j = 0; j < n; j += 4) {
                const f32x4u x = *reinterpret_cast<const f32x4u*>(p + j);
                v[j] = x.x, v[j + 1] = x.y, v[j + 2] = x.z, v[j + 3] = x.w;
            }
            return;
        }
    }
#pragma unroll
    for (int j = 0; j < n; ++j) v[j] = j < here ? p[j] : kLowest;
}
template <int n>
__device__ __forceinline__ void load_logits(const uint16_t* p, int here, float (&v)[n]) {
    if constexpr (n >= 8) {
        if (here == n) {
#pragma unroll
            for (int j = 0; j < n; j += 8) {
                const u32x4u x = *reinterpret_cast<const u32x4u*>(p + j);
                v[j] = lo_bf16(x.x), v[j + 1] = hi_bf16(x.x), v[j + 2] = lo_bf16(x.y), v[j + 3] = hi_bf16(x.y);
                v[j + 4] = lo_bf16(x.z), v[j + 5] = hi_bf16(x.z), v[j + 6] = lo_bf16(x.w), v[j + 7] = hi_bf16(x.w);
            }
            return;
        }
    }
    if constexpr (n == 4) {
        if (here == n) {
            const u32x2u x = *reinterpret_cast<const u32x2u*>(p);
            v[0] = lo_bf16(x.x), v[1] = hi_bf16(x.x), v[2] = lo_bf16(x.y), v[3] = hi_bf16(x.y);
            return;
        }
    }
#pragma unroll
    for (int j = 0; j < n; ++j) v[j] = j < here ? load_logit(p + j) : kLowest;
}

template <int n>
__device__ __forceinline__ void store_values(float* p, int here, const float (&v)[n]) {
    if constexpr (n >= 4) {
        if (here == n) {
#pragma unroll
            for (int j = 0; j < n; j += 4) *reinterpret_cast<f32x4u*>(p + j) = f32x4u{v[j], v[j + 1], v[j + 2], v[j + 3]};
            return;
        }
    }
#pragma unroll
    for (int j = 0; j < n; ++j)
        if (j < here) p[j] = v[j];
}
template <int n>
__device__ __forceinline__ void store_values(uint16_t* p, int here, const float (&v)[n]) {
    static_assert(n == 8, "16 bytes");
    if (here == n) {
        *reinterpret_cast<u32x4u*>(p) = u32x4u{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]),
                                               pack_bf16(v[6], v[7])};
        return;
    }
#pragma unroll
    for (int j = 0; j < n; ++j)
        if (j < here) p[j] = __builtin_bit_cast(uint16_t, (__bf16)v[j]);
}

// e^x, |x| <= 150 or NaN: the product with log2(e) in two parts, so that the
// error stays below 3 steps whatever x is.
__device__ __forceinline__ float exp_of(float x) {
#pragma clang fp contract(off)  // (a sum of these has the same bits wherever it is formed)
    const float t = x * 1.44269504f;
    float low = __builtin_fmaf(x, 1.44269504f, -t);
    low = __builtin_fmaf(x, 1.92596299e-8f, low);  // log2(e) - fp32(log2(e))
    return __builtin_amdgcn_exp2f(t) * __builtin_fmaf(low, 0.693147181f, 1.0f);
}
// Of a logit below the row's largest; 0 below -150 (and for -infinity).
__device__ __forceinline__ float exp_below(float x) { return x < -150.0f ? 0.0f : exp_of(x); }
__device__ __forceinline__ float sigmoid_near(float l) { return __builtin_amdgcn_rcpf(1.0f + exp_of(-l)); }
__device__ __forceinline__ float sigmoid_of(float l) {
    if (fabsf(l) > 150.0f) return l > 0.0f ? 1.0f : 0.0f;
    return sigmoid_near(l);
}

// The two largest values of a set.
struct Top2 {
    float a, b;
    __device__ __forceinline__ void add(float v) {
        b = __builtin_amdgcn_fmed3f(a, b, v);
        a = fmaxf(a, v);
    }
    // the group's score: the sum of both (finite, as a group without any has -infinity), or of the one that is there
    __device__ __forceinline__ float score(int top) const {
        return top > 1 && b != kLowest ? fmaxf(a + b, -__FLT_MAX__) : a;
    }
};
struct Keys2 {
    uint64_t a, b;
    __device__ __forceinline__ void add(uint64_t k) {
        const uint64_t lower = k < a ? k : a;
        a = k > a ? k : a;
        b = lower > b ? lower : b;
    }
    __device__ __forceinline__ uint64_t score(int top) const {
        return top > 1 && b != 0 ? key_of(value_of(a) + value_of(b)) : a;
    }
};

// Sums over the team's lanes up to this one.
template <int W>
__device__ __forceinline__ int team_scan(int v, int a) {
    const auto from = [&](auto d) {  // of the lane d before, in a row of 16 lanes; 0 outside of it
        constexpr int D = decltype(d)::value;
        const int before = __builtin_amdgcn_update_dpp(0, v, 0x110 | D, 0xF, 0xF, true);  // row_shr
        return W >= 16 || a >= D ? before : 0;
    };
    v += from(std::integral_constant<int, 1>{});
    v += from(std::integral_constant<int, 2>{});
    v += from(std::integral_constant<int, 4>{});
    if constexpr (W >= 16) v += from(std::integral_constant<int, 8>{});
#pragma unroll
    for (int d = 16; d < W; d *= 2) {  // the last lane of the rows before
        const int before = __shfl(v, (a & ~(d - 1)) - 1, W);
        if (a & d) v += before;
    }
    return v;
}

// Orders LDS accesses of the lanes of one wave.
__device__ __forceinline__ void wave_sync() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// L: float or uint16_t (bf16).
template <class L, int W, int ITEMS>
__global__ __launch_bounds__(kThreads, ITEMS <= 16 ? 6 : 1) void router_kernel(RouterArgs g, int32_t lanes_per_group) {
    constexpr int kTeams = kThreads / W;
    constexpr int kList = 2 * W;  // candidates that are ranked
    __shared__ uint64_t list_key[kTeams][kList];
    __shared__ double list_part[kTeams][kList];
    __shared__ int32_t list_expert[kTeams][kList];
    __shared__ uint64_t chosen_key[kTeams][W + 1];
    __shared__ double chosen_part[kTeams][W];
    __shared__ int32_t chosen_expert[kTeams][W];
    __shared__ float sum32[kTeams];
    const int lane = threadIdx.x & 63;
    const int a = lane & (W - 1);
    const int team = threadIdx.x / W;
    const int64_t token = (int64_t)blockIdx.x * kTeams + team;
    const bool live = token < g.T;
    const L* const row = (const L*)g.logits + (live ? token : 0) * g.ldl;
    const int size = g.E / g.groups;
    const int group = a / lanes_per_group;
    const int first = a % lanes_per_group * ITEMS;  // in the group
    const int here = !live || group >= g.groups ? 0 : size - first < 0 ? 0 : size - first < ITEMS ? size - first : ITEMS;
    const int base = group * size + first;
    const bool sigmoid = g.flags & MX_ROUTER_SIGMOID, renorm = g.flags & MX_ROUTER_RENORM;
    // without a bias, and with one choice per group score, the logits have the order of the choices
    const bool by_logit = g.bias == nullptr && (g.groups == 1 || g.top == 1);
    const auto larger = [](float p, float q) { return fmaxf(p, q); };

    float l[ITEMS];
    load_logits<ITEMS>(row + base, here, l);
    float top = kLowest;
#pragma unroll
    for (int j = 0; j < ITEMS; ++j) top = fmaxf(top, l[j]);
    top = team_reduce<W>(top, larger);

    float least_logit = -kLowest;
#pragma unroll
    for (int j = 0; j < ITEMS; ++j) least_logit = fminf(least_logit, l[j]);
    // the same in all lanes: no logit of the wave is -infinity, or so far off that its exponential has to be cut
    const bool plain = __ballot(!(sigmoid ? least_logit > -100.0f && top < 100.0f : least_logit - top > -100.0f)) == 0;

    // scores in binary32
    float c[ITEMS];
    float over = 1.0f;  // 1 / the softmax's sum
    double sum = 1.0;
    if (!by_logit || g.scores != nullptr || (!sigmoid && !renorm)) {
        if (sigmoid) {
            if (plain) {
#pragma unroll
                for (int j = 0; j < ITEMS; ++j) c[j] = sigmoid_near(l[j]);
            } else {
#pragma unroll
                for (int j = 0; j < ITEMS; ++j) c[j] = sigmoid_of(l[j]);
            }
        } else {
            float part = 0.0f;
            if (plain) {
#pragma unroll
                for (int j = 0; j < ITEMS; ++j) part += c[j] = exp_of(l[j] - top);
            } else {
#pragma unroll
                for (int j = 0; j < ITEMS; ++j) part += c[j] = l[j] == kLowest ? 0.0f : exp_below(l[j] - top);
            }
            part = team_sum<W>(part);
            sum = (double)part;
            over = part == 0.0f ? 0.0f : 1.0f / part;
            if (a == 0) sum32[team] = part;
#pragma unroll
            for (int j = 0; j < ITEMS; ++j) c[j] *= over;
        }
        if (g.scores != nullptr) store_values<ITEMS>(g.scores + token * g.E + base, here, c);
    }
    // (of finite logits, or NaN; a softmax's score is this over the sum)
    const auto part64 = [&](float v) { return sigmoid ? 1.0 / (1.0 + exp(-(double)v)) : exp((double)v - (double)top); };
    const auto choice64 = [&](int32_t expert, double* part) {  // as a key; 0: cannot be chosen
        const float v = load_logit(row + expert), b = g.bias != nullptr ? g.bias[expert] : 0.0f;
        const double s = *part = part64(v);
        return v == kLowest || b == kLowest ? 0 : key_of(by_logit ? (double)v + 0.0 : (sigmoid ? s : s / sum) + (double)b);
    };
    // The softmax's sum above is of binary32, ITEMS terms in a row, 6 joins and 8 half steps of a term off at most (here:
    // twice that): choices that are no more than that part of the largest score apart are formed again with one of binary64
    // (a pair in thousands; all of them: 512 experts, 16384 tokens 29 us, now 15).
    constexpr float kSumError = (ITEMS + 14) * 0x1p-23f;
    bool exact = sigmoid || by_logit;
    const auto sum_exactly = [&]() {
        if (exact) return;
        exact = true;
        sum = 0.0;
#pragma unroll 2
        for (int j = 0; j < here; ++j) {  // (read again: registers have no index)
            const float v = load_logit(row + base + j);
            if (v != kLowest) sum += exp((double)v - (double)top);
        }
        sum = team_reduce<W>(sum, [](double p, double q) { return p + q; });
    };

    // choices in binary32: -infinity what cannot be chosen, +infinity also for NaN
    if (by_logit) {
#pragma unroll
        for (int j = 0; j < ITEMS; ++j) c[j] = fminf(l[j], -kLowest);
    } else {
        if (g.bias != nullptr) {
            float b[ITEMS];
            load_logits<ITEMS>(g.bias + base, here, b);
#pragma unroll
            for (int j = 0; j < ITEMS; ++j) c[j] += b[j];
        }
#pragma unroll
        for (int j = 0; j < ITEMS; ++j) c[j] = fminf(c[j], -kLowest);
        if (!plain) {
#pragma unroll
            for (int j = 0; j < ITEMS; ++j) c[j] = l[j] == kLowest ? kLowest : c[j];
        }
    }
    // a score is within this of its true value: 2^-19 of the largest one (rounding of l - max, 3 steps of the exponential, 2
    // of the quotient; |x| e^x < 0.4) and the sum's error, or it has underflowed
    const float off = by_logit ? 0.0f : (sigmoid ? 0x1p-19f * sigmoid_of(top) : (0x1p-19f + kSumError) * over) + 0x1p-120f;

    if (g.groups > 1) {
        Top2 t{kLowest, kLowest};
#pragma unroll
        for (int j = 0; j < ITEMS; ++j) t.add(c[j]);
        t = team_reduce(t, lanes_per_group, [](Top2 p, Top2 q) {
            p.b = fmaxf(p.b, q.b);
            p.add(q.a);
            return p;
        });
        const float mine = t.score(g.top);
        int ahead = 0;
        for (int h = 0; h < g.groups; ++h) {
            const float other = __shfl(mine, h * lanes_per_group, W);
            ahead += other > mine || (other == mine && h < group);
        }
        // the last one kept and the first one dropped, of those that can be chosen
        const float next = team_reduce<W>(ahead < g.kept ? kLowest : mine, larger);
        bool undecided;
        float tau = 0.0f;
        if (by_logit) {
            undecided = next == -kLowest;  // (a NaN is above infinity)
        } else {
            const float last = team_reduce<W>(ahead < g.kept && mine != kLowest ? mine : -kLowest,
                                              [](float p, float q) { return fminf(p, q); });
            // each of the four sums is half a step off, and so are the two of them
            float size = mine == kLowest ? 0.0f : fabsf(t.a);
            if (g.top > 1 && t.b != kLowest) size += fabsf(t.b);
            size = team_reduce<W>(size, larger);
            tau = off + 0x1p-24f * size;
            undecided = next != kLowest && !(last - next > 4.0f * tau);
        }
        if (__ballot(undecided) != 0) {
            sum_exactly();
            const float from = fmaxf((g.top > 1 ? t.b : t.a) - 2.0f * tau, -__FLT_MAX__);  // (of NaN: the lowest)
            uint64_t some = 0;
#pragma unroll
            for (int j = 0; j < ITEMS; ++j) some |= c[j] >= from ? 1ull << j : 0;
            Keys2 u{0, 0};
            while (some != 0) {
                double part;
                u.add(choice64(base + __builtin_ctzll(some), &part));
                some &= some - 1;
            }
            for (int d = 1; d < lanes_per_group; d *= 2) {
                const uint64_t oa = __shfl_xor((unsigned long long)u.a, d), ob = __shfl_xor((unsigned long long)u.b, d);
                u.b = u.b > ob ? u.b : ob;
                u.add(oa);
            }
            const uint64_t score = u.score(g.top);
            ahead = 0;
            for (int h = 0; h < g.groups; ++h) {
                const uint64_t other = __shfl((unsigned long long)score, h * lanes_per_group, W);
                ahead += other > score || (other == score && h < group);
            }
        }
        if (ahead >= g.kept)
#pragma unroll
            for (int j = 0; j < ITEMS; ++j) c[j] = kLowest;
    }

    // threshold
    float least = -__FLT_MAX__;
    if constexpr (W * ITEMS > kList) {
        constexpr int kBlocks = ITEMS <= 16 ? 2 : ITEMS / 8;
        uint32_t block[kBlocks];
#pragma unroll
        for (int b = 0; b < kBlocks; ++b) {
            float v = kLowest;
#pragma unroll
            for (int j = b * (ITEMS / kBlocks); j < (b + 1) * (ITEMS / kBlocks); ++j) v = fmaxf(v, c[j]);
            block[b] = v == kLowest ? 0 : key_of(v + 0.0f);  // (no -0)
        }
        // k times the next lower value: subtracting the last one wraps the lower ones around, above all others
        uint32_t at = 0, highest = 0;
        for (int i = 0; i <= g.k; ++i) {
            uint32_t best = 0;
#pragma unroll
            for (int b = 0; b < kBlocks; ++b) {
                const uint32_t d = block[b] - at;
                best = d > best ? d : best;
            }
            best = at + team_reduce<W>(best, [](uint32_t p, uint32_t q) { return p > q ? p : q; });
            if (i == 0) highest = best;
            at = i == 0 || best < at ? best : at;  // (nothing is lower: all blocks reach it)
        }
        if (at != 0) {
            least = value_of(at);
            if (!by_logit) {
                // the sums with the bias are half a step off, of the largest of these
                const float tau = off + 0x1p-22f * fmaxf(fabsf(least), fabsf(value_of(highest)));
                least = fmaxf(least - 2.0f * tau, -__FLT_MAX__);  // (of NaN: the lowest)
            }
        }
    }

    // candidates, in the order of their indices
    int count = 0;
#pragma unroll
    for (int j = 0; j < ITEMS; ++j) count += c[j] >= least;
    int place = team_scan<W>(count, a);
    const int candidates = __shfl(place, W - 1, W);
    place -= count;
    uint64_t mask = 0;  // those that are not in the list yet, the first one in the highest bit
    if (__ballot(candidates > kList) == 0) {
        int32_t* entry = &list_expert[team][place];
#pragma unroll
        for (int j = 0; j < ITEMS; ++j)
            if (c[j] >= least) *entry++ = base + j;
    } else {
        sum_exactly();
#pragma unroll
        for (int j = 0; j < ITEMS; ++j) mask |= c[j] >= least ? 1ull << (ITEMS - 1 - j) : 0;
    }

    int taken = 0, held = 0;  // candidates that were in the list, entries that stay in it
    while (true) {
        while (mask != 0 && place - taken + held < kList) {
            const int high = 63 - __clzll(mask);
            mask ^= 1ull << high;
            list_expert[team][place++ - taken + held] = base + ITEMS - 1 - high;
        }
        wave_sync();
        const int entries = candidates - taken + held < kList ? candidates - taken + held : kList;
        const int passes = __ballot(entries > W) == 0 ? 1 : kList / W;  // (mostly 1)
        for (int p = 0; p < passes; ++p) {
            const int at = p * W + a;
            if (at >= held && at < entries)
                list_key[team][at] = choice64(list_expert[team][at], &list_part[team][at]);
            else if (at >= entries)
                list_key[team][at] = 0;
        }
        wave_sync();
        // among equal ones the lower place is the lower index: what stayed comes first
        for (int p = 0; p < passes; ++p) {
            const int at = p * W + a;
            const uint64_t mine = at < entries ? list_key[team][at] : 0;
            int rank = 0;
            for (int i = 0; i < entries; i += 4) {  // (kList is a multiple; what is behind the entries does not count)
                uint64_t other[4];
#pragma unroll
                for (int u = 0; u < 4; ++u) other[u] = list_key[team][i + u];
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    rank += other[u] > mine || (other[u] == mine && i + u < at);
            }
            if (at < entries && rank == g.k) chosen_key[team][rank] = mine;
            if (at < entries && rank < g.k) {
                chosen_key[team][rank] = mine;
                chosen_expert[team][rank] = mine != 0 ? list_expert[team][at] : -1;
                chosen_part[team][rank] = list_part[team][at];
            }
        }
        wave_sync();
        if (!exact) {  // (then all candidates are in the list)
            const bool close = a < g.k && a + 1 < entries &&
                               !(value_of(chosen_key[team][a]) - value_of(chosen_key[team][a + 1]) > (double)(kSumError * over));
            if (__ballot(close) != 0) {
                sum_exactly();
                continue;
            }
        }
        taken += entries - held;
        held = entries < g.k ? entries : g.k;
        if (__ballot(taken < candidates) == 0) break;
        if (a < held) {
            list_key[team][a] = chosen_key[team][a];
            list_expert[team][a] = chosen_expert[team][a];
            list_part[team][a] = chosen_part[team][a];
        }
        wave_sync();
    }

    // lane i < k has choice i (a team has k lanes at least)
    const bool mine = live && a < g.k;
    const int32_t expert = mine && a < held ? chosen_expert[team][a] : -1;
    double s = expert >= 0 ? chosen_part[team][a] : 0.0;
    if (!sigmoid && expert >= 0 && sum != sum) s = sum;  // (a NaN, or +infinity, makes all scores of the token NaN)
    if (renorm) {
        const double total = team_reduce<W>(s, [](double p, double q) { return p + q; });
        s = expert < 0 || total == 0.0 ? 0.0 : s / total;
    } else if (!sigmoid && expert >= 0) {
        // of binary32 in every token: `sum` may be another one here, where a token of the wave, this or another, had choices
        // close to each other
        s /= (double)sum32[team];
    }
    if (mine) {
        g.experts[token * g.k + a] = expert;
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
    if (items <= 8) return run_router<L, W, 8>(g, lanes_per_group, stream);
    if (items <= 16) return run_router<L, W, 16>(g, lanes_per_group, stream);
    if constexpr (W == 64) {
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
    // the narrowest team that has a lane for each choice and group and at most `items` experts per lane
    const auto team = [&](int items, int choices) {
        int W = 8;
        while (W < 64 && (W < choices || W < padded || size > items * (W / padded))) W *= 2;
        return W;
    };
    // A narrow team has less work per token (32768 tokens, 256 experts: 64 lanes 46 us, 32 27, 16 21) but a longer way
    // through it (1024 tokens: 6.9, 7.0, 9.9): taken where the waves fill the 1024 vector units once, or twice, and
    // where its list has room for 4 k candidates.
    int W = team(4, g.k);
    if (g.T * team(8, 2 * g.k) >= 1 * 1024 * 64) W = team(8, 2 * g.k);
    if (g.T * team(16, 2 * g.k) >= 2 * 1024 * 64) W = team(16, 2 * g.k);
    const int lanes = W / padded;
    const int items = (size + lanes - 1) / lanes;
    if (W == 8) return pick_items<L, 8>(g, items, lanes, stream);
    if (W == 16) return pick_items<L, 16>(g, items, lanes, stream);
    if (W == 32) return pick_items<L, 32>(g, items, lanes, stream);
    return pick_items<L, 64>(g, items, lanes, stream);
}

// ---------------------------------------------------------------------------
// Gradient.  With p_i = s_i / S over the choices (renormalised weights),
//   softmax   dl_i = scale p_i (g_i - sum_j p_j g_j), 0 elsewhere
//   sigmoid   dl_i = scale p_i (1 - s_i) (g_i - sum_j p_j g_j), or
//                    scale s_i (1 - s_i) g_i without renormalising
// depend on the chosen logits only: the others are not read.  Softmax weights
// as they are, and a gradient of the scores, take the whole row:
//   dl_e = s_e (ds_e - sum_f s_f ds_f), or s_e (1 - s_e) ds_e.
// A team of W lanes has a token: lane i < k its choice i, and each lane 8
// consecutive experts of every 8 W, which it stores in one piece.  The choices'
// parts find their experts through a row in LDS (comparing every expert with
// every choice took 32 us for the first of what follows).
// What bounds it: the latency of the gathered logits, and a launch.  Measured:
// 32768 tokens, 8 of 256 experts, sigmoid, renormalised, bf16 8 us (2.2 TB/s
// written); 4096 tokens, 8 of 128, softmax with a gradient of the scores 5.0.
// ---------------------------------------------------------------------------

// s(v) and 1 - s(v) of the sigmoid, each with its own relative precision.
__device__ __forceinline__ void sigmoid_pair(float v, float& s, float& rest) {
    const float e = exp_below(-fabsf(v)), r = __builtin_amdgcn_rcpf(1.0f + e);
    s = v < 0.0f ? e * r : r;
    rest = v < 0.0f ? r : e * r;
}

// CHUNKS: pieces of 8 experts per lane.
template <class L, int W, int CHUNKS>
__global__ __launch_bounds__(kThreads) void router_backward_kernel(RouterBackwardArgs g) {
    constexpr int kTeams = kThreads / W;
    __shared__ __attribute__((aligned(16))) float rows[kTeams][8 * W * CHUNKS];
    const int a = threadIdx.x & (W - 1);
    const int64_t token = (int64_t)blockIdx.x * kTeams + threadIdx.x / W;
    const bool live = token < g.T;
    const int64_t t = live ? token : 0;
    const L* const logits = (const L*)g.logits + t * g.ldl;
    float* const row = rows[threadIdx.x / W];
    const bool sigmoid = g.flags & MX_ROUTER_SIGMOID, renorm = g.flags & MX_ROUTER_RENORM;
    const bool direct = sigmoid || renorm;              // the choices' parts are gradients of their own logits only
    const bool dense = !direct || g.dscores != nullptr;  // the whole row is read
    const auto larger = [](float p, float q) { return fmaxf(p, q); };

    // the choices
    int32_t expert = live && a < g.k ? g.experts[t * g.k + a] : -1;
    if (expert < 0 || expert >= g.E) expert = -1;
    const float mine = expert >= 0 ? load_logit(logits + expert) : kLowest;
    float part = expert >= 0 ? g.dweights[t * g.k + a] : 0.0f;
    if (direct) {
        float s = 0.0f, rest = 1.0f;
        if (sigmoid) {
            if (expert >= 0) sigmoid_pair(mine, s, rest);
        } else {
            const float top = team_reduce<W>(mine, larger);
            if (mine != kLowest) s = exp_below(mine - top);  // (the softmax's sum cancels)
        }
        if (renorm) {
            float total = team_sum<W>(s);
            if (sigmoid && __ballot(!(total >= 0.5f)) != 0) {
                // All chosen logits of a token are negative: s over the largest one's e^l, so that no s has to be held; 0
                // where mx_router's sum is, of binary64 (1 + e^-l is infinite from here on).
                const float top = team_reduce<W>(mine, larger);
                const float over_top = top > -709.782715f ? exp_below(mine - top) * rest : mine != mine ? mine : 0.0f;
                const float sum = team_sum<W>(over_top);
                if (!(total >= 0.5f)) s = over_top, total = sum;
            }
            const float p = s == 0.0f ? 0.0f : s / total;
            const float average = team_sum<W>(p == 0.0f ? 0.0f : p * part);
            part = p == 0.0f ? 0.0f : p * (part - average);
        } else {
            part = s == 0.0f ? 0.0f : s * part;
        }
        part = mine == kLowest ? 0.0f : part * rest;
    }
    part *= g.scale;

    // to their experts; a repeated one gets the sum of its parts, in order
    if (expert >= 0) reinterpret_cast<int32_t*>(row)[expert] = a;
    wave_sync();
    const bool repeated = expert >= 0 && reinterpret_cast<int32_t*>(row)[expert] != a;
    bool writes = expert >= 0;
    if (__ballot(repeated) != 0) {
        float sum = 0.0f;
        for (int i = g.k - 1; i >= 0; --i) {
            const int32_t other = __shfl(expert, i, W);
            const float more = __shfl(part, i, W);
            if (other == expert) {
                sum += more;
                writes = expert >= 0 && i == a;  // (in the end: the first one)
            }
        }
        part = sum;
    }
    wave_sync();
#pragma unroll
    for (int c = 0; c < CHUNKS; ++c) {
        float4* const p = reinterpret_cast<float4*>(row + (c * W + a) * 8);
        p[0] = p[1] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    }
    wave_sync();
    if (writes) row[expert] = part;
    wave_sync();

    const auto load_dscores = [&](int c, float (&ds)[8]) {
        const int e = (c * W + a) * 8, here = !live ? 0 : g.E - e < 0 ? 0 : g.E - e < 8 ? g.E - e : 8;
        if (g.dscores != nullptr) load_logits<8>(g.dscores + t * g.E + e, here, ds);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (g.dscores == nullptr || j >= here) ds[j] = 0.0f;
    };
    float over = 0.0f, top = 0.0f, mean = 0.0f;
    float l[CHUNKS][8];
    if (dense) {
#pragma unroll
        for (int c = 0; c < CHUNKS; ++c) {
            const int e = (c * W + a) * 8, here = !live ? 0 : g.E - e < 0 ? 0 : g.E - e < 8 ? g.E - e : 8;
            load_logits<8>(logits + e, here, l[c]);
        }
        if (!sigmoid) {
            top = kLowest;
#pragma unroll
            for (int c = 0; c < CHUNKS; ++c)
#pragma unroll
                for (int j = 0; j < 8; ++j) top = fmaxf(top, l[c][j]);
            top = team_reduce<W>(top, larger);
            float sum = 0.0f, dot = 0.0f;
#pragma unroll
            for (int c = 0; c < CHUNKS; ++c) {
                float ds[8];
                load_dscores(c, ds);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float s = l[c][j] == kLowest ? 0.0f : exp_below(l[c][j] - top);
                    if (!direct) ds[j] += row[(c * W + a) * 8 + j];
                    sum += s;
                    dot += s == 0.0f ? 0.0f : s * ds[j];
                }
            }
            over = 1.0f / team_sum<W>(sum);
            mean = team_sum<W>(dot) * over;
        }
    }
#pragma unroll
    for (int c = 0; c < CHUNKS; ++c) {
        const int e = (c * W + a) * 8, here = !live ? 0 : g.E - e < 0 ? 0 : g.E - e < 8 ? g.E - e : 8;
        float out[8];
#pragma unroll
        for (int j = 0; j < 8; j += 4) {
            const float4 p = *reinterpret_cast<const float4*>(row + e + j);
            out[j] = p.x, out[j + 1] = p.y, out[j + 2] = p.z, out[j + 3] = p.w;
        }
        if (dense) {
            float ds[8];
            load_dscores(c, ds);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float v = l[c][j];
                if (!direct) ds[j] += out[j];
                float s, rest = 1.0f;
                if (sigmoid) sigmoid_pair(v, s, rest);
                else s = exp_below(v - top) * over;
                const float whole = sigmoid ? s * rest * ds[j] : s * (ds[j] - mean);
                out[j] = v == kLowest ? 0.0f : direct ? out[j] + whole : whole;
            }
        }
        if (here > 0) store_values<8>((L*)g.dlogits + t * g.ldd + e, here, out);
    }
}

template <class L, int W, int CHUNKS>
hipError_t run_backward(const RouterBackwardArgs& g, hipStream_t stream) {
    const int64_t blocks = (g.T + kThreads / W - 1) / (kThreads / W);
    hipLaunchKernelGGL((router_backward_kernel<L, W, CHUNKS>), dim3((unsigned)blocks), dim3(kThreads), 0, stream, g);
    return hipGetLastError();
}

// The narrowest team with a lane for each choice and at most 8 experts per lane.
template <class L>
hipError_t pick_backward(const RouterBackwardArgs& g, hipStream_t stream) {
    if (g.k <= 8 && g.E <= 64) return run_backward<L, 8, 1>(g, stream);
    if (g.k <= 16 && g.E <= 128) return run_backward<L, 16, 1>(g, stream);
    if (g.k <= 32 && g.E <= 256) return run_backward<L, 32, 1>(g, stream);
    if (g.E <= 512) return run_backward<L, 64, 1>(g, stream);
    if (g.E <= 1024) return run_backward<L, 64, 2>(g, stream);
    if (g.E <= 2048) return run_backward<L, 64, 4>(g, stream);
    return run_backward<L, 64, 8>(g, stream);
}

}  // namespace

hipError_t launch_router(const RouterArgs& a, hipStream_t stream) {
    return a.flags & MX_ROUTER_LOGITS_BF16 ? pick_team<uint16_t>(a, stream) : pick_team<float>(a, stream);
}

hipError_t launch_router_backward(const RouterBackwardArgs& a, hipStream_t stream) {
    return a.flags & MX_ROUTER_LOGITS_BF16 ? pick_backward<uint16_t>(a, stream) : pick_backward<float>(a, stream);
}

}  // namespace mx
