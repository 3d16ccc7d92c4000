// The optimizer step over many tensors at once: AdamW with states in 32 or
// in 8 bits, and the global norm of the gradients that clips it.
//
// Mathematics (fp32, per element; t = step count after this step, c = the
// gradients' factor):
//   g' = c g,  m = b1 m + (1 - b1) g',  v = b2 v + (1 - b2) g'^2
//   w  = [1 - lr d] w - [lr / (1 - b1^t)] (m / (sqrt(v) [1 / sqrt(1 - b2^t)] + eps))
// (the factors in brackets once a step, in double).
// 8-bit states hold m and sqrt(v) as E4M3 codes under one fp32 scale per 256
// elements, scale = max(amax, 2^-100) / 448.  sqrt(v) and not v: E4M3 spans
// 2^17.8 from its smallest code to 448, which is 2^35 in v.  The scale is a
// float and not a power of two so that it follows the block's largest value
// as that decays by less than a code's step; the other codes of the block
// keep their ratio to it.  Codes of v > 0 are never zero: m / eps would
// follow in a later step.
//
// Rounding of the codes.  To nearest, a state that changes by less than half
// a code's step (3 to 6 %) in a step of the optimizer does not change at all:
// sqrt(v) falls by 1 - sqrt(b2) at most, 2.5 % at 0.95 and 0.05 % at 0.999,
// and an element that is not its block's largest keeps its code for as long
// as that one keeps its value (a gradient that falls to a hundredth leaves v
// at 10^4 times what it should be, for good).  Tensors marked
// MX_ADAMW_UNBIASED round up or down at random, with the probabilities at
// which the expected values of m and of v (not of sqrt(v)) are the exact ones;
// both recursions are linear, so those of all later steps are too.  m as well:
// to nearest, 0.9 times a code of 4 units or fewer is that code again, and
// would move a weight without gradients for ever once its v has fallen.  The
// random numbers are a function of the step and the element's index: the same
// step gives the same bits.  Same time (1.16 ms, below): the vector units wait
// for HBM.
//
// What bounds it: HBM, with about as much written as read.  Nothing is read
// twice; per element 10 to 30 bytes move and 50 to 80 vector operations run
// (the vector units could run 180 in the time of 28 bytes).  Measured on 48
// tensors, 337 10^6 elements: float32 states, float32 masters, bf16 weights
// and gradients (28 bytes) 1.74-1.79 ms, 5.3 TB/s; 8-bit states, float32
// gradients (18 bytes) 1.16 ms, 5.2 TB/s; the norm of bf16 gradients 0.21 ms
// right after a step, whose written data then leaves the caches.  96 short
// tensors (115 10^3 elements): 8-11 us a step, 6.5 us the norm, latency.
//
// Layout: one launch for all tensors.  The plan cuts every tensor into
// chunks of 4096 elements and names the tensor of each; workgroups of 4
// waves take chunks with a stride of the grid, reading the plan ahead and all
// of a chunk before they store any of it.  A wave takes 256 consecutive
// elements at a time, 4 per lane, so that every load and store of a wave is
// one contiguous piece (256 B of codes to 1 KB of floats) and a block of an
// 8-bit state is exactly one wave: its maximum is a reduction in registers.
#include <type_traits>

#include "mx_train.h"

namespace mx {
namespace {

constexpr int kThreads = 256;
constexpr int kPer = 4;                                 // elements per lane and block
constexpr int kBlocks = kAdamwChunk / (64 * kPer) / 4;  // blocks of 256 per wave and chunk
static_assert(64 * kPer == MX_ADAMW_BLOCK, "a wave is a block");

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// Constants of a step, the same in every lane.
struct Step {
    float c;          // factor of the gradients
    float b1, a1;     // beta1, 1 - beta1
    float b2, a2;     // beta2, 1 - beta2
    double lr;
    float size;       // lr / (1 - beta1^t)
    float root;       // 1 / sqrt(1 - beta2^t)
    float eps;
    uint32_t key;     // random numbers of the step
};

// A mixing of 32 bits (one to one): shifts and products with odd numbers, the
// fractions of the square roots of 2 and 3.
__device__ __forceinline__ uint32_t mixed(uint32_t x) {
    x = (x ^ (x >> 16)) * 0x6A09E667u;
    x = (x ^ (x >> 15)) * 0xBB67AE85u;
    return x ^ (x >> 16);
}
// Of step t, and of element i in it.
__device__ __forceinline__ uint32_t step_key(int64_t t) {
    return mixed((uint32_t)t * 0x9E3779B1u + mixed((uint32_t)((uint64_t)t >> 32)));
}
__device__ __forceinline__ uint32_t element_bits(uint32_t key, int64_t i) {
    return mixed((uint32_t)i + key + (uint32_t)((uint64_t)i >> 32) * 0x9E3779B1u);
}

__device__ __forceinline__ double power(double b, int64_t t) {
    double r = 1.0;
    for (uint64_t e = (uint64_t)t; e != 0; e >>= 1, b *= b)
        if (e & 1) r *= b;
    return r;
}

// Largest value over the wave's 64 lanes (non-negative values).
__device__ __forceinline__ float wave_max(float v) {
    const auto dpp = [](float x, auto ctrl) {
        return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, x), decltype(ctrl)::value,
                                                                  0xF, 0xF, false));
    };
    v = fmaxf(v, dpp(v, std::integral_constant<int, 0xB1>{}));   // quad_perm [1,0,3,2]
    v = fmaxf(v, dpp(v, std::integral_constant<int, 0x4E>{}));   // quad_perm [2,3,0,1]
    v = fmaxf(v, dpp(v, std::integral_constant<int, 0x141>{}));  // row_half_mirror
    v = fmaxf(v, dpp(v, std::integral_constant<int, 0x140>{}));  // row_mirror
    const uint32_t a = __builtin_bit_cast(uint32_t, v);
    const auto p = __builtin_amdgcn_permlane16_swap(a, a, false, false);
    v = fmaxf(__builtin_bit_cast(float, (uint32_t)p[0]), __builtin_bit_cast(float, (uint32_t)p[1]));
    const uint32_t b = __builtin_bit_cast(uint32_t, v);
    const auto q = __builtin_amdgcn_permlane32_swap(b, b, false, false);
    return fmaxf(__builtin_bit_cast(float, (uint32_t)q[0]), __builtin_bit_cast(float, (uint32_t)q[1]));
}

// 4 consecutive elements from i on, as float.  `live`: how many of them exist
// (0 to 4); the others read as zero.  With `fast` all 4 exist and are aligned.
__device__ __forceinline__ void load4(const float* p, int64_t i, int live, bool fast, float (&v)[4]) {
    if (fast) {
        const f32x4 x = __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(p + i));
        for (int e = 0; e < 4; ++e) v[e] = x[e];
    } else {
        for (int e = 0; e < 4; ++e) v[e] = e < live ? p[i + e] : 0.0f;
    }
}
__device__ __forceinline__ void load4(const uint16_t* p, int64_t i, int live, bool fast, float (&v)[4]) {
    if (fast) {
        const u32x2 x = __builtin_nontemporal_load(reinterpret_cast<const u32x2*>(p + i));
        v[0] = __builtin_bit_cast(float, x[0] << 16);
        v[1] = __builtin_bit_cast(float, x[0] & 0xFFFF0000u);
        v[2] = __builtin_bit_cast(float, x[1] << 16);
        v[3] = __builtin_bit_cast(float, x[1] & 0xFFFF0000u);
    } else {
        for (int e = 0; e < 4; ++e) v[e] = e < live ? __builtin_bit_cast(float, (uint32_t)p[i + e] << 16) : 0.0f;
    }
}
__device__ __forceinline__ uint32_t load_codes(const uint8_t* p, int64_t i, int live, bool fast) {
    if (fast) return __builtin_nontemporal_load(reinterpret_cast<const uint32_t*>(p + i));
    uint32_t x = 0;
    for (int e = 0; e < 4; ++e) x |= (e < live ? (uint32_t)p[i + e] : 0u) << (8 * e);
    return x;
}
__device__ __forceinline__ void store4(float* p, int64_t i, int live, bool fast, const float (&v)[4]) {
    if (fast) {
        __builtin_nontemporal_store(f32x4{v[0], v[1], v[2], v[3]}, reinterpret_cast<f32x4*>(p + i));
    } else {
        for (int e = 0; e < 4; ++e)
            if (e < live) p[i + e] = v[e];
    }
}
// rounded to nearest even (the weights' only rounding to fewer bits)
__device__ __forceinline__ void store4(uint16_t* p, int64_t i, int live, bool fast, const float (&v)[4]) {
    uint16_t b[4];
    for (int e = 0; e < 4; ++e) b[e] = __builtin_bit_cast(uint16_t, (__bf16)v[e]);
    if (fast) {
        const u32x2 x{(uint32_t)b[0] | ((uint32_t)b[1] << 16), (uint32_t)b[2] | ((uint32_t)b[3] << 16)};
        __builtin_nontemporal_store(x, reinterpret_cast<u32x2*>(p + i));
    } else {
        for (int e = 0; e < 4; ++e)
            if (e < live) p[i + e] = b[e];
    }
}
__device__ __forceinline__ void store_codes(uint8_t* p, int64_t i, int live, bool fast, uint32_t x) {
    if (fast) {
        __builtin_nontemporal_store(x, reinterpret_cast<uint32_t*>(p + i));
    } else {
        for (int e = 0; e < 4; ++e)
            if (e < live) p[i + e] = (uint8_t)(x >> (8 * e));
    }
}

__device__ __forceinline__ void decode4(uint32_t x, float (&v)[4]) {
    const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)x, false);
    const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)x, true);
    v[0] = lo[0];
    v[1] = lo[1];
    v[2] = hi[0];
    v[3] = hi[1];
}
__device__ __forceinline__ uint32_t encode4(const float (&v)[4]) {
    int x = __builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[1], 0, false);
    x = __builtin_amdgcn_cvt_pk_fp8_f32(v[2], v[3], x, true);
    return (uint32_t)x;
}

constexpr float kTiny = 0x1p-100f;  // smallest block maximum that a scale is made for
constexpr float kTop = 448.0f;      // largest E4M3 value
constexpr float kLeast = 0x1p-9f;   // smallest E4M3 value

// Value scaled for a code: not past the largest one (x / amax may round
// up); a NaN passes.
__device__ __forceinline__ float in_range(float y) { return y > kTop ? kTop : (y < -kTop ? -kTop : y); }

// E4M3 values have 3 bits after the leading one and a smallest step of 2^-9:
// the neighbours of y >= 0 are those of y + 2^-6 with 3 bits kept where
// y < 2^-6 (2^-6 has the step 2^-9).  u: 16 random bits.  Exact values stay.
__device__ __forceinline__ float e4m3_shift(float y) { return y < 0x1p-6f ? 0x1p-6f : 0.0f; }

// |y| rounded to a neighbour, with expected value y; y's sign.
__device__ __forceinline__ float round_unbiased(float y, uint32_t u) {
#pragma clang fp contract(off)
    const float shift = e4m3_shift(fabsf(y));
    const uint32_t b = (__builtin_bit_cast(uint32_t, fabsf(y) + shift) + (u << 4 | 8u)) & ~0xFFFFFu;
    const float r = copysignf(__builtin_bit_cast(float, b) - shift, y);
    return y == y ? r : y;
}
// y >= 0 rounded to a neighbour, with expected square y^2.
__device__ __forceinline__ float round_square_unbiased(float y, uint32_t u) {
#pragma clang fp contract(off)
    const float shift = e4m3_shift(y);
    const uint32_t b = __builtin_bit_cast(uint32_t, y + shift) & ~0xFFFFFu;
    const float lo = __builtin_bit_cast(float, b) - shift, hi = __builtin_bit_cast(float, b + 0x100000u) - shift;
    const float p = ((float)u + 0.5f) * 0x1p-16f;
    const float r = p * ((hi - lo) * (hi + lo)) < (y - lo) * (y + lo) ? hi : lo;
    return y == y ? r : y;
}

// A block's values in a lane, as they are in memory.
template <int W, bool GB, bool S8>
struct Block {
    float g[4], m[4], v[4], w[4];
    uint32_t mc, vc;
    float ms, vs;

    __device__ __forceinline__ void load(const mx_adamw_tensor& t, int64_t block, int64_t i, int live, bool fast) {
        typedef typename std::conditional<GB, uint16_t, float>::type grad_t;
        load4((const grad_t*)t.g, i, live, fast, g);
        if (S8) {
            ms = t.m_scale[block];
            vs = t.v_scale[block];
            mc = load_codes((const uint8_t*)t.m, i, live, fast);
            vc = load_codes((const uint8_t*)t.v, i, live, fast);
        } else {
            load4((const float*)t.m, i, live, fast, m);
            load4((const float*)t.v, i, live, fast, v);
        }
        if (W == 0) load4((const float*)t.w, i, live, fast, w);
        if (W == 1) load4(t.master, i, live, fast, w);
        if (W == 2) load4((const uint16_t*)t.w, i, live, fast, w);
    }

    __device__ __forceinline__ void step_and_store(const mx_adamw_tensor& t, const Step& s, float keep, int64_t block,
                                                   int64_t i, int live, bool fast, int lane) {
        // every operation rounded by itself: which of them would be fused is
        // the compiler's choice otherwise, and a code of the next step could
        // hang on it
#pragma clang fp contract(off)
        if (S8) {
            decode4(mc, m);
            decode4(vc, v);
        }
        float r[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (S8) {
                m[e] *= ms;
                v[e] *= vs;
                v[e] *= v[e];
            }
            const float x = g[e] * s.c;
            m[e] = s.b1 * m[e] + s.a1 * x;
            v[e] = s.b2 * v[e] + s.a2 * (x * x);
            r[e] = __builtin_sqrtf(v[e]);
            const float update = m[e] / (r[e] * s.root + s.eps);
            w[e] = keep * w[e] - s.size * update;
        }
        if (W == 0) store4((float*)t.w, i, live, fast, w);
        if (W == 1) store4(t.master, i, live, fast, w);
        if (W != 0) store4((uint16_t*)t.w, i, live, fast, w);
        if (!S8) {
            store4((float*)t.m, i, live, fast, m);
            store4((float*)t.v, i, live, fast, v);
            return;
        }
        float am = 0.0f, av = 0.0f;  // (lanes past the end hold zeros)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            am = fmaxf(am, fabsf(m[e]));
            av = fmaxf(av, r[e]);
        }
        am = fmaxf(wave_max(am), kTiny);
        av = fmaxf(wave_max(av), kTiny);
        const float im = 1.0f / am * kTop, iv = 1.0f / av * kTop;
        const bool unbiased = (t.types & MX_ADAMW_UNBIASED) != 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            m[e] = in_range(m[e] * im);
            float y = in_range(r[e] * iv);
            const bool least = r[e] > 0.0f && y < kLeast;
            if (unbiased) {
                const uint32_t bits = element_bits(s.key, i + e);
                m[e] = round_unbiased(m[e], bits & 0xFFFFu);
                y = round_square_unbiased(y, bits >> 16);
            }
            v[e] = least ? kLeast : y;
        }
        store_codes((uint8_t*)t.m, i, live, fast, encode4(m));
        store_codes((uint8_t*)t.v, i, live, fast, encode4(v));
        if (lane == 0) {
            t.m_scale[block] = am * (1.0f / kTop);
            t.v_scale[block] = av * (1.0f / kTop);
        }
    }
};

// One chunk of one tensor.  W: 0 float32 weights, 1 bf16 weights with
// float32 masters, 2 bf16 weights alone.  A whole aligned chunk reads all of
// its blocks before it stores the first one (a load is not moved over a
// store by itself: they could be to the same memory).
template <int W, bool GB, bool S8>
__device__ __forceinline__ void step_chunk(const mx_adamw_tensor& t, int64_t chunk, const Step& s, int wave, int lane) {
    const float keep = (float)(1.0 - s.lr * (double)t.weight_decay);
    const int64_t block0 = chunk * (kAdamwChunk / MX_ADAMW_BLOCK) + wave;
    if ((t.types & kAdamwAligned) != 0 && (chunk + 1) * kAdamwChunk <= t.n) {
        Block<W, GB, S8> b[kBlocks];
#pragma unroll
        for (int u = 0; u < kBlocks; ++u)
            b[u].load(t, block0 + 4 * u, (block0 + 4 * u) * MX_ADAMW_BLOCK + lane * kPer, 4, true);
#pragma unroll
        for (int u = 0; u < kBlocks; ++u)
            b[u].step_and_store(t, s, keep, block0 + 4 * u, (block0 + 4 * u) * MX_ADAMW_BLOCK + lane * kPer, 4, true,
                                lane);
        return;
    }
    // a tensor's end, or any alignment: the same, element by element where
    // 4 do not exist or are not aligned
    const bool vec = (t.types & kAdamwAligned) != 0;
    Block<W, GB, S8> b[kBlocks];
    const auto live_of = [&](int u) {
        const int64_t left = t.n - (block0 + 4 * u) * MX_ADAMW_BLOCK - lane * kPer;
        return left >= 4 ? 4 : (left > 0 ? (int)left : 0);
    };
#pragma unroll
    for (int u = 0; u < kBlocks; ++u) {
        const int64_t block = block0 + 4 * u;
        if (block * MX_ADAMW_BLOCK < t.n)  // the same in every lane of the wave
            b[u].load(t, block, block * MX_ADAMW_BLOCK + lane * kPer, live_of(u), vec && live_of(u) == 4);
    }
#pragma unroll
    for (int u = 0; u < kBlocks; ++u) {
        const int64_t block = block0 + 4 * u;
        if (block * MX_ADAMW_BLOCK < t.n)
            b[u].step_and_store(t, s, keep, block, block * MX_ADAMW_BLOCK + lane * kPer, live_of(u),
                                vec && live_of(u) == 4, lane);
    }
}

template <int W, bool GB>
__device__ __forceinline__ void step_state(const mx_adamw_tensor& t, int64_t chunk, const Step& s, int wave, int lane) {
    if (t.types & MX_ADAMW_STATE_8BIT) step_chunk<W, GB, true>(t, chunk, s, wave, lane);
    else step_chunk<W, GB, false>(t, chunk, s, wave, lane);
}
template <int W>
__device__ __forceinline__ void step_grad(const mx_adamw_tensor& t, int64_t chunk, const Step& s, int wave, int lane) {
    if (t.types & MX_ADAMW_G_BF16) step_state<W, true>(t, chunk, s, wave, lane);
    else step_state<W, false>(t, chunk, s, wave, lane);
}

// The chunks k = first, first + stride, ... of a workgroup.  What the plan
// says of a chunk is read ahead (its tensor two chunks ahead, the tensor's
// entry one), by scalar loads: the plan is constant while a kernel runs.
typedef const __attribute__((address_space(4))) AdamwEntry* entry_ptr;
typedef const __attribute__((address_space(4))) int32_t* owner_ptr;
template <typename F>
__device__ __forceinline__ void for_chunks(const AdamwEntry* entries, const int32_t* owner, int64_t chunks, F work) {
    const entry_ptr ep = (entry_ptr)entries;
    const owner_ptr op = (owner_ptr)owner;
    int64_t k = blockIdx.x;
    const int64_t stride = gridDim.x;
    if (k >= chunks) return;
    const auto entry_of = [&](int32_t i) {
        AdamwEntry e;
        e.t.w = ep[i].t.w;
        e.t.master = ep[i].t.master;
        e.t.g = ep[i].t.g;
        e.t.m = ep[i].t.m;
        e.t.v = ep[i].t.v;
        e.t.m_scale = ep[i].t.m_scale;
        e.t.v_scale = ep[i].t.v_scale;
        e.t.n = ep[i].t.n;
        e.t.weight_decay = ep[i].t.weight_decay;
        e.t.types = ep[i].t.types;
        e.first_chunk = ep[i].first_chunk;
        return e;
    };
    AdamwEntry e = entry_of(op[k]);
    int32_t next = k + stride < chunks ? op[k + stride] : 0;
    for (; k < chunks; k += stride) {
        const AdamwEntry ahead = entry_of(next);
        next = k + 2 * stride < chunks ? op[k + 2 * stride] : 0;
        work(e.t, k - e.first_chunk);
        e = ahead;
    }
}

__global__ __launch_bounds__(kThreads) void adamw_kernel(AdamwArgs a) {
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const float c = a.grad_scale ? *a.grad_scale : 1.0f;
    const bool skip = !(c >= 0.0f && c <= __FLT_MAX__);
    const int64_t done = *a.steps;
    const int64_t t = done + 1;
    Step s;
    s.c = c;
    s.b1 = (float)a.beta1;
    s.a1 = (float)(1.0 - a.beta1);
    s.b2 = (float)a.beta2;
    s.a2 = (float)(1.0 - a.beta2);
    const double lr = a.lr_device ? (double)*a.lr_device : a.lr;
    s.lr = lr;
    s.size = (float)(lr / (1.0 - power(a.beta1, t)));
    s.root = (float)(1.0 / sqrt(1.0 - power(a.beta2, t)));
    s.eps = (float)a.eps;
    s.key = step_key(t);
    if (!skip)
        for_chunks(a.entries, a.owner, a.chunks, [&](const mx_adamw_tensor& tensor, int64_t chunk) {
            if (!(tensor.types & MX_ADAMW_W_BF16)) step_grad<0>(tensor, chunk, s, wave, lane);
            else if (tensor.master) step_grad<1>(tensor, chunk, s, wave, lane);
            else step_grad<2>(tensor, chunk, s, wave, lane);
        });
    // Every wave has read the count when its workgroup draws a ticket here;
    // the last workgroup to draw one raises it.
    __syncthreads();
    if (threadIdx.x == 0) {
        asm volatile("" ::"s"(done) : "memory");  // (the count is in a register by now)
        const int64_t ticket = __hip_atomic_fetch_add(a.steps + 1, (int64_t)1, __ATOMIC_RELAXED,
                                                      __HIP_MEMORY_SCOPE_AGENT);
        if (ticket == (int64_t)gridDim.x - 1) {
            __hip_atomic_store(a.steps + 1, (int64_t)0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            if (!skip) __hip_atomic_store(a.steps, t, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
    }
}

// Sum of squares of one chunk, in double: squares of finite gradients do not
// overflow there, and a sum over 10^9 elements keeps far more than the 24
// bits of the result.
template <typename T>
__device__ __forceinline__ void norm_chunk(const mx_adamw_tensor& t, int64_t chunk, double& sum) {
    constexpr int kWide = 16 / sizeof(T), kLoads = kAdamwChunk / (kThreads * kWide);
    const T* const g = (const T*)t.g;
    const int64_t first = chunk * kAdamwChunk;
    const auto add = [&](float x) { sum = fma((double)x, (double)x, sum); };
    if (((uintptr_t)g & 15) == 0 && first + kAdamwChunk <= t.n) {
        uint4 x[kLoads];
#pragma unroll
        for (int u = 0; u < kLoads; ++u) {
            // (an ordinary load: what stays in the caches is read again by the step.  With a
            // non-temporal one this kernel is 5 % faster and the step after it 2.5 % slower,
            // 1.96 against 2.00 ms for both at 337 10^6 gradients)
            x[u] = *(const uint4*)(g + first + (u * kThreads + threadIdx.x) * kWide);
        }
#pragma unroll
        for (int u = 0; u < kLoads; ++u)
            for (uint32_t w : {x[u].x, x[u].y, x[u].z, x[u].w}) {
                if (sizeof(T) == 4) {
                    add(__builtin_bit_cast(float, w));
                } else {
                    add(__builtin_bit_cast(float, w << 16));
                    add(__builtin_bit_cast(float, w & 0xFFFF0000u));
                }
            }
        return;
    }
    constexpr int kEach = kAdamwChunk / kThreads;  // a tensor's end, or any alignment
    T x[kEach];
#pragma unroll
    for (int u = 0; u < kEach; ++u) {
        const int64_t i = first + u * kThreads + threadIdx.x;
        x[u] = i < t.n ? g[i] : (T)0;
    }
#pragma unroll
    for (int u = 0; u < kEach; ++u) {
        if constexpr (sizeof(T) == 4) add(x[u]);
        else add(__builtin_bit_cast(float, (uint32_t)x[u] << 16));
    }
}

// Sum over the workgroup (valid in thread 0), in a fixed order.
__device__ __forceinline__ double group_sum(double v, double* part) {
    for (int d = 32; d > 0; d >>= 1) v += __shfl_down(v, d, 64);
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
    __syncthreads();
    return part[0] + part[1] + part[2] + part[3];
}

// Each workgroup sums the chunks k = blockIdx, blockIdx + grid, ... in order;
// the last one to finish sums the workgroups' results in order.
__global__ __launch_bounds__(kThreads) void grad_norm_kernel(const AdamwEntry* entries, const int32_t* owner,
                                                             int64_t chunks, float max_norm, NormWorkspace* ws,
                                                             float* out) {
    __shared__ double part[4], part2[4];
    __shared__ bool last;
    double sum = 0.0;
    for_chunks(entries, owner, chunks, [&](const mx_adamw_tensor& t, int64_t chunk) {
        if (t.types & MX_ADAMW_G_BF16) norm_chunk<uint16_t>(t, chunk, sum);
        else norm_chunk<float>(t, chunk, sum);
    });
    const double total = group_sum(sum, part);
    if (threadIdx.x == 0) {
        __hip_atomic_store(ws->part + blockIdx.x, total, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        last = __hip_atomic_fetch_add(&ws->ticket, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) == gridDim.x - 1;
    }
    __syncthreads();
    if (!last) return;
    double v = 0.0;
    for (int k = threadIdx.x; k < (int)gridDim.x; k += kThreads)
        v += __hip_atomic_load(ws->part + k, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    const double all = group_sum(v, part2);
    if (threadIdx.x == 0) {
        const double norm = sqrt(all);
        const float rounded = (float)norm;
        out[0] = rounded;
        // (one division: the reciprocal of a norm below 2^-128 is infinite)
        out[1] = rounded <= __FLT_MAX__ ? fminf(max_norm / rounded, 1.0f) : __builtin_nanf("");
        __hip_atomic_store(&ws->ticket, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
}

}  // namespace

hipError_t launch_adamw(const AdamwArgs& a, hipStream_t stream) {
    // 32 workgroups per CU: with 8 (all of them resident at once) 3 % slower,
    // the last chunks of the fastest ones leave the others' unread
    const int64_t most = 8192;
    const unsigned grid = (unsigned)(a.chunks < 1 ? 1 : (a.chunks < most ? a.chunks : most));
    hipLaunchKernelGGL(adamw_kernel, dim3(grid), dim3(kThreads), 0, stream, a);
    return hipGetLastError();
}

hipError_t launch_grad_norm(const AdamwEntry* entries, const int32_t* owner, int64_t chunks, float max_norm,
                            NormWorkspace* ws, float* out, hipStream_t stream) {
    const unsigned grid = (unsigned)(chunks < 1 ? 1 : (chunks < kNormParts ? chunks : kNormParts));
    hipLaunchKernelGGL(grad_norm_kernel, dim3(grid), dim3(kThreads), 0, stream, entries, owner, chunks, max_norm, ws,
                       out);
    return hipGetLastError();
}

}  // namespace mx
