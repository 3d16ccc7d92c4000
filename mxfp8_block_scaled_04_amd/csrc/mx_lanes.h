// Reductions over teams of W neighbouring lanes (W = 1, 2, 4, ... 64, teams
// aligned to W) in registers: after step d every lane of an aligned block of
// 2 d lanes holds that block's result, so that the next step can exchange with
// any lane of the other half (mirrored rows in place of xor).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mx {

// v of a lane in the other half of the aligned block of 2 D lanes.
template <int D>
__device__ __forceinline__ uint32_t other_half(uint32_t v) {
    static_assert(D == 1 || D == 2 || D == 4 || D == 8, "inside a row of 16 lanes");
    constexpr int ctrl = D == 1 ? 0xB1 : D == 2 ? 0x4E : D == 4 ? 0x141 : 0x140;  // quad_perm, half mirror, mirror
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, ctrl, 0xF, 0xF, true);  // (no lane reads outside its row)
}

// op(v, v of the other half) with op commutative; T of 4 or 8 bytes.
template <int D, class T, class Op>
__device__ __forceinline__ T joined(T v, Op op) {
    constexpr int words = sizeof(T) / 4;
    static_assert(sizeof(T) == 4 || sizeof(T) == 8, "whole registers");
    struct Words {
        uint32_t w[words];
    };
    const Words in = __builtin_bit_cast(Words, v);
    Words a, b;
#pragma unroll
    for (int i = 0; i < words; ++i) {
        if constexpr (D <= 8) {
            a.w[i] = in.w[i];
            b.w[i] = other_half<D>(in.w[i]);
        } else if constexpr (D == 16) {
            const auto p = __builtin_amdgcn_permlane16_swap(in.w[i], in.w[i], false, false);
            a.w[i] = p[0];
            b.w[i] = p[1];
        } else {
            const auto p = __builtin_amdgcn_permlane32_swap(in.w[i], in.w[i], false, false);
            a.w[i] = p[0];
            b.w[i] = p[1];
        }
    }
    return op(__builtin_bit_cast(T, a), __builtin_bit_cast(T, b));
}

// The team's result in all of its lanes.
template <int W, class T, class Op>
__device__ __forceinline__ T team_reduce(T v, Op op) {
    if constexpr (W >= 2) v = joined<1>(v, op);
    if constexpr (W >= 4) v = joined<2>(v, op);
    if constexpr (W >= 8) v = joined<4>(v, op);
    if constexpr (W >= 16) v = joined<8>(v, op);
    if constexpr (W >= 32) v = joined<16>(v, op);
    if constexpr (W >= 64) v = joined<32>(v, op);
    return v;
}
// The same where W is known at run time only (and the same in all lanes).
template <class T, class Op>
__device__ __forceinline__ T team_reduce(T v, int W, Op op) {
    if (W >= 2) v = joined<1>(v, op);
    if (W >= 4) v = joined<2>(v, op);
    if (W >= 8) v = joined<4>(v, op);
    if (W >= 16) v = joined<8>(v, op);
    if (W >= 32) v = joined<16>(v, op);
    if (W >= 64) v = joined<32>(v, op);
    return v;
}

template <int W>
__device__ __forceinline__ float team_sum(float v) {
    return team_reduce<W>(v, [](float a, float b) { return a + b; });
}

}  // namespace mx
