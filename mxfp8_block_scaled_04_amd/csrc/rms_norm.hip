// Root-mean-square norm with the residual's addition before it and an MXFP8
// copy of its output, and its gradients (include/libmxmoe_block.h).
//
// Mathematics per row of N columns: h = x + residual (rounded to the stream's
// type), r = 1 / sqrt(mean(h^2) + eps), y = bf16(h r w), MXFP8 of y as
// quantize_rows_kernel has it.  Backward with g = dy + dy2, a = g w, z = h r:
// dh = dh_in + r (a - z mean(a z)), dw = sum over rows of g z.
//
// One pass: a row stays in the registers of its team of lanes, 8 columns a
// lane and vector, from the loads to the stores; the sum over the row is a
// reduction in registers and, for teams of several waves, LDS.
#include "mx_bf16.h"
#include "mx_block.h"
#include "mx_device.h"
#include "mx_lanes.h"

namespace mx {
namespace {

struct Eight {
    float v[8];
};

__device__ __forceinline__ Eight unpack(uint4 d) {
    return Eight{{lo_bf16(d.x), hi_bf16(d.x), lo_bf16(d.y), hi_bf16(d.y), lo_bf16(d.z), hi_bf16(d.z), lo_bf16(d.w),
                  hi_bf16(d.w)}};
}
__device__ __forceinline__ uint4 pack(const Eight& e) {
    return make_uint4(pack_bf16(e.v[0], e.v[1]), pack_bf16(e.v[2], e.v[3]), pack_bf16(e.v[4], e.v[5]),
                      pack_bf16(e.v[6], e.v[7]));
}
__device__ __forceinline__ Eight load8(const uint16_t* p) { return unpack(*reinterpret_cast<const uint4*>(p)); }
__device__ __forceinline__ Eight load8(const float* p) {
    const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
    return Eight{{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}};
}
// Rounded to the stream's type, in place, and stored.
__device__ __forceinline__ void store8(uint16_t* p, Eight& e) {
    const uint4 d = pack(e);
    *reinterpret_cast<uint4*>(p) = d;
    e = unpack(d);
}
__device__ __forceinline__ void store8(float* p, Eight& e) {
    *reinterpret_cast<float4*>(p) = make_float4(e.v[0], e.v[1], e.v[2], e.v[3]);
    *reinterpret_cast<float4*>(p + 4) = make_float4(e.v[4], e.v[5], e.v[6], e.v[7]);
}

constexpr int kMaxWaves = 16;

// The team's sum in all of its lanes.  LANES: 16, 32, 64 (several teams per
// workgroup), or 0: the workgroup is the team (`buffer`: one float per wave,
// another one in the next call, so that one barrier is enough).
template <int LANES>
__device__ __forceinline__ float row_sum(float v, float* buffer) {
    if constexpr (LANES > 0) return team_sum<LANES>(v);
    v = team_sum<64>(v);
    const int waves = blockDim.x >> 6;
    if ((threadIdx.x & 63) == 0) buffer[threadIdx.x >> 6] = v;
    __syncthreads();
    float all = 0.0f;
    for (int w = 0; w < waves; ++w) all += buffer[w];
    return all;
}

// S: the stream's type, WT: the weight's (uint16_t: bf16).
template <class S, class WT, int LANES, int V>
__global__ __launch_bounds__(LANES > 0 ? 256 : 64 * kMaxWaves) void rms_norm_kernel(NormArgs g, int64_t rows) {
    __shared__ float buffer[2][kMaxWaves];
    const int team = LANES > 0 ? LANES : blockDim.x;
    const int a = LANES > 0 ? threadIdx.x & (LANES - 1) : threadIdx.x;
    const int64_t teams = LANES > 0 ? 256 / LANES : 1;
    const int64_t mine = LANES > 0 ? threadIdx.x / LANES : 0;
    const int64_t N = g.N;
    int turn = 0;
    for (int64_t r0 = (int64_t)blockIdx.x * teams; r0 < rows; r0 += (int64_t)gridDim.x * teams, turn ^= 1) {
        const int64_t row = r0 + mine;
        const bool live = row < g.M;
        Eight h[V];
        float sum = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int64_t c = (int64_t)(v * team + a) * 8;
            h[v] = Eight{};
            if (live && c < N) {
                if (g.residual != nullptr) {
                    h[v] = load8((const uint16_t*)g.x + row * g.ldx + c);
                    const Eight r = load8((const S*)g.residual + row * g.ldr + c);
#pragma unroll
                    for (int i = 0; i < 8; ++i) h[v].v[i] += r.v[i];
                    store8((S*)g.h + row * g.ldh + c, h[v]);
                } else {
                    h[v] = load8((const S*)g.x + row * g.ldx + c);
                }
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) sum = __builtin_fmaf(h[v].v[i], h[v].v[i], sum);
        }
        sum = row_sum<LANES>(sum, buffer[turn]);
        const float r = 1.0f / sqrtf(sum / (float)N + g.eps);
        if (g.rstd != nullptr && live && a == 0) g.rstd[row] = r;
        if (g.y == nullptr && g.q == nullptr) continue;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int64_t c = (int64_t)(v * team + a) * 8;
            uint4 out = make_uint4(0, 0, 0, 0);
            if (live && c < N) {
                const Eight w = load8((const WT*)g.weight + c);
                Eight e;
#pragma unroll
                for (int i = 0; i < 8; ++i) e.v[i] = h[v].v[i] * r * w.v[i];
                out = pack(e);
                if (g.y != nullptr) store16(g.y + row * g.ldy + c, out);
            }
            if (g.q == nullptr) continue;
            const uint32_t scale = scale_from_maxmag(quad_max_u32(max_mag8(out)));
            if (live && c < N) mx::store8(g.q + row * N + c, quant8(out, scale));
            // the unit's scale bytes of this row: two dwords, of the even and
            // the odd blocks, byte b / 2; 4 lanes have a block, 32 a unit
            const int in_unit = threadIdx.x & (LANES == 16 ? 15 : 31), b = in_unit >> 2;
            uint32_t word = scale << (8 * (b >> 1));
            word |= (uint32_t)__builtin_amdgcn_mov_dpp((int)word, 0x128, 0xF, 0xF, false);  // row_ror:8 (block b ^ 2)
            if constexpr (LANES != 16) {
                const auto p = __builtin_amdgcn_permlane16_swap(word, word, false, false);  // block b ^ 4
                word = p[0] | p[1];
            }
            const int64_t unit = c / 256, units = (N + 255) / 256;
            if ((in_unit == 0 || in_unit == 4) && unit < units && row < rows)
                *reinterpret_cast<uint32_t*>(g.s + row / 32 * 256 * units + unit * 256 +
                                             4 * (32 * (b & 1) + row % 32)) = word;
        }
    }
}

template <class S, class WT, int LANES, int V>
hipError_t run_norm(const NormArgs& g, int threads, hipStream_t stream) {
    const int64_t rows = g.q != nullptr ? (g.M + 31) / 32 * 32 : g.M;  // with the padding rows of the scales
    const int64_t teams = LANES > 0 ? 256 / LANES : 1;
    int64_t blocks = (rows + teams - 1) / teams;
    if (blocks > (1 << 20)) blocks = 1 << 20;
    hipLaunchKernelGGL((rms_norm_kernel<S, WT, LANES, V>), dim3((unsigned)blocks), dim3(threads), 0, stream, g, rows);
    return hipGetLastError();
}

template <class S, class WT>
hipError_t pick_norm(const NormArgs& g, hipStream_t stream) {
    const int64_t vectors = g.N / 8;
    if (vectors <= 16) return run_norm<S, WT, 16, 1>(g, 256, stream);
    if (vectors <= 32) return run_norm<S, WT, 32, 1>(g, 256, stream);
    if (vectors <= 64) return run_norm<S, WT, 64, 1>(g, 256, stream);
    if (vectors <= 128) return run_norm<S, WT, 64, 2>(g, 256, stream);
    const auto threads = [&](int V) { return (int)((vectors + 64 * V - 1) / (64 * V)) * 64; };
    if (vectors <= 64 * kMaxWaves) return run_norm<S, WT, 0, 1>(g, threads(1), stream);
    if (vectors <= 2 * 64 * kMaxWaves) return run_norm<S, WT, 0, 2>(g, threads(2), stream);
    return run_norm<S, WT, 0, 4>(g, threads(4), stream);
}

// ---------------------------------------------------------------------------
// Backward.  Persistent workgroups take rows with a stride of the grid and
// hold the sums of g z for their columns in registers; each writes one row of
// partial sums, which a second kernel adds up in order.
// ---------------------------------------------------------------------------

template <class S, class WT, int V>
__global__ __launch_bounds__(64 * kMaxWaves) void norm_backward_kernel(NormBackwardArgs g) {
    __shared__ float buffer[2][kMaxWaves];
    const int64_t N = g.N;
    Eight dw[V], w[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int64_t c = (int64_t)(v * blockDim.x + threadIdx.x) * 8;
        dw[v] = Eight{};
        w[v] = Eight{};
        if (c < N) w[v] = load8((const WT*)g.weight + c);
    }
    int turn = 0;
    for (int64_t row = blockIdx.x; row < g.M; row += gridDim.x, turn ^= 1) {
        const float r = g.rstd[row];
        Eight z[V], e[V];
        float sum = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int64_t c = (int64_t)(v * blockDim.x + threadIdx.x) * 8;
            z[v] = Eight{};
            e[v] = Eight{};
            if (c < N) {
                z[v] = load8((const S*)g.h + row * g.ldh + c);
                e[v] = load8(g.dy + row * g.ldy + c);
                if (g.dy2 != nullptr) {
                    const Eight more = load8(g.dy2 + row * g.ldy2 + c);
#pragma unroll
                    for (int i = 0; i < 8; ++i) e[v].v[i] += more.v[i];
                }
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                z[v].v[i] *= r;
                dw[v].v[i] = __builtin_fmaf(e[v].v[i], z[v].v[i], dw[v].v[i]);
                e[v].v[i] *= w[v].v[i];
                sum = __builtin_fmaf(e[v].v[i], z[v].v[i], sum);
            }
        }
        const float mean = row_sum<0>(sum, buffer[turn]) / (float)N;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int64_t c = (int64_t)(v * blockDim.x + threadIdx.x) * 8;
            if (c >= N) continue;
            Eight in{};
            if (g.dh_in != nullptr) in = load8((const S*)g.dh_in + row * g.ldi + c);
            Eight out;
#pragma unroll
            for (int i = 0; i < 8; ++i) out.v[i] = in.v[i] + r * (e[v].v[i] - z[v].v[i] * mean);
            if (g.dx != nullptr) store16(g.dx + row * g.lddx + c, pack(out));
            store8((S*)g.dh + row * g.ldo + c, out);
        }
    }
    if (g.dweight == nullptr) return;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int64_t c = (int64_t)(v * blockDim.x + threadIdx.x) * 8;
        if (c < N) store8(g.workspace + (int64_t)blockIdx.x * N + c, dw[v]);
    }
}

__global__ __launch_bounds__(256) void norm_dweight_kernel(const float* __restrict__ part, int32_t parts, int64_t N,
                                                           void* __restrict__ dweight, bool fp32, bool accumulate) {
    const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (c >= N) return;
    float sum = 0.0f;
    for (int32_t p = 0; p < parts; ++p) sum += part[(int64_t)p * N + c];
    if (!fp32)
        ((uint16_t*)dweight)[c] = __builtin_bit_cast(uint16_t, (__bf16)sum);
    else
        ((float*)dweight)[c] = accumulate ? ((float*)dweight)[c] + sum : sum;
}

template <class S, class WT>
hipError_t run_backward(const NormBackwardArgs& g, hipStream_t stream) {
    const int32_t parts = norm_backward_parts(g.M, g.N);
    if (parts > 0) {
        const int64_t vectors = g.N / 8;
        const auto threads = [&](int V) { return (int)((vectors + 64 * V - 1) / (64 * V)) * 64; };
        if (vectors <= 64 * kMaxWaves)
            hipLaunchKernelGGL((norm_backward_kernel<S, WT, 1>), dim3(parts), dim3(threads(1)), 0, stream, g);
        else if (vectors <= 2 * 64 * kMaxWaves)
            hipLaunchKernelGGL((norm_backward_kernel<S, WT, 2>), dim3(parts), dim3(threads(2)), 0, stream, g);
        else
            hipLaunchKernelGGL((norm_backward_kernel<S, WT, 4>), dim3(parts), dim3(threads(4)), 0, stream, g);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if (g.dweight == nullptr) return hipSuccess;
    hipLaunchKernelGGL(norm_dweight_kernel, dim3((unsigned)((g.N + 255) / 256)), dim3(256), 0, stream, g.workspace,
                       parts, g.N, g.dweight, g.dw_fp32, g.accumulate);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_rms_norm(const NormArgs& a, hipStream_t stream) {
    const bool wide = a.flags & MX_NORM_STREAM_FP32, wide_weight = a.flags & MX_NORM_WEIGHT_FP32;
    if (wide) return wide_weight ? pick_norm<float, float>(a, stream) : pick_norm<float, uint16_t>(a, stream);
    return wide_weight ? pick_norm<uint16_t, float>(a, stream) : pick_norm<uint16_t, uint16_t>(a, stream);
}

int32_t norm_backward_parts(int64_t M, int64_t N) {
    (void)N;
    return (int32_t)(M < 512 ? M : 512);
}

hipError_t launch_rms_norm_backward(const NormBackwardArgs& a, hipStream_t stream) {
    const bool wide = a.flags & MX_NORM_STREAM_FP32, wide_weight = a.flags & MX_NORM_WEIGHT_FP32;
    if (wide) return wide_weight ? run_backward<float, float>(a, stream) : run_backward<float, uint16_t>(a, stream);
    return wide_weight ? run_backward<uint16_t, float>(a, stream) : run_backward<uint16_t, uint16_t>(a, stream);
}

}  // namespace mx
