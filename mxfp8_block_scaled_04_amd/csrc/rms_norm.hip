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
#include <type_traits>

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

// Vectors of 8 columns a lane has, and the workgroup's threads, of rows that a workgroup has alone.
constexpr int64_t kTeamVectors = 256;  // up to here a wave has a row
int block_vectors(int64_t vectors) { return vectors <= 64 * kMaxWaves ? 1 : vectors <= 2 * 64 * kMaxWaves ? 2 : 4; }
int block_threads(int64_t vectors) {
    const int V = block_vectors(vectors);
    return (int)((vectors + 64 * V - 1) / (64 * V)) * 64;
}
int team_lanes(int64_t vectors) { return vectors <= 16 ? 16 : vectors <= 32 ? 32 : 64; }

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
    if (vectors <= 192) return run_norm<S, WT, 64, 3>(g, 256, stream);
    if (vectors <= kTeamVectors) return run_norm<S, WT, 64, 4>(g, 256, stream);
    const int threads = block_threads(vectors);
    if (block_vectors(vectors) == 1) return run_norm<S, WT, 0, 1>(g, threads, stream);
    if (block_vectors(vectors) == 2) return run_norm<S, WT, 0, 2>(g, threads, stream);
    return run_norm<S, WT, 0, 4>(g, threads, stream);
}

// ---------------------------------------------------------------------------
// Backward.  Persistent workgroups take rows with a stride of the grid and
// hold the sums of g z for their columns in registers (the row's loads are
// issued before the row in front of it is finished); the teams of a workgroup
// are added up in LDS, each workgroup writes one row of partial sums, and a
// second kernel adds these up in order.
// ---------------------------------------------------------------------------

// A row's values as they are loaded.
template <class S, int V>
struct Row {
    typedef typename std::conditional<sizeof(S) == 2, uint4, Eight>::type Wide;
    uint4 dy[V], dy2[V];
    Wide h[V], in[V];
    float r;
};
__device__ __forceinline__ Eight values(uint4 d) { return unpack(d); }
__device__ __forceinline__ Eight values(const Eight& e) { return e; }
__device__ __forceinline__ void raw8(const uint16_t* p, uint4& d) { d = *reinterpret_cast<const uint4*>(p); }
__device__ __forceinline__ void raw8(const float* p, Eight& d) { d = load8(p); }

template <class S, int V>
__device__ __forceinline__ void load_row(const NormBackwardArgs& g, int64_t row, bool live, int first, int step,
                                         Row<S, V>& x) {
    x.r = live ? g.rstd[row] : 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int64_t c = first + v * step;
        x.dy[v] = x.dy2[v] = make_uint4(0, 0, 0, 0);
        x.h[v] = typename Row<S, V>::Wide{};
        x.in[v] = typename Row<S, V>::Wide{};
        if (!live || c >= g.N) continue;
        raw8((const S*)g.h + row * g.ldh + c, x.h[v]);
        raw8(g.dy + row * g.ldy + c, x.dy[v]);
        if (g.dy2 != nullptr) raw8(g.dy2 + row * g.ldy2 + c, x.dy2[v]);
        if (g.dh_in != nullptr) raw8((const S*)g.dh_in + row * g.ldi + c, x.in[v]);
    }
}

constexpr int kTeamThreads = 256;  // of a workgroup of several teams

template <class S, class WT, int LANES, int V>
__global__ __launch_bounds__(LANES > 0 ? kTeamThreads : 64 * kMaxWaves) void norm_backward_kernel(NormBackwardArgs g) {
    __shared__ float buffer[2][kMaxWaves];
    const int team = LANES > 0 ? LANES : blockDim.x;
    const int a = LANES > 0 ? threadIdx.x & (LANES - 1) : threadIdx.x;
    constexpr int kTeams = LANES > 0 ? kTeamThreads / (LANES > 0 ? LANES : 1) : 1;
    const int64_t mine = LANES > 0 ? threadIdx.x / LANES : 0;
    const int64_t N = g.N;
    const int first = a * 8, step = team * 8;
    Eight dw[V], w[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        dw[v] = Eight{};
        w[v] = Eight{};
        if (first + v * step < N) w[v] = load8((const WT*)g.weight + first + v * step);
    }
    const int64_t stride = (int64_t)gridDim.x * kTeams;
    int64_t row = (int64_t)blockIdx.x * kTeams + mine;
    Row<S, V> next;
    load_row<S, V>(g, row, row < g.M, first, step, next);
    int turn = 0;
    for (int64_t r0 = (int64_t)blockIdx.x * kTeams; r0 < g.M; r0 += stride, row += stride, turn ^= 1) {
        const bool live = row < g.M;
        const float r = next.r;
        Eight z[V], e[V];
        typename Row<S, V>::Wide in[V];
        float sum = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            z[v] = values(next.h[v]);
            e[v] = unpack(next.dy[v]);
            const Eight more = unpack(next.dy2[v]);
            in[v] = next.in[v];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (g.dy2 != nullptr) e[v].v[i] += more.v[i];
                z[v].v[i] *= r;
                dw[v].v[i] = __builtin_fmaf(e[v].v[i], z[v].v[i], dw[v].v[i]);
                e[v].v[i] *= w[v].v[i];
                sum = __builtin_fmaf(e[v].v[i], z[v].v[i], sum);
            }
        }
        if (V <= 2) load_row<S, V>(g, row + stride, row + stride < g.M, first, step, next);
        const float mean = row_sum<LANES>(sum, buffer[turn]) / (float)N;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int64_t c = first + v * step;
            if (!live || c >= N) continue;
            const Eight from = values(in[v]);
            Eight out;
#pragma unroll
            for (int i = 0; i < 8; ++i) out.v[i] = from.v[i] + r * (e[v].v[i] - z[v].v[i] * mean);
            if (g.dx != nullptr) store16(g.dx + row * g.lddx + c, pack(out));
            store8((S*)g.dh + row * g.ldo + c, out);
        }
        if (V > 2) load_row<S, V>(g, row + stride, row + stride < g.M, first, step, next);
    }
    if (g.dweight == nullptr) return;
    float* const part = g.workspace + (int64_t)blockIdx.x * N;
    if constexpr (LANES == 0) {
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (first + v * step < N) store8(part + first + v * step, dw[v]);
    } else {
        __shared__ float sums[kTeams][LANES * 8 * V];
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int i = 0; i < 8; ++i) sums[mine][first + v * step + i] = dw[v].v[i];
        __syncthreads();
        for (int c = threadIdx.x; c < N; c += kTeamThreads) {
            float all = 0.0f;
#pragma unroll
            for (int t = 0; t < kTeams; ++t) all += sums[t][c];
            part[c] = all;
        }
    }
}

// Columns [COLUMNS b, ...) of the parts' sum: 1024 / COLUMNS threads share the
// parts of a column out, then add up in LDS.
template <int COLUMNS>
__global__ __launch_bounds__(1024) void norm_dweight_kernel(const float* __restrict__ part, int32_t parts, int64_t N,
                                                            void* __restrict__ dweight, bool fp32, bool accumulate) {
    constexpr int kShares = 1024 / COLUMNS;
    __shared__ float sums[kShares][COLUMNS + 1];
    const int column = threadIdx.x % COLUMNS, share = threadIdx.x / COLUMNS;
    const int64_t c = (int64_t)blockIdx.x * COLUMNS + column;
    float sum = 0.0f;
    if (c < N) {
#pragma unroll 8
        for (int32_t p = share; p < parts; p += kShares) sum += part[(int64_t)p * N + c];
    }
    sums[share][column] = sum;
    for (int half = kShares / 2; half > 0; half /= 2) {
        __syncthreads();
        if (share < half) sums[share][column] += sums[share + half][column];
    }
    if (share != 0 || c >= N) return;
    sum = sums[0][column];
    if (!fp32)
        ((uint16_t*)dweight)[c] = __builtin_bit_cast(uint16_t, (__bf16)sum);
    else
        ((float*)dweight)[c] = accumulate ? ((float*)dweight)[c] + sum : sum;
}

template <class S, class WT, int LANES, int V>
void run_rows(const NormBackwardArgs& g, int32_t parts, int threads, hipStream_t stream) {
    hipLaunchKernelGGL((norm_backward_kernel<S, WT, LANES, V>), dim3(parts), dim3(threads), 0, stream, g);
}

template <class S, class WT>
hipError_t run_backward(const NormBackwardArgs& g, hipStream_t stream) {
    const int32_t parts = norm_backward_parts(g.M, g.N);
    if (parts > 0) {
        const int64_t n = g.N / 8;
        if (n <= 16) run_rows<S, WT, 16, 1>(g, parts, kTeamThreads, stream);
        else if (n <= 32) run_rows<S, WT, 32, 1>(g, parts, kTeamThreads, stream);
        else if (n <= 64) run_rows<S, WT, 64, 1>(g, parts, kTeamThreads, stream);
        else if (n <= 128) run_rows<S, WT, 64, 2>(g, parts, kTeamThreads, stream);
        else if (n <= 192) run_rows<S, WT, 64, 3>(g, parts, kTeamThreads, stream);
        else if (n <= kTeamVectors) run_rows<S, WT, 64, 4>(g, parts, kTeamThreads, stream);
        else if (block_vectors(n) == 1) run_rows<S, WT, 0, 1>(g, parts, block_threads(n), stream);
        else if (block_vectors(n) == 2) run_rows<S, WT, 0, 2>(g, parts, block_threads(n), stream);
        else run_rows<S, WT, 0, 4>(g, parts, block_threads(n), stream);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if (g.dweight == nullptr) return hipSuccess;
    if (g.N <= 1024)
        hipLaunchKernelGGL((norm_dweight_kernel<8>), dim3((unsigned)((g.N + 7) / 8)), dim3(1024), 0, stream, g.workspace,
                           parts, g.N, g.dweight, g.dw_fp32, g.accumulate);
    else
        hipLaunchKernelGGL((norm_dweight_kernel<32>), dim3((unsigned)((g.N + 31) / 32)), dim3(1024), 0, stream,
                           g.workspace, parts, g.N, g.dweight, g.dw_fp32, g.accumulate);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_rms_norm(const NormArgs& a, hipStream_t stream) {
    const bool wide = a.flags & MX_NORM_STREAM_FP32, wide_weight = a.flags & MX_NORM_WEIGHT_FP32;
    if (wide) return wide_weight ? pick_norm<float, float>(a, stream) : pick_norm<float, uint16_t>(a, stream);
    return wide_weight ? pick_norm<uint16_t, float>(a, stream) : pick_norm<uint16_t, uint16_t>(a, stream);
}

int32_t norm_backward_parts(int64_t M, int64_t N) {
    const int64_t n = N / 8;
    const int64_t rows = n <= kTeamVectors ? kTeamThreads / team_lanes(n) : 1;  // that a workgroup takes at a time
    const int64_t threads = n <= kTeamVectors ? kTeamThreads : block_threads(n);
    const int64_t most = 256 * (2048 / threads), wanted = (M + rows - 1) / rows;  // as many as the 256 CUs hold
    return (int32_t)(wanted < most ? wanted : most);
}

hipError_t launch_rms_norm_backward(const NormBackwardArgs& a, hipStream_t stream) {
    const bool wide = a.flags & MX_NORM_STREAM_FP32, wide_weight = a.flags & MX_NORM_WEIGHT_FP32;
    if (wide) return wide_weight ? run_backward<float, float>(a, stream) : run_backward<float, uint16_t>(a, stream);
    return wide_weight ? run_backward<uint16_t, float>(a, stream) : run_backward<uint16_t, uint16_t>(a, stream);
}

}  // namespace mx
