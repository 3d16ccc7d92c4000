// Root-mean-square norm with the residual's addition before it and an MXFP8
// copy of its output, and its gradients (include/libmxmoe_block.h).
//
// Mathematics per row of N columns: h = x + residual (rounded to the stream's
// type), r = 1 / sqrt(mean(h^2) + eps), y = bf16(h r w), MXFP8 of y as
// quantize_rows_kernel has it.  Backward with g = dy + dy2, a = g w, z = h r:
// dh = dh_in + r (a - z mean(a z)), dw = sum over rows of g z.
//
// What bounds it: HBM.  A row stays in the registers of its team of lanes, 8
// columns a lane and vector, from the loads to the stores, so that everything
// is read and written once; the sum over the row is a reduction in registers
// and, where a workgroup is the team, LDS.  Measured on 32768 rows of 7168,
// bf16: forward with residual and MXFP8 rows (9.03 bytes an element)
// 351 us, 6.05 TB/s; backward with both output gradients and the
// stream's (10 bytes) 414 us, 5.7 TB/s; a copy reaches 5.1
// TB/s, the 2:1 stream of mx_stream21 6.6.
//
// Teams: a wave, half, a quarter or an eighth of one for rows of up to 1024,
// 256, 128 and 64 columns (no barrier); a workgroup for longer ones (2048
// columns: 173 us forward and backward, with a wave 186 and 213).  1.3 10^8
// elements, bf16 without MXFP8: 5.5 to 6.2 TB/s forward and 5.0 to 6.2 backward
// from 64 to 16384 columns; float32 streams 5.2 to 5.9.
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
__device__ __forceinline__ uint4 four(const Eight& e, int i) {
    return __builtin_bit_cast(uint4, make_float4(e.v[i], e.v[i + 1], e.v[i + 2], e.v[i + 3]));
}

// Eight values of a row as they are loaded: bf16 stay packed until they are used.
template <class S>
using Raw = typename std::conditional<sizeof(S) == 2, uint4, Eight>::type;
__device__ __forceinline__ Eight values(uint4 d) { return unpack(d); }
__device__ __forceinline__ const Eight& values(const Eight& e) { return e; }

// Rows are read once: `far`, by non-temporal loads (forward as above 410 ->
// 370 us), in calls that are large enough to pass the caches (below); in others
// they may still be there (forward, 2048 rows of 7168 in turn with two others: 26 us
// with them, 21.5 without).  Not of float32, where an instruction takes every
// other 16 bytes: the second one finds its lines in the cache then (8192
// columns, residual in float32: 303 -> 287 us; the stores as well, 505 -> 303).
__device__ __forceinline__ uint4 load_raw(const uint16_t* p, bool far) {
    return far ? load_stream16(p) : *reinterpret_cast<const uint4*>(p);
}
__device__ __forceinline__ Eight load_raw(const float* p, bool) {
    const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
    return Eight{{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}};
}
// The weight is read for every row.
__device__ __forceinline__ Eight load_kept(const uint16_t* p) { return unpack(*reinterpret_cast<const uint4*>(p)); }
__device__ __forceinline__ Eight load_kept(const float* p) { return load_raw(p, false); }

// Outputs of large calls leave the caches before anything reads them: from
// 2^25 elements on their stores are non-temporal (forward 370 -> 353 us, backward
// 454 -> 415), and so are the loads of bf16; smaller ones are left where the next
// kernel finds them.  Not the stores of a float32 stream (above).  The number is
// where calls with a residual and MXFP8 rows pass the 256 MB of the Infinity
// Cache (9 bytes an element, cached against non-temporal: 16384 and 32768 rows
// of 1024 26.0 and 29.3 us, 58.3 and 56.8).  Calls of fewer bytes an element
// pass it later and are slower in between (4 bytes, without a residual: 65536
// rows 47.9 and 50.4, 131072 101.0 and 93.7; 6 bytes, backward: 32768 rows 44.7
// and 46.3, 65536 82.0 and 79.2).
constexpr int64_t kFar = (int64_t)1 << 25;
__device__ __forceinline__ void store_out(void* p, uint4 d, bool far) {
    if (far) store_stream16(p, d);
    else store16(p, d);
}
// Rounded to the stream's type, in place, and stored.
__device__ __forceinline__ void store_row(uint16_t* p, Eight& e, bool far) {
    const uint4 d = pack(e);
    store_out(p, d, far);
    e = unpack(d);
}
__device__ __forceinline__ void store_row(float* p, Eight& e, bool) {
    store16(p, four(e, 0));
    store16(p + 4, four(e, 4));
}

constexpr int kMaxWaves = 16;
constexpr int kTeamThreads = 256;  // of a workgroup of several teams

// The team's sum in all of its lanes.  LANES: 8, 16, 32, 64 (several teams per
// workgroup), or 0: the workgroup is the team (`buffer`: one float per wave,
// another one in the next call, so that one barrier is enough).  The waves'
// sums are joined in pairs as the lanes' are: one after the other, each of 16
// could lose half a step of what is there already (r of 16384 columns 5.1 10^-8
// off, root mean square; in pairs 4.4).
template <int LANES>
__device__ __forceinline__ float row_sum(float v, float* buffer) {
    if constexpr (LANES > 0) return team_sum<LANES>(v);
    v = team_sum<64>(v);
    const int lane = threadIdx.x & 63, waves = blockDim.x >> 6;
    if (lane == 0) buffer[threadIdx.x >> 6] = v;
    __syncthreads();
    const int W = waves <= 4 ? 4 : waves <= 8 ? 8 : 16, w = lane & (W - 1);
    return team_reduce(w < waves ? buffer[w] : 0.0f, W, [](float p, float q) { return p + q; });
}

// A team for rows of `vectors` times 8 columns.
struct Shape {
    int lanes;    // of a wave, or 0: a workgroup
    int vectors;  // per lane
    int threads;  // of a workgroup
    int teams;    // in it
};
// The forward pass: a lane of a workgroup has 1, 2 or 4 vectors (4096 columns:
// 169, 176, 182 us; 8192: 185, 176, 182).  The backward pass, whose rows take
// more registers: 1 up to 8192 columns.
Shape shape_of(int64_t vectors, int64_t most_of_one) {
    for (int lanes = 8; lanes <= 64; lanes *= 2)
        if (vectors <= lanes) return Shape{lanes, 1, kTeamThreads, kTeamThreads / lanes};
    if (vectors <= 128) return Shape{64, 2, kTeamThreads, kTeamThreads / 64};
    const int each = vectors <= most_of_one ? 1 : vectors <= 2 * 64 * kMaxWaves ? 2 : 4;
    return Shape{0, each, (int)((vectors + 64 * each - 1) / (64 * each)) * 64, 1};
}

// S: the stream's type, WT: the weight's (uint16_t: bf16).
template <class S, class WT, int LANES, int V>
__global__ __launch_bounds__(LANES > 0 ? kTeamThreads : 64 * kMaxWaves) void rms_norm_kernel(NormArgs g, int64_t rows,
                                                                                             bool far) {
    __shared__ float buffer[2][kMaxWaves];
    constexpr int kTeams = LANES > 0 ? kTeamThreads / (LANES > 0 ? LANES : 1) : 1;
    const int team = LANES > 0 ? LANES : blockDim.x;
    const int a = LANES > 0 ? threadIdx.x & (LANES - 1) : threadIdx.x;
    const int64_t mine = LANES > 0 ? threadIdx.x / LANES : 0;
    const int64_t N = g.N;
    // Workgroups go round the 8 XCDs: 32 rows in a row to each, so that the 4-byte pieces of a unit of scales meet in one L2
    // (364 -> 355 us).
    int64_t block = blockIdx.x;
    if (LANES == 0 && (block | 255) < gridDim.x) block = (block & ~(int64_t)255) + (block % 8) * 32 + (block % 256) / 8;
    int turn = 0;
    for (int64_t r0 = block * kTeams; r0 < rows; r0 += (int64_t)gridDim.x * kTeams, turn ^= 1) {
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
                    h[v] = unpack(load_raw((const uint16_t*)g.x + row * g.ldx + c, far));
                    const Eight r = values(load_raw((const S*)g.residual + row * g.ldr + c, far));
#pragma unroll
                    for (int i = 0; i < 8; ++i) h[v].v[i] += r.v[i];
                    store_row((S*)g.h + row * g.ldh + c, h[v], far);
                } else {
                    h[v] = values(load_raw((const S*)g.x + row * g.ldx + c, far));
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
                const Eight w = load_kept((const WT*)g.weight + c);
                Eight e;
#pragma unroll
                for (int i = 0; i < 8; ++i) e.v[i] = h[v].v[i] * r * w.v[i];
                out = pack(e);
                if (g.y != nullptr) store_out(g.y + row * g.ldy + c, out, far);
            }
            if (g.q == nullptr) continue;
            const uint32_t scale = scale_from_maxmag(quad_max_u32(max_mag8(out)));
            if (live && c < N) {
                const uint2 codes = quant8(out, scale);
                if (far) store_stream8(g.q + row * N + c, codes);
                else store8(g.q + row * N + c, codes);
            }
            // the unit's scale bytes of this row: two dwords, of the even and
            // the odd blocks, byte b / 2; 4 lanes have a block, 32 a unit
            constexpr int kUnit = LANES == 8 || LANES == 16 ? LANES : 32;
            const int in_unit = threadIdx.x & (kUnit - 1), b = in_unit >> 2;
            uint32_t word = scale << (8 * (b >> 1));
            if constexpr (kUnit >= 16)
                word |= (uint32_t)__builtin_amdgcn_mov_dpp((int)word, 0x128, 0xF, 0xF, false);  // row_ror:8 (block b ^ 2)
            if constexpr (kUnit == 32) {
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
hipError_t run_norm(const NormArgs& g, const Shape& at, hipStream_t stream) {
    const int64_t rows = g.q != nullptr ? (g.M + 31) / 32 * 32 : g.M;  // with the padding rows of the scales
    int64_t blocks = (rows + at.teams - 1) / at.teams;
    if (blocks > (1 << 20)) blocks = 1 << 20;
    hipLaunchKernelGGL((rms_norm_kernel<S, WT, LANES, V>), dim3((unsigned)blocks), dim3(at.threads), 0, stream, g, rows,
                       g.M * g.N >= kFar);
    return hipGetLastError();
}

template <class S, class WT>
hipError_t pick_norm(const NormArgs& g, hipStream_t stream) {
    const Shape at = shape_of(g.N / 8, 512);
    switch (at.lanes + at.vectors) {
        case 8 + 1: return run_norm<S, WT, 8, 1>(g, at, stream);
        case 16 + 1: return run_norm<S, WT, 16, 1>(g, at, stream);
        case 32 + 1: return run_norm<S, WT, 32, 1>(g, at, stream);
        case 64 + 1: return run_norm<S, WT, 64, 1>(g, at, stream);
        case 64 + 2: return run_norm<S, WT, 64, 2>(g, at, stream);
        case 0 + 1: return run_norm<S, WT, 0, 1>(g, at, stream);
        case 0 + 2: return run_norm<S, WT, 0, 2>(g, at, stream);
        default: return run_norm<S, WT, 0, 4>(g, at, stream);
    }
}

// ---------------------------------------------------------------------------
// Backward.  Persistent workgroups take rows with a stride of the grid and
// hold the sums of g z for their columns in registers; the teams of a
// workgroup are added up in LDS, each workgroup writes one row of partial
// sums, and a second kernel adds these up in order (5 us at 7168 columns).
// Two workgroups per CU: more take as long or longer, and write more parts
// (2048 columns: 173, 181 and 194 us with 2, 3 and 4).
//
// AHEAD: the next row's loads are issued before this row is finished, and the
// weight is kept.  Without it neither, and dh_in is read after the sum, so that
// 2 workgroups of up to 16 waves fit a CU: above 4096 columns (7168: 415 us
// against 430; 4096: 193 against 182).
// ---------------------------------------------------------------------------

// A row's values as they are loaded; nothing where there is no row.
template <class S, int V, bool AHEAD>
struct Row {
    uint4 dy[V], dy2[V];
    Raw<S> h[V], in[AHEAD ? V : 1];
    float r;
    __device__ __forceinline__ void load(const NormBackwardArgs& g, int64_t row, int first, int step, bool far) {
        const bool live = row < g.M;
        r = live ? g.rstd[row] : 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int64_t c = first + v * step;
            dy[v] = dy2[v] = make_uint4(0, 0, 0, 0);
            h[v] = Raw<S>{};
            if constexpr (AHEAD) in[v] = Raw<S>{};
            if (!live || c >= g.N) continue;
            h[v] = load_raw((const S*)g.h + row * g.ldh + c, far);
            dy[v] = load_raw(g.dy + row * g.ldy + c, far);
            if (g.dy2 != nullptr) dy2[v] = load_raw(g.dy2 + row * g.ldy2 + c, far);
            if constexpr (AHEAD)
                if (g.dh_in != nullptr) in[v] = load_raw((const S*)g.dh_in + row * g.ldi + c, far);
        }
    }
    // z, and g in e
    __device__ __forceinline__ void take(const NormBackwardArgs& a, int v, Eight& z, Eight& e) const {
        z = values(h[v]);
        e = unpack(dy[v]);
        const Eight more = unpack(dy2[v]);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (a.dy2 != nullptr) e.v[i] += more.v[i];
            z.v[i] *= r;
        }
    }
};

__device__ __forceinline__ void write_dweight(const NormBackwardArgs& g, int64_t c, float sum) {
    if (!g.dw_fp32)
        ((uint16_t*)g.dweight)[c] = __builtin_bit_cast(uint16_t, (__bf16)sum);
    else
        ((float*)g.dweight)[c] = g.accumulate ? ((float*)g.dweight)[c] + sum : sum;
}

// dweight of 32 columns over all rows, by one workgroup: 4 lanes have a row's 8
// columns each, and a wave 16 rows at a time.
constexpr int kSlice = 32;
template <class S>
__device__ __forceinline__ void dweight_slice(const NormBackwardArgs& g, int64_t slice) {
    __shared__ float sums[kMaxWaves][kSlice];
    const int lane = threadIdx.x & 63, waves = blockDim.x >> 6;
    const int c = (int)slice * kSlice + (lane & 3) * 8;
    Eight acc{};
#pragma unroll 4
    for (int64_t row = threadIdx.x >> 2; row < g.M; row += blockDim.x >> 2) {
        Row<S, 1, false> x;
        x.load(g, row, c, 0, false);
        Eight z, e;
        x.take(g, 0, z, e);
#pragma unroll
        for (int i = 0; i < 8; ++i) acc.v[i] = __builtin_fmaf(e.v[i], z.v[i], acc.v[i]);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
#pragma unroll
        for (int d = 4; d < 64; d *= 2) acc.v[i] += __shfl_xor(acc.v[i], d);
        if (lane < 4) sums[threadIdx.x >> 6][lane * 8 + i] = acc.v[i];
    }
    __syncthreads();
    if (threadIdx.x >= kSlice || slice * kSlice + threadIdx.x >= g.N) return;
    float sum = 0.0f;
    for (int w = 0; w < waves; ++w) sum += sums[w][threadIdx.x];
    write_dweight(g, slice * kSlice + threadIdx.x, sum);
}

// FEW: the first `slices` workgroups of the grid have dweight, 32 columns each,
// and the others the rows (an instance of its own: 6 registers more would keep
// the second workgroup of 14 waves off a CU, 415 -> 457 us).
template <class S, class WT, int LANES, int V, bool AHEAD, bool FEW>
__global__ __launch_bounds__(LANES > 0 ? kTeamThreads : 64 * kMaxWaves) void norm_backward_kernel(NormBackwardArgs g,
                                                                                                  int32_t slices,
                                                                                                  bool far) {
    if constexpr (FEW) {
        if ((int32_t)blockIdx.x < slices) {
            dweight_slice<S>(g, blockIdx.x);
            return;
        }
    } else {
        slices = 0;
    }
    const int64_t block = blockIdx.x - slices, blocks = gridDim.x - slices;
    __shared__ float buffer[2][kMaxWaves];
    constexpr int kTeams = LANES > 0 ? kTeamThreads / (LANES > 0 ? LANES : 1) : 1;
    const int team = LANES > 0 ? LANES : blockDim.x;
    const int a = LANES > 0 ? threadIdx.x & (LANES - 1) : threadIdx.x;
    const int64_t mine = LANES > 0 ? threadIdx.x / LANES : 0;
    const int64_t N = g.N;
    const int first = a * 8, step = team * 8;
    const auto weight = [&](int v) {
        const int c = first + v * step;
        return c < N ? load_kept((const WT*)g.weight + c) : Eight{};
    };
    Eight dw[V], kept[AHEAD ? V : 1];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        dw[v] = Eight{};
        if constexpr (AHEAD) kept[v] = weight(v);
    }
    const int64_t stride = blocks * kTeams;
    int64_t row = block * kTeams + mine;
    Row<S, V, AHEAD> x;
    if constexpr (AHEAD) x.load(g, row, first, step, far);
    int turn = 0;
    for (int64_t r0 = block * kTeams; r0 < g.M; r0 += stride, row += stride, turn ^= 1) {
        Eight z[V], e[V];
        Raw<S> in[V];
        float sum = 0.0f;
        if constexpr (!AHEAD) x.load(g, row, first, step, far);
        const float r = x.r;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            x.take(g, v, z[v], e[v]);
            if constexpr (AHEAD) in[v] = x.in[v];
            Eight w;
            if constexpr (AHEAD) w = kept[v];
            else w = weight(v);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                dw[v].v[i] = __builtin_fmaf(e[v].v[i], z[v].v[i], dw[v].v[i]);
                e[v].v[i] *= w.v[i];
                sum = __builtin_fmaf(e[v].v[i], z[v].v[i], sum);
            }
        }
        if constexpr (AHEAD) x.load(g, row + stride, first, step, far);
        const float mean = row_sum<LANES>(sum, buffer[turn]) / (float)N;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int64_t c = first + v * step;
            if (row >= g.M || c >= N) continue;
            if constexpr (!AHEAD) {
                in[v] = Raw<S>{};
                if (g.dh_in != nullptr) in[v] = load_raw((const S*)g.dh_in + row * g.ldi + c, far);
            }
            const Eight from = values(in[v]);
            Eight out;
#pragma unroll
            for (int i = 0; i < 8; ++i) out.v[i] = from.v[i] + r * (e[v].v[i] - z[v].v[i] * mean);
            if (g.dx != nullptr) store_out(g.dx + row * g.lddx + c, pack(out), far);
            store_row((S*)g.dh + row * g.ldo + c, out, far);
        }
    }
    if (FEW || g.dweight == nullptr) return;
    float* const part = g.workspace + block * N;
    if constexpr (LANES == 0) {
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (first + v * step < N) store_row(part + first + v * step, dw[v], false);
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

// Rows above 16384 columns: their values do not fit the registers (kept, they
// spill: 500 us at 32768 columns, 314 here).  The sums of g z are in LDS, and
// a row is read again after its sum.
template <class S, class WT>
__global__ __launch_bounds__(64 * kMaxWaves) void norm_backward_long_kernel(NormBackwardArgs g, bool far) {
    __shared__ __attribute__((aligned(16))) float dw[MX_NORM_MAX_N];  // (a thread uses its own columns only)
    __shared__ float buffer[2][kMaxWaves];
    const int N = (int)g.N, first = threadIdx.x * 8, step = blockDim.x * 8;
    const auto columns = [&](int c) { return reinterpret_cast<float4*>(dw + c); };
    for (int c = first; c < N; c += step) columns(c)[0] = columns(c)[1] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    int turn = 0;
    for (int64_t row = blockIdx.x; row < g.M; row += gridDim.x, turn ^= 1) {
        float sum = 0.0f;
#pragma unroll 2
        for (int c = first; c < N; c += step) {
            Row<S, 1, false> x;
            x.load(g, row, c, 0, far);
            Eight z, e;
            x.take(g, 0, z, e);
            const Eight w = load_kept((const WT*)g.weight + c);
            Eight d = load_kept(dw + c);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                d.v[i] = __builtin_fmaf(e.v[i], z.v[i], d.v[i]);
                sum = __builtin_fmaf(e.v[i] * w.v[i], z.v[i], sum);
            }
            columns(c)[0] = make_float4(d.v[0], d.v[1], d.v[2], d.v[3]);
            columns(c)[1] = make_float4(d.v[4], d.v[5], d.v[6], d.v[7]);
        }
        const float mean = row_sum<0>(sum, buffer[turn]) / (float)N;
#pragma unroll 2
        for (int c = first; c < N; c += step) {
            Row<S, 1, true> x;
            x.load(g, row, c, 0, far);
            Eight z, e;
            x.take(g, 0, z, e);
            const Eight w = load_kept((const WT*)g.weight + c), from = values(x.in[0]);
            Eight out;
#pragma unroll
            for (int i = 0; i < 8; ++i) out.v[i] = from.v[i] + x.r * (e.v[i] * w.v[i] - z.v[i] * mean);
            if (g.dx != nullptr) store_out(g.dx + row * g.lddx + c, pack(out), far);
            store_row((S*)g.dh + row * g.ldo + c, out, far);
        }
    }
    if (g.dweight == nullptr) return;
    for (int c = first; c < N; c += step) {
        Eight d = load_kept(dw + c);
        store_row(g.workspace + (int64_t)blockIdx.x * N + c, d, false);
    }
}

// Columns [COLUMNS b, ...) of the parts' sum: 1024 / COLUMNS threads share the
// parts of a column out, then add up in LDS.  8 columns where there are few (a
// workgroup for each), else 32 (whole lines of the parts).
template <int COLUMNS>
__global__ __launch_bounds__(1024) void norm_dweight_kernel(NormBackwardArgs g, int32_t parts) {
    const float* const part = g.workspace;
    const int64_t N = g.N;
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
    write_dweight(g, c, sums[0][column]);
}

template <class S>
__global__ __launch_bounds__(64 * kMaxWaves) void norm_slices_kernel(NormBackwardArgs g) {
    dweight_slice<S>(g, blockIdx.x);
}

constexpr int64_t kBackwardOne = 64 * kMaxWaves;  // rows of up to so many vectors: one per lane

// Up to so many rows (of up to 16384 columns) dweight is computed from the rows
// again, which are in the caches, instead of from parts: one launch for all of
// it, no workspace, and 3 us less on the host.  Rows read again against parts:
// 256 rows of 64 columns 5.1 and 5.7 us, of 1480 5.8 and 7.3, of 7168 7.5 and
// 11.7, of 16384 15.2 and 17.9; 384 rows of 64 5.7 and 5.8, of 16384 20.2 and
// 19.1; 1024 rows of 1480 14.5 and 10.5.  Where an output replaces an input, it
// is computed before.
constexpr int64_t kFewRows = 256;
bool few_rows(int64_t M, int64_t N) { return M > 0 && M <= kFewRows && N <= 16 * 64 * kMaxWaves; }

template <class S, class WT, int LANES, int V, bool AHEAD>
void run_rows(const NormBackwardArgs& g, const Shape& at, int32_t blocks, int32_t slices, hipStream_t stream) {
    const bool far = g.M * g.N >= kFar;
    if (slices > 0)
        hipLaunchKernelGGL((norm_backward_kernel<S, WT, LANES, V, AHEAD, true>), dim3(slices + blocks), dim3(at.threads), 0,
                           stream, g, slices, far);
    else
        hipLaunchKernelGGL((norm_backward_kernel<S, WT, LANES, V, AHEAD, false>), dim3(blocks), dim3(at.threads), 0, stream,
                           g, 0, far);
}

template <class S, class WT>
hipError_t run_backward(const NormBackwardArgs& g, hipStream_t stream) {
    const bool few = g.dweight != nullptr && few_rows(g.M, g.N);
    const int32_t columns = (int32_t)((g.N + kSlice - 1) / kSlice);
    int32_t slices = few ? columns : 0;
    const auto replaces = [&](const void* out) {  // what dweight is computed from
        return out != nullptr && (out == (const void*)g.dy || out == (const void*)g.dy2 || out == g.h);
    };
    if (few && (replaces(g.dh) || replaces(g.dx))) {
        hipLaunchKernelGGL((norm_slices_kernel<S>), dim3(columns), dim3(64 * kMaxWaves), 0, stream, g);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        slices = 0;
    }
    NormBackwardArgs rows = g;
    if (few && slices == 0) rows.dweight = nullptr;  // (it is there)
    const Shape at = shape_of(g.N / 8, kBackwardOne);
    const int32_t parts = norm_backward_parts(g.M, g.N);
    if (parts > 0) {
        switch (at.lanes + at.vectors) {
            case 8 + 1: run_rows<S, WT, 8, 1, true>(rows, at, parts, slices, stream); break;
            case 16 + 1: run_rows<S, WT, 16, 1, true>(rows, at, parts, slices, stream); break;
            case 32 + 1: run_rows<S, WT, 32, 1, true>(rows, at, parts, slices, stream); break;
            case 64 + 1: run_rows<S, WT, 64, 1, true>(rows, at, parts, slices, stream); break;
            case 64 + 2: run_rows<S, WT, 64, 2, true>(rows, at, parts, slices, stream); break;
            case 0 + 1:
                if (at.threads <= 512) run_rows<S, WT, 0, 1, true>(rows, at, parts, slices, stream);
                else run_rows<S, WT, 0, 1, false>(rows, at, parts, slices, stream);
                break;
            case 0 + 2: run_rows<S, WT, 0, 2, false>(rows, at, parts, slices, stream); break;
            default:
                hipLaunchKernelGGL((norm_backward_long_kernel<S, WT>), dim3(parts), dim3(at.threads), 0, stream, rows,
                                   g.M * g.N >= kFar);
        }
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if (g.dweight == nullptr || few) return hipSuccess;
    if (g.N <= 1024)
        hipLaunchKernelGGL((norm_dweight_kernel<8>), dim3((unsigned)((g.N + 7) / 8)), dim3(1024), 0, stream, g, parts);
    else
        hipLaunchKernelGGL((norm_dweight_kernel<32>), dim3((unsigned)((g.N + 31) / 32)), dim3(1024), 0, stream, g,
                           parts);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_rms_norm(const NormArgs& a, hipStream_t stream) {
    const bool wide = a.flags & MX_NORM_STREAM_FP32, wide_weight = a.flags & MX_NORM_WEIGHT_FP32;
    if (wide) return wide_weight ? pick_norm<float, float>(a, stream) : pick_norm<float, uint16_t>(a, stream);
    return wide_weight ? pick_norm<uint16_t, float>(a, stream) : pick_norm<uint16_t, uint16_t>(a, stream);
}

bool norm_backward_needs_parts(int64_t M, int64_t N) { return M > 0 && !few_rows(M, N); }

int32_t norm_backward_parts(int64_t M, int64_t N) {
    const Shape at = shape_of(N / 8, kBackwardOne);
    const int64_t wanted = (M + at.teams - 1) / at.teams;  // one step of rows each
    // On each of 256 CUs one workgroup of many registers or much LDS, two of others (1531 rows of 1480, float32 stream: 256
    // parts 12.4 us, 384 12.8, 512 11.8, 1024 14.2), and four of 3 waves where there are rows for them (8192: 25.1 -> 24.4).
    int64_t most = 512;
    if (at.lanes == 0 && at.vectors > 1) most = 256;
    else if (at.lanes == 0 && at.threads <= 192 && wanted >= 8192) most = 1024;
    if (wanted < most) most = 256;
    return (int32_t)(wanted < most ? wanted : most);
}

hipError_t launch_rms_norm_backward(const NormBackwardArgs& a, hipStream_t stream) {
    const bool wide = a.flags & MX_NORM_STREAM_FP32, wide_weight = a.flags & MX_NORM_WEIGHT_FP32;
    if (wide) return wide_weight ? run_backward<float, float>(a, stream) : run_backward<float, uint16_t>(a, stream);
    return wide_weight ? run_backward<uint16_t, float>(a, stream) : run_backward<uint16_t, uint16_t>(a, stream);
}

}  // namespace mx
