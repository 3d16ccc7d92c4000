// Products grouped by expert on bf16 operands, fp32 accumulation:
//   forward  out[r] = x[r] w[g]^T     dgrad  dx[r] = dy[r] w[g]
//   wgrad    dw[g] (+)= sum over the rows r of g of dy[r]^T x[r]
//
// One kernel computes all three as C[i][j] = sum_k A(i, k) B(j, k); they
// differ in which index of an operand is contiguous in memory.  An operand
// whose contraction index is contiguous (forward: both; dgrad: dy) is staged
// as rows of 64 contraction elements and read as 16-byte fragments; one
// whose contraction index is the row (dgrad: w; wgrad: both) is staged as it
// lies, 64 rows of the tile's width, and read with the transposing LDS read
// (ds_read_b64_tr_b16), so that no transposed copy of anything is made.
//
// What bounds it: the matrix pipes, where groups have many rows; reading the
// weights, where they have few.
//
// Layout: persistent workgroups (one 256 x 256 tile per CU with 8 waves of
// 128 x 64, or two 128 x 128 tiles per CU with 4 waves of 64 x 64 each),
// v_mfma_f32_32x32x16_bf16.  A stage is 64 contraction elements of both
// operands (64 KB for the large tile), loaded straight into LDS by 16-byte
// direct loads, two stages in LDS.  Within a stage there are 4 steps of 16;
// the fragments of a step are read while the one before is multiplied, also
// across stages and tiles: the wait for the next stage and the barrier sit
// before a stage's last step, whose fragments are in registers by then, and
// the loads of the stage after the next go into the buffer freed by that
// barrier.
//
// Bounds: all loads go through buffer descriptors that end at the operand's
// last valid element; what lies past it reads as zero.  Rows of a tile past
// its group, contraction indices past K (N for dgrad, the group's rows for
// wgrad) and stages past the last tile need no other care, except granules
// past K inside a row, whose offsets are moved out of range.
#include "mx_train.h"

namespace mx {
namespace {

constexpr int SK = 64;          // contraction elements per stage
constexpr int kLptGroups = 512;  // wgrad: groups taken longest first up to this many
constexpr int kBand = 4;         // row tiles per band of the tile order
// An offset past every descriptor (fewer than 2^31 bytes: 256 rows of fewer
// than 2^22 elements), which no scalar offset of a load (below 2^31 too)
// carries past 2^32.
constexpr uint32_t kOut = 0x80000000u;

typedef __attribute__((address_space(3))) void lds_t;
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

enum Mode { kForward = 0, kDgrad = 1, kWgrad = 2 };
enum Store { kBf16 = 0, kFp32 = 1, kFp32Add = 2 };

struct Args {
    const uint16_t* a;  // forward x, dgrad dy, wgrad dy
    const uint16_t* b;  // forward w, dgrad w, wgrad x
    const int32_t* offsets;
    void* out;
    int64_t lda, ldb, ldo;  // row strides, elements
    int64_t M;              // rows of the activations
    int64_t I, J;           // the output: [M][J] (I unused), wgrad [G][I][J]
    int64_t K;              // contraction length (wgrad: the group's rows)
    int32_t G;
};

__device__ __forceinline__ uint32_t uni(uint32_t v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ uint32_t lds_addr(const void* p) { return (uint32_t)(uintptr_t)(lds_t*)p; }

// Buffer descriptor over [p, p + bytes): loads past it give zeros.
__device__ __forceinline__ i32x4 descriptor(const void* base, uint32_t bytes) {
    const uint64_t p = (uint64_t)(uintptr_t)base;
    i32x4 r;
    r[0] = (int)uni((uint32_t)p);
    r[1] = (int)uni((uint32_t)(p >> 32) & 0xFFFFu);
    r[2] = (int)uni(bytes);
    r[3] = (int)uni(0x00020000u);
    return r;
}

// 16 bytes per lane from the descriptor straight into LDS, lane l to
// [lds + 16 l, lds + 16 l + 16).  In assembly without an output register:
// the compiler would otherwise wait for it before every LDS read.  It is
// waited for by wait_loads and a barrier before the data is read.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void load_to_lds(const i32x4& rs, uint32_t voff, uint32_t soff, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %3\n\ts_nop 0\n\tbuffer_load_dwordx4 %0, %1, %2 offen lds" ::"v"(voff), "s"(rs),
                 "s"(soff), "s"(lds)
                 : "memory", "m0");
}
#pragma clang diagnostic pop
template <int N>
__device__ __forceinline__ void wait_loads() {
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// Range-checked stores and loads of the result.
typedef __amdgpu_buffer_rsrc_t rsrc_t;
__device__ __forceinline__ rsrc_t out_rsrc(void* base, uint32_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(base, (short)0, (int)bytes, 0x00020000);
}

// ---- an operand in LDS -----------------------------------------------------
//
// ROWS elements of the tile x SK contraction elements, 128 ROWS bytes.
//
// T = false: row r at 128 r, its 16-byte granule c (contraction 8 c ...) at
// position c ^ ((r >> 1) & 7): a fragment read (64 lanes, rows 0..31, two
// neighbouring granules) then meets each bank as often as every other.
//
// T = true: contraction row k at 2 ROWS k; its 32-byte unit u (tile rows 16 u
// ...) at position u ^ f(k), f(k) = 2 (k & 3) | (k >> 3 & 1).  A transposing
// read of 64 lanes takes 64 bytes from each of the 8 contraction rows
// k0 + {0..3, 8..11}; f puts them into different banks.
template <int ROWS, int WAVES, bool T>
struct Operand {
    static constexpr int kBytes = ROWS * SK * 2;
    static constexpr int kLoads = kBytes / 1024 / WAVES;  // load instructions per wave and stage
    // contraction rows (T) or tile rows of one load instruction
    static constexpr int kRowsPerLoad = T ? 64 / (ROWS / 8) : 8;

    __device__ __forceinline__ static uint32_t swizzled(uint32_t row, uint32_t pos) {
        if (T) {
            const uint32_t f = ((row & 3u) << 1) | ((row >> 3) & 1u);
            return (((pos >> 1) ^ f) << 1) | (pos & 1u);
        }
        return pos ^ ((row >> 1) & 7u);
    }
};

// Loads of one stage of an operand by one wave.
template <int ROWS, int WAVES, bool T>
__device__ __forceinline__ void issue_loads(const i32x4& rs, uint32_t ld2, uint32_t lds, int wave, int lane,
                                            int left) {
    using O = Operand<ROWS, WAVES, T>;
    constexpr int per_row = T ? ROWS / 8 : 8;  // granules per staged row
#pragma unroll
    for (int j = 0; j < O::kLoads; ++j) {
        const uint32_t q = (uint32_t)(wave * O::kLoads + j);
        const uint32_t row = q * O::kRowsPerLoad + (uint32_t)(lane / per_row);
        const uint32_t g = O::swizzled(row, (uint32_t)(lane % per_row));
        uint32_t voff = (uint32_t)(lane / per_row) * ld2 + g * 16u;
        if (!T && (int)(g * 8u) >= left) voff = kOut;  // past the contraction's end
        load_to_lds(rs, voff, uni(q * O::kRowsPerLoad * ld2), uni(lds + q * 1024u));
    }
}

// Fragment of tile rows [32 blk, 32 blk + 32), contraction step s: lane l
// holds row l % 32, contraction elements 8 (l / 32) .. + 7 of the step.
template <int ROWS, bool T>
struct Reader {
    uint32_t base[4];  // T: per block modulo 4; else [0] only

    // blk0: the wave's first block
    __device__ __forceinline__ void init(int blk0, int nblk, int lane) {
        const uint32_t h = (uint32_t)lane >> 5;
        if (T) {
            const uint32_t k = ((uint32_t)lane & 15u) >> 2;  // + 8 h + 4 i + 16 s
            const uint32_t f = (k << 1) | h;
            const uint32_t c = (((uint32_t)lane >> 4) & 1u) ^ f;
#pragma unroll
            for (int b = 0; b < 4; ++b)
                if (b < nblk)
                    base[b] = (k + 8u * h) * (2u * ROWS) + (((2u * (uint32_t)(blk0 + b)) ^ c) * 32u) +
                              8u * ((uint32_t)lane & 3u);
        } else {
            const uint32_t r = (uint32_t)blk0 * 32u + ((uint32_t)lane & 31u);
            base[0] = r * 128u + ((h ^ ((r >> 1) & 7u)) * 16u);
        }
    }
    __device__ __forceinline__ bf16x8 read(const uint8_t* lds, int b, int s) const {
        if (T) {
            const uint8_t* const p = lds + base[b] + s * 16 * (2 * ROWS);
            const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(lds_t*)p);
            const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(lds_t*)(p + 4 * (2 * ROWS)));
            typedef short s16x8 __attribute__((ext_vector_type(8)));
            return __builtin_bit_cast(bf16x8, (s16x8)__builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
        }
        return *reinterpret_cast<const bf16x8*>(lds + ((base[0] ^ (uint32_t)(32 * s)) + b * 32 * 128));
    }
};

// ---- tiles -----------------------------------------------------------------

// One output tile (wave-uniform).
struct Tile {
    const uint16_t* a;    // first row / column of the operand at contraction 0
    const uint16_t* b;
    int64_t out;          // element offset of the tile's first output element
    int64_t k;            // contraction length
    int32_t rows, cols;   // valid part (0 rows: no tile)
    int32_t stages;       // at least 1
};

// Walks the tiles slot, slot + nwg, ... of a workgroup (wgrad, longest groups
// first: alternating directions, which evens out the sums).
struct Walk {
    int64_t tile;
    int g;     // position in tile order
    bool odd;
};

template <int MODE, int TM, int TN>
struct Sched {
    int64_t total;
    int nwg, slot;
    bool lpt;
    const int32_t* tile_end;  // LDS: inclusive prefix of tiles per position
    const int32_t* order;     // LDS: group at a position (lpt)

    __device__ __forceinline__ static int64_t bound(const Args& p, int g) {
        const int64_t v = p.offsets[g];
        return v < 0 ? 0 : (v > p.M ? p.M : v);
    }
    __device__ __forceinline__ static int64_t rows_of(const Args& p, int g) {
        const int64_t n = bound(p, g + 1) - bound(p, g);
        return n > 0 ? n : 0;
    }

    __device__ __forceinline__ Tile decode(const Args& p, Walk& w) const {
        Tile T;
        if (w.tile >= total) {
            T.a = p.a;
            T.b = p.b;
            T.out = 0;
            T.k = 0;
            T.rows = T.cols = 0;
            T.stages = 1;
            return T;
        }
        while (tile_end[w.g] <= w.tile) ++w.g;
        w.g = (int)uni((uint32_t)w.g);
        const int first = w.g > 0 ? (int)uni((uint32_t)tile_end[w.g - 1]) : 0;
        const uint32_t local = uni((uint32_t)(w.tile - first));
        const int grp = lpt ? (int)uni((uint32_t)order[w.g]) : w.g;
        const int64_t o0 = bound(p, grp), mg = rows_of(p, grp);
        const int64_t ilen = MODE == kWgrad ? p.I : mg;
        const uint32_t nI = (uint32_t)((ilen + TM - 1) / TM), nJ = (uint32_t)((p.J + TN - 1) / TN);
        const uint32_t band = local / (kBand * nJ), r = local - band * (kBand * nJ);
        const uint32_t high = nI - band * kBand < (uint32_t)kBand ? nI - band * kBand : (uint32_t)kBand;
        const uint32_t nt = r / high, mt = band * kBand + (r - nt * high);
        const int64_t i0 = (int64_t)mt * TM, j0 = (int64_t)nt * TN;
        const int64_t il = ilen - i0, jl = p.J - j0;
        T.rows = (int32_t)(il < TM ? il : TM);
        T.cols = (int32_t)(jl < TN ? jl : TN);
        if (MODE == kWgrad) {
            T.a = p.a + o0 * p.lda + i0;
            T.b = p.b + o0 * p.ldb + j0;
            T.out = ((int64_t)grp * p.I + i0) * p.J + j0;
            T.k = mg;
        } else {
            T.a = p.a + (o0 + i0) * p.lda;
            T.b = MODE == kForward ? p.b + ((int64_t)grp * p.J + j0) * p.K : p.b + (int64_t)grp * p.K * p.J + j0;
            T.out = (o0 + i0) * p.ldo + j0;
            T.k = p.K;
        }
        T.stages = (int32_t)((T.k + SK - 1) / SK);
        if (T.stages < 1) T.stages = 1;
        return T;
    }
    __device__ __forceinline__ void next(Walk& w) const {
        w.tile += !lpt ? nwg : (w.odd ? 2 * (int64_t)slot + 1 : 2 * (int64_t)(nwg - slot) - 1);
        w.odd = !w.odd;
    }
};

__device__ __forceinline__ uint32_t pack2(float x, float y) {
    return (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)x) | ((uint32_t)__builtin_bit_cast(uint16_t, (__bf16)y) << 16);
}

template <int MODE, int TM, int TN, int WM, int WN, int OUT>
__global__ __launch_bounds__((TM / WM) * (TN / WN) * 64, 2) void grouped_bf16_kernel(Args p) {
    constexpr int kWaves = (TM / WM) * (TN / WN);
    constexpr int MI = WM / 32, NJ = WN / 32;
    constexpr bool TA = MODE == kWgrad, TB = MODE != kForward;
    constexpr int kThreads = kWaves * 64;
    __shared__ __attribute__((aligned(16))) uint8_t lds_a[2][TM * SK * 2];
    __shared__ __attribute__((aligned(16))) uint8_t lds_b[2][TN * SK * 2];
    __shared__ int32_t part[kThreads];
    extern __shared__ int32_t table[];  // tile_end [G], then order [G] (wgrad, few groups)

    const int t = threadIdx.x, wave = (int)uni((uint32_t)t >> 6), lane = t & 63;
    const int wm = wave / (TN / WN), wn = wave % (TN / WN);
    const int nwg = gridDim.x, bid = blockIdx.x;
    const int G = p.G;

    Sched<MODE, TM, TN> S;
    S.nwg = nwg;
    // each XCD (workgroups are dealt to the 8 of them in turn) takes a
    // contiguous range of the tiles and shares operands through its L2
    S.slot = nwg % 8 == 0 ? (bid % 8) * (nwg / 8) + bid / 8 : bid;
    S.lpt = MODE == kWgrad && G <= kLptGroups;
    S.tile_end = table;
    S.order = table + G;
    {
        int32_t* const order = table + G;
        if (S.lpt) {  // rank by length, longest first, ties by index
            for (int g = t; g < G; g += kThreads) table[g] = (int32_t)S.rows_of(p, g);
            __syncthreads();
            for (int g = t; g < G; g += kThreads) {
                const int32_t n = table[g];
                int rank = 0;
                for (int h = 0; h < G; ++h) rank += table[h] > n || (table[h] == n && h < g) ? 1 : 0;
                order[rank] = g;
            }
            __syncthreads();
        }
        // tiles per position and their inclusive prefix
        const int64_t nJ = (p.J + TN - 1) / TN;
        const int per = (G + kThreads - 1) / kThreads;
        int32_t sum = 0;
        for (int e = 0; e < per; ++e) {
            const int g = t * per + e;
            if (g >= G) break;
            const int64_t mg = S.rows_of(p, S.lpt ? order[g] : g);
            // a weight gradient without rows is zero: one empty stage, unless it is added to
            const int64_t tiles = MODE == kWgrad ? (OUT == kFp32Add && mg == 0 ? 0 : (p.I + TM - 1) / TM * nJ)
                                                 : (mg + TM - 1) / TM * nJ;
            sum += (int32_t)tiles;
            table[g] = sum;
        }
        part[t] = sum;
        __syncthreads();
        for (int d = 1; d < kThreads; d <<= 1) {
            const int32_t v = t >= d ? part[t - d] : 0;
            __syncthreads();
            part[t] += v;
            __syncthreads();
        }
        const int32_t before = part[t] - sum;
        for (int e = 0; e < per; ++e)
            if (t * per + e < G) table[t * per + e] += before;
        __syncthreads();
    }
    S.total = (int64_t)uni((uint32_t)table[G - 1]);
    if (S.slot >= S.total) return;

    const uint32_t lda2 = (uint32_t)p.lda * 2u, ldb2 = (uint32_t)p.ldb * 2u;
    const uint32_t la = lds_addr(lds_a[0]), lb = lds_addr(lds_b[0]);
    Reader<TM, TA> ra;
    Reader<TN, TB> rb;
    ra.init(wm * MI, MI, lane);
    rb.init(wn * NJ, NJ, lane);

    // The loads run up to two stages ahead of the products, over the ends of
    // tiles: they have a walk of their own.
    Walk lw{S.slot, 0, false}, cw{S.slot, 0, false};
    Tile L = S.decode(p, lw);
    int ls = 0;
    auto issue = [&](int buf) {
        if (L.rows > 0) {
            const int64_t k0 = (int64_t)ls * SK;
            const int left = (int)(L.k - k0 < SK ? L.k - k0 : SK);  // <= 0: an empty contraction
            const uint32_t some = left > 0 ? 1u : 0u;
            const uint32_t abytes = TA ? ((uint32_t)(left - 1) * lda2 + (uint32_t)L.rows * 2u)
                                       : ((uint32_t)(L.rows - 1) * lda2 + (uint32_t)left * 2u);
            const uint32_t bbytes = TB ? ((uint32_t)(left - 1) * ldb2 + (uint32_t)L.cols * 2u)
                                       : ((uint32_t)(L.cols - 1) * ldb2 + (uint32_t)left * 2u);
            const i32x4 da = descriptor(L.a + (TA ? k0 * p.lda : k0), some * abytes);
            const i32x4 db = descriptor(L.b + (TB ? k0 * p.ldb : k0), some * bbytes);
            issue_loads<TM, kWaves, TA>(da, lda2, la + (uint32_t)buf * (TM * SK * 2), wave, lane, left);
            issue_loads<TN, kWaves, TB>(db, ldb2, lb + (uint32_t)buf * (TN * SK * 2), wave, lane, left);
            if (++ls == L.stages) {
                S.next(lw);
                L = S.decode(p, lw);
                ls = 0;
            }
        }
    };
    f32x16 acc[MI][NJ];
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;

    bf16x8 fa[2][MI], fb[2][NJ];
    auto read = [&](int set, int buf, int s) {
#pragma unroll
        for (int i = 0; i < MI; ++i) fa[set][i] = ra.read(lds_a[buf], i, s);
#pragma unroll
        for (int j = 0; j < NJ; ++j) fb[set][j] = rb.read(lds_b[buf], j, s);
    };
    // B rows as the instruction's rows and A rows as its columns: a lane then
    // holds 4 consecutive output columns of one output row
    auto multiply = [&](int set) {
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
            for (int j = 0; j < NJ; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fb[set][j], fa[set][i], acc[i][j], 0, 0, 0);
    };

    issue(0);
    issue(1);
    wait_loads<0>();
    __syncthreads();
    read(0, 0, 0);

    Tile C = S.decode(p, cw);
    int buf = 0;
    while (C.rows > 0) {
        for (int s = 0; s < C.stages; ++s) {
            read(1, buf, 1);
            multiply(0);
            read(0, buf, 2);
            multiply(1);
            read(1, buf, 3);
            multiply(0);
            wait_loads<0>();
            __syncthreads();
            issue(buf);
            buf ^= 1;
            read(0, buf, 0);
            multiply(1);
        }
        // lane l: output row 32 i + l % 32 of the wave's part and, in element
        // 4 q + u, column 32 j + 8 q + 4 (l / 32) + u
        const int h = lane >> 5, r32 = lane & 31;
        if (OUT == kBf16) {
            uint16_t* const out = (uint16_t*)p.out + C.out;
            const uint32_t ldo2 = (uint32_t)p.ldo * 2u;
            const rsrc_t rs = out_rsrc(out, (uint32_t)(C.rows - 1) * ldo2 + (uint32_t)C.cols * 2u);
#pragma unroll
            for (int i = 0; i < MI; ++i) {
                const int row = wm * WM + i * 32 + r32;
#pragma unroll
                for (int j = 0; j < NJ; ++j)
#pragma unroll
                    for (int q = 0; q < 4; q += 2) {
                        const uint32_t x0 = pack2(acc[i][j][4 * q + 0], acc[i][j][4 * q + 1]);
                        const uint32_t y0 = pack2(acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]);
                        const uint32_t x1 = pack2(acc[i][j][4 * q + 4], acc[i][j][4 * q + 5]);
                        const uint32_t y1 = pack2(acc[i][j][4 * q + 6], acc[i][j][4 * q + 7]);
                        // lanes l and l + 32 trade halves: 8 consecutive columns each
                        const auto sx = __builtin_amdgcn_permlane32_swap(x0, x1, false, false);
                        const auto sy = __builtin_amdgcn_permlane32_swap(y0, y1, false, false);
                        const int col = wn * WN + j * 32 + 8 * q + 8 * h;
                        const uint32_t off = row < C.rows && col < C.cols ? (uint32_t)row * ldo2 + (uint32_t)col * 2u
                                                                         : kOut;
                        __builtin_amdgcn_raw_buffer_store_b128(
                            u32x4{(uint32_t)sx[0], (uint32_t)sy[0], (uint32_t)sx[1], (uint32_t)sy[1]}, rs, (int)off, 0,
                            0);
                    }
            }
        } else {
            float* const out = (float*)p.out + C.out;
            const uint32_t ldo4 = (uint32_t)p.ldo * 4u;
#pragma unroll
            for (int i = 0; i < MI; ++i) {
                const int row = wm * WM + i * 32 + r32;
#pragma unroll
                for (int j = 0; j < NJ; ++j)
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int col = wn * WN + j * 32 + 8 * q + 4 * h;
                        if (row < C.rows && col < C.cols) {
                            f32x4* const d = (f32x4*)((char*)out + ((uint64_t)((uint32_t)row * (uint64_t)ldo4) + (uint32_t)col * 4u));
                            f32x4 v{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
                            if (OUT == kFp32Add) v += *d;
                            *d = v;
                        }
                    }
            }
        }
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
            for (int j = 0; j < NJ; ++j)
#pragma unroll
                for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;
        S.next(cw);
        C = S.decode(p, cw);
    }
    wait_loads<0>();
}

int cus() {
    static int cached[64] = {0};
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return 256;
    if (cached[dev] == 0) {
        int n = 0;
        if (hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || n <= 0) n = 256;
        cached[dev] = n;
    }
    return cached[dev];
}

int64_t tiles(int64_t n, int64_t t) { return (n + t - 1) / t; }

// Upper bound of the tiles of a launch: the rows split among G groups.
template <int MODE>
int64_t tile_bound(const Args& p, int64_t tm, int64_t tn) {
    if (MODE == kWgrad) return (int64_t)p.G * tiles(p.I, tm) * tiles(p.J, tn);
    const int64_t groups = p.G < p.M ? p.G : p.M;  // groups that can have rows
    return (tiles(p.M, tm) + groups) * tiles(p.J, tn);
}

template <int MODE, int OUT>
hipError_t launch(const Args& p, hipStream_t stream) {
    const unsigned table = 4u * (unsigned)p.G * (MODE == kWgrad && p.G <= kLptGroups ? 2u : 1u);
    const int64_t n = cus();
    const int64_t big = tile_bound<MODE>(p, 256, 256);
    if (big >= n) {
        const int64_t nwg = big < n ? big : n;
        hipLaunchKernelGGL((grouped_bf16_kernel<MODE, 256, 256, 128, 64, OUT>), dim3((unsigned)nwg), dim3(512), table,
                           stream, p);
    } else {
        const int64_t small = tile_bound<MODE>(p, 128, 128);
        const int64_t nwg = small < 2 * n ? small : 2 * n;
        hipLaunchKernelGGL((grouped_bf16_kernel<MODE, 128, 128, 64, 64, OUT>), dim3((unsigned)nwg), dim3(256), table,
                           stream, p);
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_grouped_bf16(const uint16_t* x, int64_t ldx, const uint16_t* w, const int32_t* offsets, int32_t G,
                               int64_t M, int64_t N, int64_t K, uint16_t* out, int64_t ldo, hipStream_t stream) {
    Args p = {x, w, offsets, out, ldx, K, ldo, M, 0, N, K, G};
    return launch<kForward, kBf16>(p, stream);
}

hipError_t launch_grouped_bf16_dgrad(const uint16_t* dy, int64_t ldy, const uint16_t* w, const int32_t* offsets,
                                     int32_t G, int64_t M, int64_t N, int64_t K, uint16_t* dx, int64_t ldx,
                                     hipStream_t stream) {
    Args p = {dy, w, offsets, dx, ldy, K, ldx, M, 0, K, N, G};
    return launch<kDgrad, kBf16>(p, stream);
}

hipError_t launch_grouped_bf16_wgrad(const uint16_t* dy, int64_t ldy, const uint16_t* x, int64_t ldx,
                                     const int32_t* offsets, int32_t G, int64_t M, int64_t N, int64_t K, void* dw,
                                     bool fp32, bool accumulate, hipStream_t stream) {
    Args p = {dy, x, offsets, dw, ldy, ldx, K, M, N, K, 0, G};
    if (!fp32) return launch<kWgrad, kBf16>(p, stream);
    return accumulate ? launch<kWgrad, kFp32Add>(p, stream) : launch<kWgrad, kFp32>(p, stream);
}

}  // namespace mx
