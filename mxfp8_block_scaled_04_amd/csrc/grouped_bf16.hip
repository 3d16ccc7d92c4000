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
// What bounds it: with many rows a group the operand loads and the matrix
// pipes, at the clock that the power limit leaves (forward, 32768 x 4096 x
// 7168, 16 groups: 1.65-1.67 ms, 1.16 PFLOP/s, pipes busy 68 %; dgrad, 7168 x
// 2048: 0.89 ms, of which 15 % are a last round of tiles for a quarter of the
// CUs; wgrad of the same to bf16 0.84 ms, to fp32 0.95 ms, added to fp32 values
// 1.13 ms, of which the values are 1.9 GB); with few rows reading the weights
// (few_rows_kernel); with thousands of groups finding the tiles' groups (256 x
// 256 weights, 16 rows a group: 128 groups 19 us, 1024 groups 109 us, 4096
// groups 856 us).
//
// Layout: persistent workgroups of 4 waves, one 256 x 256 tile per CU (128 x
// 128 per wave) or two 128 x 128 tiles per CU (64 x 64 per wave),
// v_mfma_f32_32x32x16_bf16.  A stage is 64 contraction elements of both
// operands (64 KB for the large tile), loaded straight into LDS by 16-byte
// direct loads; two stages in LDS (four for small tiles that have a CU to
// themselves).  A stage has 4 steps of 16: the fragments of a step are read
// while the one before is multiplied, also across stages and tiles.  The wait
// for the next stage and the barrier sit before a stage's last step, whose
// fragments are in registers by then; the loads of the stage after the next go
// into the buffer freed by that barrier, spread over two steps.
// Tried and slower at 32768 x 4096 x 7168 (16 groups, 1.63 ms as it is, 1.18
// ms without its loads): 8 waves of 128 x 64 (1.73 ms: a third more LDS
// reads), the same in two groups of opposite phase (1.72 ms), stages of 32
// with 4 in LDS (1.78 ms: 64-byte pieces of rows double the requests to L2),
// all loads in one step (1.74 ms), loads spread over three (1.63 ms).
//
// Bounds: all loads go through buffer descriptors that end at the operand's
// last valid element; what lies past it reads as zero.  Rows of a tile past
// its group, contraction indices past K (N for dgrad, the group's rows for
// wgrad) and stages past the last tile need no other care, except granules
// past K inside a row, whose offsets are moved out of range.
#include <type_traits>

#include "mx_debug.h"
#include "mx_train.h"

namespace mx {
namespace {

constexpr int SK = 64;          // contraction elements per stage
constexpr int kSteps = SK / 16;  // matrix instructions along it
constexpr int kLptGroups = 512;  // wgrad: groups taken longest first up to this many
constexpr int kBand = 4;         // row tiles per band of the tile order
// An offset past every descriptor (fewer than 2^31 bytes: 256 rows of fewer
// than 2^22 elements), which no scalar offset of a load (below 2^31 too)
// carries past 2^32.
constexpr uint32_t kOut = 0x80000000u;
// The same for the result, whose tile can span up to 2^32 - 8192 bytes and
// whose accesses have no scalar offset.
constexpr uint32_t kOutStore = 0xFFFFFFF0u;

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
    int32_t G;              // groups (wgrad: slices, `split` of each group)
    int32_t split;          // wgrad: slices of each group's rows (1 otherwise)
    int32_t max_tiles;      // what valid offsets can give at most (malformed ones are cut off there)
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
// [lds + OFF + 16 l, lds + OFF + 16 l + 16).  In assembly without an output
// register: the compiler would otherwise wait for it before every LDS read.
// It is waited for by wait_loads and a barrier before the data is read.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
template <int OFF>
__device__ __forceinline__ void load_to_lds(const i32x4& rs, uint32_t voff, uint32_t soff, uint32_t lds) {
    asm volatile("s_add_u32 m0, %3, %4\n\ts_nop 0\n\tbuffer_load_dwordx4 %0, %1, %2 offen lds" ::"v"(voff), "s"(rs),
                 "s"(soff), "s"(lds), "n"(OFF)
                 : "memory", "m0", "scc");
}
#pragma clang diagnostic pop
template <int N>
__device__ __forceinline__ void wait_loads() {
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// A barrier of the workgroup at which this wave's LDS reads are complete and
// over which the compiler moves nothing.  (No wait for its loads to LDS.)
__device__ __forceinline__ void meet() {
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
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
// position c ^ (r >> 1 & 7).  A fragment read takes one granule of each of 32
// rows and is served 16 lanes (256 bytes) at a time; the swizzle spreads them
// over all banks.
//
// T = true: contraction row k at 2 ROWS k; its 32-byte unit u (tile rows 16 u
// ...) at position u ^ f(k), f(k) = 2 (k & 3) | (k >> 3 & 1).  A transposing
// read of 64 lanes takes 64 bytes from each of the 8 contraction rows
// k0 + {0..3, 8..11}; f puts them into different banks.

// Position of granule `pos` of staged row `row` (and back: the swizzles are
// their own inverses).
template <bool T>
__device__ __forceinline__ uint32_t swizzled(uint32_t row, uint32_t pos) {
    if (T) {
        const uint32_t f = ((row & 3u) << 1) | ((row >> 3) & 1u);
        return (((pos >> 1) ^ f) << 1) | (pos & 1u);
    }
    return pos ^ ((row >> 1) & 7u);
}

// The loads of a stage of one operand by the 4 waves: kLoads instructions of
// 1 KB each, wave w those from w kLoads on; instruction q covers the staged
// rows [q kRows, (q + 1) kRows), 128-byte pieces or longer (with 64-byte
// pieces L2 is asked twice as often and the address unit is busy twice as
// long).  A lane's granule follows from the swizzle of its row, which takes
// kKinds values over the instructions of a wave.
template <int ROWS, bool T>
struct Loader {
    static constexpr int kLoads = ROWS * SK * 2 / 1024 / 4;
    static constexpr int kPerRow = T ? ROWS / 8 : SK / 8;  // granules per staged row
    static constexpr int kRows = 64 / kPerRow;
    static constexpr int kKinds = T && ROWS == 256 ? 4 : 2;
    __device__ __forceinline__ static constexpr int kind(int j) {
        return !T ? j & 1 : ROWS == 256 ? (j & 1) | (j >> 2 & 1) << 1 : j >> 1 & 1;
    }
    uint32_t voff[kKinds];   // byte offset of the lane's granule in an instruction's rows
    uint32_t whole[kKinds];  // T = false: the same without the contraction's end
    uint32_t soff[kLoads], lds0;
    i32x4 d;        // descriptor of the stage to load
    int64_t rest;   // contraction elements of the tile from that stage on
    uint32_t lds;

    __device__ __forceinline__ void init(uint32_t ld2, uint32_t lds_base, int wave, int lane) {
        const uint32_t row = (uint32_t)(lane / kPerRow), pos = (uint32_t)(lane % kPerRow);
        const uint32_t row0 = (uint32_t)(wave * kLoads * kRows);
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
            const uint32_t g = swizzled<T>(row0 + (uint32_t)(j * kRows) + row, pos);
            voff[kind(j)] = whole[kind(j)] = row * ld2 + g * 16u;
            soff[j] = uni((row0 + (uint32_t)(j * kRows)) * ld2);
        }
        lds0 = uni(lds_base + (uint32_t)(wave * kLoads) * 1024u);
    }
    // Descriptor of a stage of `left` (1 .. SK) contraction elements at p;
    // `wide`: valid tile rows.
    __device__ __forceinline__ void aim(const void* p, uint32_t wide, uint32_t left, uint32_t ld2) {
        d = descriptor(p, T ? (left - 1) * ld2 + wide * 2u : (wide - 1) * ld2 + left * 2u);
        if (!T) {  // granules past the contraction's end
            const uint32_t ld_row = (uint32_t)((threadIdx.x & 63) / kPerRow) * ld2;
#pragma unroll
            for (int k = 0; k < kKinds; ++k) voff[k] = whole[k] - ld_row < left * 2u ? whole[k] : kOut;
        }
    }
    // The first stage of a tile; without one (wide = 0) an endless row of
    // stages that end at once.
    __device__ __forceinline__ void start(const void* p, uint32_t wide, int64_t k, uint32_t ld2) {
        rest = k;
        if (wide == 0 || k <= 0) {
            d = descriptor(p, 0);
            if (wide == 0) rest = INT64_MAX;
        } else {
            aim(p, wide, (uint32_t)(k < SK ? k : SK), ld2);
        }
    }
    // On to the next stage; false at the tile's end.
    __device__ __forceinline__ bool advance(uint32_t wide, uint32_t ld2) {
        rest -= SK;
        const uint64_t base = ((uint64_t)(uint32_t)d[1] << 32 | (uint32_t)d[0]) + (T ? SK * (uint64_t)ld2 : SK * 2u);
        if (rest >= SK) {
            d[0] = (int)(uint32_t)base;
            d[1] = (int)(uint32_t)(base >> 32);
            return true;
        }
        if (rest <= 0) return false;
        aim((const void*)base, wide, (uint32_t)rest, ld2);
        return true;
    }
    __device__ __forceinline__ void begin(int slot) {
        lds = uni(lds0 + (uint32_t)slot * (ROWS * SK * 2));
    }
    template <int J>
    __device__ __forceinline__ void load() {
        load_to_lds<J * 1024>(d, voff[kind(J)], soff[J], lds);
    }
    // instruction j of the wave
    __device__ __forceinline__ void load(int j) {
        if (j == 0) load<0>();
        if (j == 1) load<1>();
        if (j == 2) load<2>();
        if (j == 3) load<3>();
        if constexpr (kLoads == 8) {
            if (j == 4) load<4>();
            if (j == 5) load<5>();
            if (j == 6) load<6>();
            if (j == 7) load<7>();
        }
    }
};

// Fragment of tile rows [32 blk, 32 blk + 32), step s of a stage: lane l
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

// A workgroup's way through its tiles, one in each round.
struct Walk {
    int r = 0;  // round of the next tile
    int g = 0;  // position in tile order, for the search of the tile's group
};

template <int MODE, int TM, int TN>
struct Sched {
    int total;
    int nwg, slot;
    bool lpt;
    const int32_t* tile_end;  // LDS: inclusive prefix of tiles per position
    const int32_t* order;     // LDS: group at a position (lpt)

    // (constant address space: a scalar load where g is uniform, which no
    // wait for vector loads delays)
    __device__ __forceinline__ static int64_t bound(const Args& p, int64_t g) {
        const int64_t v = ((const __attribute__((address_space(4))) int32_t*)p.offsets)[g];
        return v < 0 ? 0 : (v > p.M ? p.M : v);
    }
    // First row and rows of a group, or of a slice of one: slices are whole
    // stages long, the last ones of a group may be short or empty.
    __device__ __forceinline__ static int64_t range_of(const Args& p, int g, int64_t& first) {
        const int s = MODE == kWgrad && p.split > 1 ? g % p.split : 0;
        const int grp = MODE == kWgrad && p.split > 1 ? g / p.split : g;
        first = bound(p, grp);
        int64_t n = bound(p, grp + 1) - first;
        if (n < 0) n = 0;
        if (MODE == kWgrad && p.split > 1) {
            const int64_t len = ((n + p.split - 1) / p.split + SK - 1) / SK * SK;
            const int64_t skip = s * len < n ? s * len : n;
            first += skip;
            n = n - skip < len ? n - skip : len;
        }
        return n;
    }
    __device__ __forceinline__ static int64_t rows_of(const Args& p, int g) {
        int64_t first;
        return range_of(p, g, first);
    }

    __device__ __forceinline__ Tile decode(const Args& p, Walk& w) const {
        Tile T;
        const int tile = tile_of(w.r);
        if (tile >= total) {
            T.a = p.a;
            T.b = p.b;
            T.out = 0;
            T.k = 0;
            T.rows = T.cols = 0;
            T.stages = 1;
            return T;
        }
        while (tile_end[w.g] <= tile) ++w.g;
        w.g = (int)uni((uint32_t)w.g);
        const int first = w.g > 0 ? (int)uni((uint32_t)tile_end[w.g - 1]) : 0;
        const uint32_t local = uni((uint32_t)(tile - first));
        const int grp = (int)uni((uint32_t)(lpt ? order[w.g] : w.g));
        int64_t o0;
        const int64_t mg = range_of(p, grp, o0);
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
    // Round r of this workgroup: tile r nwg + slot; with the groups taken
    // longest first, in alternating directions, which evens out the sums.
    __device__ __forceinline__ int tile_of(int r) const {
        return r * nwg + (lpt && (r & 1) ? nwg - 1 - slot : slot);
    }
};

__device__ __forceinline__ uint32_t pack2(float x, float y) {
    const uint32_t lo = __builtin_bit_cast(uint16_t, (__bf16)x), hi = __builtin_bit_cast(uint16_t, (__bf16)y);
    return lo | (hi << 16);
}

// Keeps the accumulators of row blocks i and on where the matrix instructions
// leave them: otherwise all of them are copied out before the first store.
template <int MI, int NJ>
__device__ __forceinline__ void keep_acc(f32x16 (&acc)[MI][NJ], int i) {
#pragma unroll
    for (int k = 0; k < MI; ++k)
#pragma unroll
        for (int j = 0; j < NJ; ++j)
            if (k >= i) asm volatile("" : "+a"(acc[k][j]));
}

// RING: stages in LDS.
template <int MODE, int TM, int TN, int WM, int WN, int OUT, int RING>
__global__ __launch_bounds__((TM / WM) * (TN / WN) * 64, TM * RING >= 512 ? 1 : 2) void grouped_bf16_kernel(Args p) {
    constexpr int kWaves = (TM / WM) * (TN / WN);
    static_assert(kWaves == 4 && TM == TN, "each wave loads a quarter of both operands");
    constexpr int MI = WM / 32, NJ = WN / 32;
    constexpr bool TA = MODE == kWgrad, TB = MODE != kForward;
    constexpr int kThreads = kWaves * 64;
    __shared__ __attribute__((aligned(16))) uint8_t lds_a[RING][TM * SK * 2];
    __shared__ __attribute__((aligned(16))) uint8_t lds_b[RING][TN * SK * 2];
    __shared__ int64_t part[kWaves];
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
        const int groups = G / p.split;
        for (int g = t; g <= groups; g += kThreads)
            debug_flag(offsets_entry_bad(p.offsets, g, groups, p.M), kDbgOffsets);
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
        const auto tiles_at = [&](int g) {
            const int64_t mg = S.rows_of(p, S.lpt ? order[g] : g);
            // a weight gradient without rows is zero: one empty stage, unless it is added to
            return MODE == kWgrad ? (OUT == kFp32Add && mg == 0 ? 0 : (p.I + TM - 1) / TM * nJ)
                                  : (mg + TM - 1) / TM * nJ;
        };
        int64_t sum = 0;
        for (int e = 0; e < per; ++e)
            if (t * per + e < G) sum += tiles_at(t * per + e);
        int64_t upto = sum;
        for (int d = 1; d < 64; d <<= 1) {
            const int64_t v = __shfl_up(upto, d, 64);
            if (lane >= d) upto += v;
        }
        if (lane == 63) part[wave] = upto;
        __syncthreads();
        int64_t so_far = upto - sum;
        for (int w = 0; w < wave; ++w) so_far += part[w];
        for (int e = 0; e < per; ++e)
            if (t * per + e < G) {
                so_far += tiles_at(t * per + e);
                table[t * per + e] = (int32_t)(so_far < p.max_tiles ? so_far : p.max_tiles);
            }
        __syncthreads();
    }
    S.total = (int)uni((uint32_t)table[G - 1]);
    if (S.slot >= S.total) return;

    const uint32_t lda2 = (uint32_t)p.lda * 2u, ldb2 = (uint32_t)p.ldb * 2u;
    Reader<TM, TA> ra;
    Reader<TN, TB> rb;
    ra.init(wm * MI, MI, lane);
    rb.init(wn * NJ, NJ, lane);
    Loader<TM, TA> qa;
    Loader<TN, TB> qb;
    qa.init(lda2, lds_addr(lds_a[0]), wave, lane);
    qb.init(ldb2, lds_addr(lds_b[0]), wave, lane);
    constexpr int kLoads = Loader<TM, TA>::kLoads;  // of each operand, per wave and stage

    // The loads run RING stages ahead of the products, over the ends of tiles:
    // they have a walk of their own.  A's go first; L is the tile they are in,
    // and B follows a step later.
    Walk lw, cw;
    Tile L = S.decode(p, lw);
    uint32_t bcols = (uint32_t)L.cols;
    qa.start(L.a, (uint32_t)L.rows, L.k, lda2);
    qb.start(L.b, (uint32_t)L.cols, L.k, ldb2);
    auto advance_a = [&]() {
        if (!qa.advance((uint32_t)L.rows, lda2)) {
            ++lw.r;
            L = S.decode(p, lw);
            qa.start(L.a, (uint32_t)L.rows, L.k, lda2);
        }
    };
    auto advance_b = [&]() {
        if (!qb.advance(bcols, ldb2)) {
            bcols = (uint32_t)L.cols;
            qb.start(L.b, bcols, L.k, ldb2);
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
    // fragment f of step k of a stage, B's first: a step's products begin with them
    auto read = [&](int slot, int k, int f) {
        if (f < NJ) fb[k & 1][f] = rb.read(lds_b[slot], f, k);
        else fa[k & 1][f - NJ] = ra.read(lds_a[slot], f - NJ, k);
    };
    // Step k of a stage: its products, and between them the reads of the next
    // step (from ring slot rslot) and loads into slot lslot: A's of a stage in
    // the last step of a stage, B's of the same stage in the first step of the
    // next one.
    // The empty statements keep this order: the compiler would otherwise
    // gather the reads next to their first use.
    // B rows as the instruction's rows and A rows as its columns: a lane then
    // holds 4 consecutive output columns of one output row.
    auto step = [&](auto which, int rslot, int lslot) {
        constexpr int k = decltype(which)::value, set = k & 1;
        constexpr int kMul = MI * NJ, kReads = MI + NJ;
        if (k == kSteps - 1) qa.begin(lslot);
        if (k == 0) qb.begin(lslot);
#pragma unroll
        for (int m = 0; m < kMul; ++m) {
            const int i = m / NJ, j = m % NJ;
            acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fb[set][j], fa[set][i], acc[i][j], 0, 0, 0);
#pragma unroll
            for (int f = 0; f < kReads; ++f)
                if (f * kMul * 5 / 8 / kReads == m) read(rslot, (k + 1) % kSteps, f);
#pragma unroll
            for (int q = kLoads * m / kMul; q < kLoads * (m + 1) / kMul; ++q) {
                if (k == kSteps - 1) qa.load(q);
                if (k == 0) qb.load(q);
            }
            if (m + 1 < kMul) asm volatile("" : "+v"(fb[set][j]), "+v"(fa[set][(m + 1) / NJ]) : : "memory");
        }
    };

    // the first RING stages but for B's part of the last one, which the first
    // step loads
#pragma unroll
    for (int k = 0; k < RING; ++k) {
        qa.begin(k);
#pragma unroll
        for (int m = 0; m < kLoads; ++m) qa.load(m);
        if (k + 1 < RING) {
            qb.begin(k);
#pragma unroll
            for (int m = 0; m < kLoads; ++m) qb.load(m);
            advance_a();
            advance_b();
        }
    }
    wait_loads<(2 * RING - 3) * kLoads>();
    meet();
#pragma unroll
    for (int f = 0; f < MI + NJ; ++f) read(0, 0, f);

    Tile C = S.decode(p, cw);
    int slot = 0;
    while (C.rows > 0) {
        for (int s = 0; s < C.stages; ++s) {
            const int next = (slot + 1) & (RING - 1);
            step(std::integral_constant<int, 0>(), slot, (slot + RING - 1) & (RING - 1));
            advance_a();
            step(std::integral_constant<int, 1>(), slot, 0);
            advance_b();
            step(std::integral_constant<int, 2>(), slot, 0);
            // the next stage has landed, and every wave has read this one
            wait_loads<(RING - 2) * 2 * kLoads>();
            meet();
            step(std::integral_constant<int, 3>(), next, slot);
            slot = next;
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
                keep_acc<MI, NJ>(acc, i);
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
                                                                         : kOutStore;
                        __builtin_amdgcn_raw_buffer_store_b128(
                            u32x4{(uint32_t)sx[0], (uint32_t)sy[0], (uint32_t)sx[1], (uint32_t)sy[1]}, rs, (int)off, 0,
                            0);
                    }
            }
        } else {
            // block by block, the values added to read a block ahead
            const uint32_t ldo4 = (uint32_t)p.ldo * 4u;
            const rsrc_t rs = out_rsrc((float*)p.out + C.out, (uint32_t)(C.rows - 1) * ldo4 + (uint32_t)C.cols * 4u);
            u32x4 old[2][4];
            const auto at = [&](int c, int q) {
                const int row = wm * WM + (c / NJ) * 32 + r32, col = wn * WN + (c % NJ) * 32 + 8 * q + 4 * h;
                return (int)(row < C.rows && col < C.cols ? (uint32_t)row * ldo4 + (uint32_t)col * 4u : kOutStore);
            };
            const auto fetch = [&](int c) {
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    old[c & 1][q] = __builtin_amdgcn_raw_buffer_load_b128(rs, at(c, q), 0, 0);
            };
            if (OUT == kFp32Add) fetch(0);
#pragma unroll
            for (int c = 0; c < MI * NJ; ++c) {
                keep_acc<MI, NJ>(acc, c / NJ);
                __builtin_amdgcn_sched_barrier(0);  // (all reads at once would not fit in registers)
                if (OUT == kFp32Add && c + 1 < MI * NJ) fetch(c + 1);
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const f32x16& x = acc[c / NJ][c % NJ];
                    f32x4 v{x[4 * q], x[4 * q + 1], x[4 * q + 2], x[4 * q + 3]};
                    if (OUT == kFp32Add) v += __builtin_bit_cast(f32x4, old[c & 1][q]);
                    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, v), rs, at(c, q), 0, 0);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
            for (int j = 0; j < NJ; ++j)
#pragma unroll
                for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;
        ++cw.r;
        C = S.decode(p, cw);
    }
    wait_loads<0>();
}

// ---- few rows --------------------------------------------------------------
//
// Forward product where groups have few rows (a token or some in generation):
// bound by reading the weights of the groups that have any, once.  A
// workgroup takes 16 columns of the output for up to 16 rows of one group;
// its 8 waves share the contraction out in pieces of 4 steps of 32 and add
// their sums up in LDS, in a fixed order.  v_mfma_f32_16x16x32_bf16 with the
// weights as its rows: a lane reads 16 bytes of row l % 16, so that a load
// takes 64 bytes of each of 16 rows, straight into registers, and the loads
// of a piece are in flight while the one before is multiplied.  Columns and
// rows past their ends read as zeros (descriptors), and so do contraction
// indices past K.
// Measured at N 4096, K 7168: 8 rows of 8 groups 79 us, 6.0 TB/s (128-row
// tiles 119 us); 64 rows of 64 groups 386 us, 6.2 TB/s; one row 13 us (68 us).
// 32 columns and 4 waves per workgroup: 86, 434 and 18 us.
constexpr int kFewWaves = 8;
__global__ __launch_bounds__(kFewWaves * 64) void few_rows_kernel(Args p) {
    constexpr int kPiece = 4, WAVES = kFewWaves;
    __shared__ f32x4 sums[WAVES][64];
    __shared__ int32_t found[3];  // group, first row, rows
    __shared__ int32_t part[WAVES];
    const int t = threadIdx.x, wave = (int)uni((uint32_t)t >> 6), lane = t & 63;

    // The workgroup's block of up to 16 rows: the blockIdx.y-th of all groups.
    // Each thread counts the blocks of some groups; then a prefix over the
    // threads.
    {
        if (t == 0) found[0] = -1;
        for (int g = t; g <= p.G; g += WAVES * 64)
            debug_flag(offsets_entry_bad(p.offsets, g, p.G, p.M), kDbgOffsets);
        const int per = (p.G + WAVES * 64 - 1) / (WAVES * 64);
        const auto rows_at = [&](int g, int64_t& lo) {
            lo = Sched<kForward, 256, 256>::bound(p, g);
            const int64_t n = Sched<kForward, 256, 256>::bound(p, g + 1) - lo;
            return n > 0 ? n : 0;
        };
        int mine = 0;
        int64_t lo;
        for (int e = 0; e < per; ++e)
            if (t * per + e < p.G) mine += (int)((rows_at(t * per + e, lo) + 15) / 16);
        int upto = mine;
        for (int d = 1; d < 64; d <<= 1) {
            const int v = __shfl_up(upto, d, 64);
            if (lane >= d) upto += v;
        }
        if (lane == 63) part[wave] = upto;
        __syncthreads();
        int at = upto - mine;
        for (int w = 0; w < wave; ++w) at += part[w];
        const int want = (int)blockIdx.y;
        if (at <= want && want < at + mine)
            for (int e = 0; e < per; ++e) {
                if (t * per + e >= p.G) break;
                const int64_t n = rows_at(t * per + e, lo);
                const int blocks = (int)((n + 15) / 16);
                if (want < at + blocks) {
                    const int64_t first = (int64_t)(want - at) * 16;
                    found[0] = t * per + e;
                    found[1] = (int)(lo + first);
                    found[2] = (int)(n - first < 16 ? n - first : 16);
                    break;
                }
                at += blocks;
            }
        __syncthreads();
    }
    const int g = (int)uni((uint32_t)found[0]);
    if (g < 0) return;
    const int64_t row0 = (int64_t)uni((uint32_t)found[1]);
    const int rows = (int)uni((uint32_t)found[2]);
    const int64_t n0 = (int64_t)blockIdx.x * 16;
    const int cols = (int)(p.J - n0 < 16 ? p.J - n0 : 16);
    const uint32_t K = (uint32_t)p.K, lda2 = (uint32_t)p.lda * 2u;
    const rsrc_t rw = out_rsrc((void*)(p.b + ((int64_t)g * p.J + n0) * p.K), (uint32_t)cols * K * 2u);
    const rsrc_t rx = out_rsrc((void*)(p.a + row0 * p.lda), (uint32_t)(rows - 1) * lda2 + K * 2u);
    const uint32_t r16 = (uint32_t)lane & 15u, k8 = ((uint32_t)lane >> 4) * 8u;

    struct Piece {
        bf16x8 w[kPiece], x[kPiece];
    };
    const auto fetch = [&](Piece& f, uint32_t piece) {
#pragma unroll
        for (int s = 0; s < kPiece; ++s) {
            const uint32_t k = (piece * kPiece + (uint32_t)s) * 32u + k8;
            const uint32_t xo = k < K ? r16 * lda2 + k * 2u : kOutStore;
            const uint32_t wo = k < K ? r16 * K * 2u + k * 2u : kOutStore;
            f.x[s] = __builtin_bit_cast(bf16x8, __builtin_amdgcn_raw_buffer_load_b128(rx, (int)xo, 0, 0));
            f.w[s] = __builtin_bit_cast(bf16x8, __builtin_amdgcn_raw_buffer_load_b128(rw, (int)wo, 0, 0));
        }
    };
    f32x4 acc{0.0f, 0.0f, 0.0f, 0.0f};
    const auto multiply = [&](const Piece& f) {
#pragma unroll
        for (int s = 0; s < kPiece; ++s)
            acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f.w[s], f.x[s], acc, 0, 0, 0);
    };
    const uint32_t pieces = (K + 32 * kPiece - 1) / (32 * kPiece);
    if ((uint32_t)wave < pieces) {
        Piece f0, f1;
        fetch(f0, (uint32_t)wave);
        for (uint32_t c = (uint32_t)wave;; c += 2 * WAVES) {
            // (a piece past the end reads nothing: all of its indices are past K)
            fetch(f1, c + WAVES);
            multiply(f0);
            if (c + WAVES >= pieces) break;
            fetch(f0, c + 2 * WAVES);
            multiply(f1);
            if (c + 2 * WAVES >= pieces) break;
        }
    }
    sums[wave][lane] = acc;
    __syncthreads();
    // lane l: output row l % 16, columns 4 (l / 16) .. + 3
    if (wave == 0) {
        f32x4 v = sums[0][lane];
#pragma unroll
        for (int w = 1; w < WAVES; ++w) v += sums[w][lane];
        const int col = 4 * (lane >> 4);
        if ((int)r16 < rows && col < cols) {
            uint16_t* const out = (uint16_t*)p.out + (row0 + r16) * p.ldo + n0 + col;
            *(uint2*)out = make_uint2(pack2(v[0], v[1]), pack2(v[2], v[3]));
        }
    }
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

// Whether a forward product goes to few_rows_kernel: on average at most 8 rows
// a group (16 groups, 4096 x 7168: 64 rows 99 against 121 us in tiles, 128 rows
// 198 us in both, 256 rows 278 against 199; 1024 rows of 128 groups are past the
// break-even, 1520 against 1218 us), or few rows at all, where tiles leave most
// CUs idle (one group, 4096 x 7168: 16 rows 17 against 49 us, 32 rows 28 against
// 49, 64 rows 53 against 49; at 1024 x 1024, 64 rows, 11 against 13).  The host
// knows the average only: each 16 rows of a group read its weights again, so
// that 1000 rows which all fall to one of 128 groups take 798 us (108 in tiles).
bool few_rows(const Args& p) { return p.M <= 8 * (int64_t)p.G || p.M <= 64; }

template <int MODE, int OUT>
hipError_t launch(Args p, hipStream_t stream) {
    const unsigned table = 4u * (unsigned)p.G * (MODE == kWgrad && p.G <= kLptGroups ? 2u : 1u);
    const int64_t n = cus();
    const int64_t big = tile_bound<MODE>(p, 256, 256);
    // 256 x 256 tiles where they keep three quarters of the CUs busy (192
    // tiles: 87 against 115 us at 2048 x 4096 x 4096, 4 groups; 128 tiles: 46
    // against 33 us at 2048 x 2048 x 2048, 8 groups), unless the groups are
    // as short as a small tile (64 rows a group on average, 4096 x 4096 x
    // 4096: 457 against 435 us; 128 rows, 16384 x 2048 x 7168: 992 against 960)
    // In wgrad, where a short contraction leaves the writing of the tiles to
    // wait for: at least 4 tiles per CU (512 tiles, 256 rows a group: 41
    // against 35 us; 1024 tiles: 63 against 64 us), or 1024 rows a group.
    const bool fits = MODE == kWgrad ? big >= 4 * n || p.M >= 1024 * (int64_t)p.G : p.M > 128 * (int64_t)p.G;
    const auto most = [](int64_t tiles) { return (int32_t)(tiles < (1 << 30) ? tiles : 1 << 30); };
    if (big >= n * 3 / 4 && fits) {
        p.max_tiles = most(big);
        const int64_t nwg = big < n ? big : n;
        hipLaunchKernelGGL((grouped_bf16_kernel<MODE, 256, 256, 128, 128, OUT, 2>), dim3((unsigned)nwg), dim3(256),
                           table, stream, p);
        return hipGetLastError();
    }
    // 128 x 128 tiles, two workgroups per CU; with at most one per CU, four
    // stages in LDS in place of two (the loads' latency is what bounds a
    // workgroup that is alone)
    const int64_t small = tile_bound<MODE>(p, 128, 128);
    p.max_tiles = most(small);
    if (small > n) {
        const int64_t nwg = small < 2 * n ? small : 2 * n;
        hipLaunchKernelGGL((grouped_bf16_kernel<MODE, 128, 128, 64, 64, OUT, 2>), dim3((unsigned)nwg), dim3(256), table,
                           stream, p);
    } else {
        const int64_t nwg = small < n ? small : n;
        hipLaunchKernelGGL((grouped_bf16_kernel<MODE, 128, 128, 64, 64, OUT, 4>), dim3((unsigned)nwg), dim3(256), table,
                           stream, p);
    }
    return hipGetLastError();
}

// out[g][i] = (out[g][i] +) the sum of the `split` slices' products, in order
// of the slices; 4 elements per lane (n % 4 == 0).
template <int OUT>
__global__ __launch_bounds__(256) void join_kernel(const float* part, int64_t n, int32_t split, void* out) {
    const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
    if (i >= n) return;
    const float* const from = part + (int64_t)blockIdx.y * split * n + i;
    f32x4 v = *(const f32x4*)from;
    for (int s = 1; s < split; ++s) v += *(const f32x4*)(from + s * n);
    const int64_t to = (int64_t)blockIdx.y * n + i;
    if (OUT == kBf16) {
        *(uint2*)((uint16_t*)out + to) = make_uint2(pack2(v[0], v[1]), pack2(v[2], v[3]));
    } else {
        f32x4* const d = (f32x4*)((float*)out + to);
        if (OUT == kFp32Add) v += *d;
        *d = v;
    }
}

}  // namespace

#ifdef MXMOE_DEBUG
hipError_t debug_take_grouped_bf16(uint32_t* out) { return debug_take_word(out); }
#endif

hipError_t launch_grouped_bf16(const uint16_t* x, int64_t ldx, const uint16_t* w, const int32_t* offsets, int32_t G,
                               int64_t M, int64_t N, int64_t K, uint16_t* out, int64_t ldo, hipStream_t stream) {
    Args p = {x, w, offsets, out, ldx, K, ldo, M, 0, N, K, G, 1, 0};
    if (few_rows(p)) {
        const int64_t blocks = M < G + M / 16 ? M : G + M / 16;  // of 16 rows, at most
        hipLaunchKernelGGL(few_rows_kernel, dim3((unsigned)tiles(N, 16), (unsigned)blocks), dim3(kFewWaves * 64), 0,
                           stream, p);
        return hipGetLastError();
    }
    return launch<kForward, kBf16>(p, stream);
}

hipError_t launch_grouped_bf16_dgrad(const uint16_t* dy, int64_t ldy, const uint16_t* w, const int32_t* offsets,
                                     int32_t G, int64_t M, int64_t N, int64_t K, uint16_t* dx, int64_t ldx,
                                     hipStream_t stream) {
    Args p = {dy, w, offsets, dx, ldy, K, ldx, M, 0, K, N, G, 1, 0};
    return launch<kDgrad, kBf16>(p, stream);
}

// Slices of each group's rows: where small tiles leave workgroup slots empty
// and the groups are long, so that a slice has 1024 rows or more on average
// (65536 rows, 8 groups, 512 x 512, 4 slices each: 52 us, 62 us without; where
// one group has 45 % of the rows, whose slices are the longest, 109 and 195 us).
int32_t wgrad_split(int32_t G, int64_t M, int64_t N, int64_t K) {
    const int64_t small = (int64_t)G * tiles(N, 128) * tiles(K, 128), slots = 512;
    int64_t s = small > 0 ? slots / small : 1;
    if (s > M / (1024 * (int64_t)G)) s = M / (1024 * (int64_t)G);
    if (s > 32) s = 32;
    return s < 2 ? 1 : (int32_t)s;
}

hipError_t launch_grouped_bf16_wgrad(const uint16_t* dy, int64_t ldy, const uint16_t* x, int64_t ldx,
                                     const int32_t* offsets, int32_t G, int64_t M, int64_t N, int64_t K, void* dw,
                                     bool fp32, bool accumulate, float* workspace, int64_t workspace_bytes,
                                     hipStream_t stream) {
    Args p = {dy, x, offsets, dw, ldy, ldx, K, M, N, K, 0, G, 1, 0};
    const int32_t split = wgrad_split(G, M, N, K);
    if (split > 1 && workspace && workspace_bytes >= 4 * (int64_t)split * G * N * K) {
        p.out = workspace;
        p.G = G * split;
        p.split = split;
        const hipError_t e = launch<kWgrad, kFp32>(p, stream);
        if (e != hipSuccess) return e;
        const int64_t n = N * K;
        const dim3 grid((unsigned)tiles(n, 1024), (unsigned)G);
        if (!fp32) hipLaunchKernelGGL(join_kernel<kBf16>, grid, dim3(256), 0, stream, workspace, n, split, dw);
        else if (accumulate)
            hipLaunchKernelGGL(join_kernel<kFp32Add>, grid, dim3(256), 0, stream, workspace, n, split, dw);
        else hipLaunchKernelGGL(join_kernel<kFp32>, grid, dim3(256), 0, stream, workspace, n, split, dw);
        return hipGetLastError();
    }
    if (!fp32) return launch<kWgrad, kBf16>(p, stream);
    return accumulate ? launch<kWgrad, kFp32Add>(p, stream) : launch<kWgrad, kFp32>(p, stream);
}

}  // namespace mx
