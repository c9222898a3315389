// linear_kernels.hip -- the products of a linear layer on the matrix cores, each
// with its epilogue:
//   forward          y  = residual + D(act(x W^T + b))
//   gradient, input  dx = D'(dz W) * act'(z)
//   gradient, weight dW = [dW +] dz^T x,  db = [db +] column sums of dz
// All three are one kernel: C[p, q] = sum_r A(p, r) B(q, r) in bf16 with fp32
// sums, where an operand holds either its outer index in rows (r contiguous) or
// the reduction index ("reduced rows", o contiguous).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "layer_device.h"
#include "tile_device.h"

namespace zk {

constexpr int kBR = 64;             // reduction elements per staged tile

struct ProductArgs {
    ProductDesc d;
    int64_t r_per_split;            // multiple of kBR
    int32_t splits;
    int32_t tiles;                  // output tiles of the launch's kind
    int32_t np, nq;                 // down and across, the wide tiles where a launch takes their quarters
    int64_t p0, q0;                 // the first tile's first row and column
    int32_t first_wide;             // -1, or the workgroups are the quarters of the wide tiles from this
                                    // one on
    int64_t ld_part;                // row length of a split's partial products
    float* part;                    // [splits, P, ld_part], or nullptr: epilogue in place
    int32_t sum_of;                 // weight gradient with a bias: 1, 2: sums of operand a, b
    int32_t sum_rows;               // rows of partial sums
    int64_t sum_n, ld_sums;         // the bias's length, and a row of partial sums'
    float* sums;                    // [sum_rows, ld_sums]
    int64_t join_blocks;            // k_join: workgroups on the product, before those on the sums
};

// Eight elements (n of them valid, the rest 0) from any element-aligned address.
__device__ __forceinline__ v4u chunk_load(const uint16_t* p, int n) {
    if (n >= 8) return *reinterpret_cast<const v4u_any*>(p);
    v4u w = {0, 0, 0, 0};
#pragma unroll
    for (int k = 0; k < 8; ++k)
        if (k < n) w[k >> 1] |= (uint32_t)p[k] << (16 * (k & 1));
    return w;
}

// Chunk `id` of an operand's tile: what lies outside the operand becomes 0, so
// lengths, strides and alignment are arbitrary.
template <int ROWS, bool T>
__device__ __forceinline__ v4u tile_chunk(int id, const uint16_t* src, int64_t ld, int64_t o0, int64_t O,
                                          int64_t r0, int64_t r1) {
    int64_t row, col, n;
    bool in;
    if constexpr (T) {
        row = r0 + id / (ROWS / 8);
        col = o0 + 8 * (id % (ROWS / 8));
        in = row < r1;
        n = O - col;
    } else {
        row = o0 + id / (kBR / 8);
        col = r0 + 8 * (id % (kBR / 8));
        in = row < O;
        n = r1 - col;
    }
    return in && n > 0 ? chunk_load(src + row * ld + col, n < 8 ? (int)n : 8) : v4u{0, 0, 0, 0};
}
template <int ROWS, bool T>
__device__ __forceinline__ void put_chunk(uint16_t* lds, int id, v4u w) {
    int at;
    if constexpr (T) {
        const int r = id / (ROWS / 8), c = id % (ROWS / 8);
        at = r * ROWS + 8 * (c ^ perm_reduced<ROWS>(r));
    } else {
        const int o = id / (kBR / 8), c = id % (kBR / 8);
        at = o * kBR + 8 * (c ^ (o & 7));
    }
    *reinterpret_cast<v4u*>(lds + at) = w;
}

// Elements by .. 7 of eight to the front (what comes behind them does not matter).
__device__ __forceinline__ v4u chunk_shift(v4u w, int by) {
    if (by & 1) w = v4u{w[0] >> 16 | w[1] << 16, w[1] >> 16 | w[2] << 16, w[2] >> 16 | w[3] << 16, w[3] >> 16};
    if (by & 2) w = v4u{w[1], w[2], w[3], 0};
    if (by & 4) w = v4u{w[2], w[3], 0, 0};
    return w;
}

// A tile through registers into LDS: all of a thread's chunks loaded, then stored
// (Stage), or one at a time where registers are short (stage_tail). A whole tile's
// rows outside the operand read its last one instead, as they reach no output. Of
// reduced rows, the chunk that the operand's edge cuts is loaded from the row's last
// eight elements and shifted as it is stored: a load by elements on one side of a
// branch would make every load wait where the sides meet (1531 x 1001 x 2049 weight
// gradient 63 -> 40 us).
template <int ROWS, bool T, int THREADS>
struct Stage {
    static constexpr int kChunks = ROWS * kBR / 8 / THREADS;
    v4u w[kChunks];
    const uint16_t* from[kChunks];
    int by[T ? kChunks : 1];        // elements to shift
    int64_t step;
    bool edge, tiny;                // some chunk is cut; rows of fewer than eight elements
    __device__ __forceinline__ void init(const uint16_t* src, int64_t ld, int64_t o0, int64_t O, int64_t r0) {
        step = T ? kBR * ld : kBR;
        tiny = T && O < 8;
        edge = T && o0 + ROWS > O;
#pragma unroll
        for (int i = 0; i < kChunks; ++i) {
            const int id = threadIdx.x + i * THREADS;
            if constexpr (T) {
                const int64_t row = r0 + id / (ROWS / 8), col = o0 + 8 * (id % (ROWS / 8));
                const int64_t over = col + 8 - O;
                by[i] = over <= 0 || over > 7 || tiny ? 0 : (int)over;
                from[i] = src + row * ld + (tiny ? 0 : over > 0 ? O - 8 : col);
            } else {
                int64_t row = o0 + id / (kBR / 8);
                if (row >= O) row = O - 1;
                from[i] = src + row * ld + r0 + 8 * (id % (kBR / 8));
            }
        }
    }
    __device__ __forceinline__ void load(int64_t O) {
        if (T && tiny) {
#pragma unroll
            for (int i = 0; i < kChunks; ++i) w[i] = chunk_load(from[i], (int)O);
        } else {
#pragma unroll
            for (int i = 0; i < kChunks; ++i) w[i] = chunk_load(from[i], 8);
        }
#pragma unroll
        for (int i = 0; i < kChunks; ++i) from[i] += step;
    }
    __device__ __forceinline__ void store(uint16_t* lds) {
        if constexpr (T)
            if (edge)
#pragma unroll
                for (int i = 0; i < kChunks; ++i) w[i] = chunk_shift(w[i], by[i]);
#pragma unroll
        for (int i = 0; i < kChunks; ++i) put_chunk<ROWS, T>(lds, threadIdx.x + i * THREADS, w[i]);
    }
};
template <int ROWS, bool T, int THREADS>
__device__ __forceinline__ void stage_tail(uint16_t* lds, const uint16_t* src, int64_t ld, int64_t o0, int64_t O,
                                           int64_t r0, int64_t r1) {
#pragma unroll 1
    for (int id = threadIdx.x % THREADS; id < ROWS * kBR / 8; id += THREADS)
        put_chunk<ROWS, T>(lds, id, tile_chunk<ROWS, T>(id, src, ld, o0, O, r0, r1));
}

template <int ROWS, bool T>
using Fragments = TileFragments<ROWS, T, kBR, v8bf>;

// The epilogue of eight consecutive columns q .. of row p; n of them exist. What it
// reads beside the sums is asked for in one part (EpilogueIn::load), used in another,
// so that a wave has several rows' loads under way.
struct EpilogueIn {
    v4u lo, hi;                     // the residual, old value (f32: both) or pre-activation

    __device__ __forceinline__ void load_bf(const uint16_t* p, int n) { lo = chunk_load(p, n); }
    __device__ __forceinline__ void load_f(const float* p, int n) {
        if (n >= 8) {
            lo = *reinterpret_cast<const v4u_any*>(p);
            hi = *reinterpret_cast<const v4u_any*>(p + 4);
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                lo[k] = k < n ? __float_as_uint(p[k]) : 0;
                hi[k] = 4 + k < n ? __float_as_uint(p[4 + k]) : 0;
            }
        }
    }
    template <int EPI>
    __device__ __forceinline__ void load(const ProductDesc& d, int64_t p, int64_t q, int n) {
        if constexpr (EPI == kEpiGradInput) {
            if (d.z_in) load_bf(d.z_in + p * d.ld_z + q, n);
        } else if (d.res) {
            if (d.out_f32) load_f(static_cast<const float*>(d.res) + p * d.ld_res + q, n);
            else load_bf(static_cast<const uint16_t*>(d.res) + p * d.ld_res + q, n);
        }
    }
    __device__ __forceinline__ void get_bf(float t[8]) const {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            t[2 * k] = bf_lo(lo[k]);
            t[2 * k + 1] = bf_hi(lo[k]);
        }
    }
    __device__ __forceinline__ void get_f(float t[8]) const {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            t[k] = __uint_as_float(lo[k]);
            t[4 + k] = __uint_as_float(hi[k]);
        }
    }
};

// Columns q .. of the bias, the same for every row.
__device__ __forceinline__ void epilogue_bias(const ProductDesc& d, int64_t q, int n, float b[8]) {
#pragma unroll
    for (int k = 0; k < 8; ++k) b[k] = 0.0f;
    if (d.bias && n > 0) load8_bf(b, d.bias + q, n);
}

template <int EPI>
__device__ __forceinline__ void epilogue8(const ProductDesc& d, uint64_t off, int64_t p, int64_t q, float v[8],
                                          const EpilogueIn& in, const float bias[8], int n) {
    float t[8];
    if constexpr (EPI == kEpiForward) {
        if (d.bias)
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] += bias[k];
        if (d.z_out) store8_bf(d.z_out + p * d.ld_z + q, v, n);
        if (d.act != ZERO_ACT_NONE)
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = act_of(d.act, v[k]);
        if (d.drop.thr) drop8(v, d.drop, off, (uint32_t)p, (uint32_t)(q >> 3));
    }
    if constexpr (EPI == kEpiGradInput) {
        if (d.z_in) {
            in.get_bf(t);
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] *= act_slope(d.act, t[k]);
        }
        if (d.drop.thr) drop8(v, d.drop, off, (uint32_t)p, (uint32_t)(q >> 3));
    } else if (d.res) {
        if (d.out_f32) in.get_f(t);
        else in.get_bf(t);
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] += t[k];
    }
    if (d.out_f32) store8_f(static_cast<float*>(d.out) + p * d.ld_out + q, v, n);
    else store8_bf(static_cast<uint16_t*>(d.out) + p * d.ld_out + q, v, n);
}

// N loads of 16 bytes a lane from the buffer's bytes `at` to LDS, lane l of the wave to
// byte 16 l behind `to` (the same in all lanes), each load STEP bytes further on. Written
// in assembly because the compiler, which sees in its own builtin a store to LDS of
// unknown extent, waits for it before the next LDS read of any tile. It has no output
// register; what reads the tile waits with loads_landed first. The descriptor may come
// from v_readfirstlane (or a spill's v_readlane) right before: a scalar register that a
// vector instruction wrote takes five wait states until a memory instruction may read
// it, which the compiler sees to for its own instructions but not inside assembly. The
// first load's move and four of s_nop are those five, the others follow in the same
// block; m0 itself needs one. (Against no wait of their own, products are 0 to 1.5%
// slower so, and 0.4 to 2.5% with five before each load.)
template <int N, int STEP>
__device__ __forceinline__ void lds_loads(v4i rsrc, const uint32_t* at, uint32_t to) {
    static_assert(N <= 3 || N % 4 == 0, "blocks of 1, 2, 3 or 4 loads");
    if constexpr (N == 1)
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 3\n\tbuffer_load_dwordx4 %2, %1, 0 offen lds"
                     :
                     : "s"(to), "s"(rsrc), "v"(at[0])
                     : "memory", "m0");
    else if constexpr (N == 2)
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 3\n\tbuffer_load_dwordx4 %3, %1, 0 offen lds\n\t"
                     "s_add_u32 m0, %0, %2\n\ts_nop 0\n\tbuffer_load_dwordx4 %4, %1, 0 offen lds"
                     :
                     : "s"(to), "s"(rsrc), "n"(STEP), "v"(at[0]), "v"(at[1])
                     : "memory", "m0", "scc");
    else if constexpr (N == 3)
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 3\n\tbuffer_load_dwordx4 %4, %1, 0 offen lds\n\t"
                     "s_add_u32 m0, %0, %2\n\ts_nop 0\n\tbuffer_load_dwordx4 %5, %1, 0 offen lds\n\t"
                     "s_add_u32 m0, %0, %3\n\ts_nop 0\n\tbuffer_load_dwordx4 %6, %1, 0 offen lds"
                     :
                     : "s"(to), "s"(rsrc), "n"(STEP), "n"(2 * STEP), "v"(at[0]), "v"(at[1]), "v"(at[2])
                     : "memory", "m0", "scc");
    else {
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 3\n\tbuffer_load_dwordx4 %5, %1, 0 offen lds\n\t"
                     "s_add_u32 m0, %0, %2\n\ts_nop 0\n\tbuffer_load_dwordx4 %6, %1, 0 offen lds\n\t"
                     "s_add_u32 m0, %0, %3\n\ts_nop 0\n\tbuffer_load_dwordx4 %7, %1, 0 offen lds\n\t"
                     "s_add_u32 m0, %0, %4\n\ts_nop 0\n\tbuffer_load_dwordx4 %8, %1, 0 offen lds"
                     :
                     : "s"(to), "s"(rsrc), "n"(STEP), "n"(2 * STEP), "n"(3 * STEP), "v"(at[0]), "v"(at[1]),
                       "v"(at[2]), "v"(at[3])
                     : "memory", "m0", "scc");
        if constexpr (N > 4) lds_loads<N - 4, STEP>(rsrc, at + 4, to + 4 * STEP);
    }
}

// One operand's tiles from memory straight into LDS: 16 bytes a lane, lane l of a
// wave to byte 16 l behind the wave's LDS address, so the chunk permutation is
// applied to the address that a lane reads. Rows and chunks outside the operand
// read its last ones instead: they only reach outputs that do not exist. Used
// where rows start on 16 bytes and a whole tile of the reduction is left.
template <int ROWS, bool T, int THREADS, int PARTS>
struct Direct {
    static constexpr int kLoads = ROWS * kBR / 8 / THREADS;
    uint32_t at[PARTS][kLoads];     // byte offsets from `base`, of PARTS runs of ROWS outer indices
    const char* base;
    int64_t step;
    __device__ __forceinline__ void init(const uint16_t* src, int64_t ld, int64_t o0, int64_t O, int64_t r0) {
#pragma unroll
        for (int h = 0; h < PARTS; ++h)
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                const int id = threadIdx.x % THREADS + i * THREADS;
                if constexpr (T) {
                    const int r = id / (ROWS / 8);
                    int64_t c = ROWS * h + 8 * ((id % (ROWS / 8)) ^ perm_reduced<ROWS>(r));
                    if (o0 + c >= O) c = (O - 1 - o0) & ~int64_t(7);
                    at[h][i] = (uint32_t)((r * ld + c) * 2);
                } else {
                    const int in = id / (kBR / 8), c = 8 * ((id % (kBR / 8)) ^ (in & 7));
                    int64_t o = ROWS * h + in;
                    if (o0 + o >= O) o = O - 1 - o0;
                    at[h][i] = (uint32_t)((o * ld + c) * 2);
                }
            }
        base = reinterpret_cast<const char*>(src + (T ? r0 * ld + o0 : o0 * ld + r0));
        step = (T ? kBR * ld : kBR) * 2;
    }
    // Part h of the tile at `from` (base, or steps away from it) to LDS byte address
    // `tile`; `wave` is the same in all lanes. `records`: kAllRecords, or 0 for no load.
    __device__ __forceinline__ void issue(int h, const char* from, uint32_t tile, int wave, int records) const {
        lds_loads<kLoads, 16 * THREADS>(descriptor(from, records), at[h], tile + 16 * 64 * wave);
    }
    // All parts, one behind the other.
    __device__ __forceinline__ void issue_all(const char* from, uint32_t tile, int wave, int records) const {
        static_assert(kLoads == 1 && 16 * THREADS == 2 * ROWS * kBR, "a part is one load");
        uint32_t each[PARTS];
#pragma unroll
        for (int h = 0; h < PARTS; ++h) each[h] = at[h][0];
        lds_loads<PARTS, 16 * THREADS>(descriptor(from, records), each, tile + 16 * 64 * wave);
    }
};

// The output tile of a workgroup. Workgroups go to the 8 XCDs in turn, each with an
// L2 of its own, so each XCD gets a run of consecutive tiles; runs walk down blocks
// of kTileRows rows of tiles, column by column, so that the 32 workgroups that an
// XCD runs at a time share few operand rows.
// (Llama-7B shaped products: 8 rows 5% faster than tiles in order, 4 or 16 rows 2%
// behind 8 on the deepest reductions.)
constexpr int kTileRows = 8;
// With a split reduction the tiles of one split are consecutive, since they share the
// split's rows of both operands (GPT-2 projection
// gradient, 7 splits of 36 tiles: 27.2 -> 24.1 us).
__device__ __forceinline__ int tile_in_turn(const ProductArgs& g, int* split) {
    const int all = g.tiles * g.splits, id = blockIdx.x;
    const int xcd = id & 7, slot = id >> 3, each = all >> 3, more = all & 7;
    const int t = xcd * each + (xcd < more ? xcd : more) + slot;
    if (g.splits == 1) {
        *split = 0;
        return t;
    }
    const int y = t / g.tiles;
    *split = __builtin_amdgcn_readfirstlane(y);
    return __builtin_amdgcn_readfirstlane(t - y * g.tiles);
}
__device__ __forceinline__ void tile_place(int t, int np, int nq, int* tp, int* tq) {
    const int block = t / (kTileRows * nq), in = t - block * kTileRows * nq;
    const int rows = np - block * kTileRows < kTileRows ? np - block * kTileRows : kTileRows;
    const int col = in / rows;
    // the same in all lanes, which the divisions hide from the compiler
    *tq = __builtin_amdgcn_readfirstlane(col);
    *tp = __builtin_amdgcn_readfirstlane(block * kTileRows + in - col * rows);
}

// Whole tiles of kBR in this split, in 32 bits: a 64-bit comparison would put what
// depends on it into vector registers, the loads' descriptors among them.
__device__ __forceinline__ int whole_steps(const ProductArgs& g, int split) {
    const int per = (int)(g.r_per_split / kBR), left = (int)(g.d.R / kBR) - split * per;
    const int n = left < per ? left : per;
    return n > 0 ? n : 0;
}

// The bias gradient rides on the weight's: each output tile has dz in one of its
// operands, so the tiles that share a run of dz's columns take turns at its
// reduction tiles and multiply the operand's blocks by ones as well, which sums
// their columns: 4 more matrix instructions for 64, once in as many tiles as share.
struct SumTurn {
    int32_t turn, others;           // this workgroup's reduction tiles: k % others == turn
    bool on;
    int32_t left;                   // tiles until its next one
    __device__ __forceinline__ SumTurn(int t, int n, bool o) : turn(t), others(n), on(o), left(t) {}
    // Whether the next tile, in order, is this workgroup's.
    __device__ __forceinline__ bool next() {
        const bool now = left == 0;
        left = now ? others - 1 : left - 1;
        return on && now;
    }
};
__device__ __forceinline__ v8bf ones8() {
    const __bf16 one = (__bf16)1.0f;
    return v8bf{one, one, one, one, one, one, one, one};
}
// Lane l of the product's block holds the sum of column l & 15, in all its rows.
__device__ __forceinline__ void put_sums(const ProductArgs& g, int split, const SumTurn& t, int64_t col, v4f v) {
    const int lane = threadIdx.x & 63;
    if (lane < 16 && col + lane < g.sum_n)
        g.sums[((int64_t)split * t.others + t.turn) * g.ld_sums + col + lane] = v[0];
}

// The epilogue of a workgroup's tile, through LDS: kRun rows of a wave's blocks at a
// time, so that a lane gets eight consecutive columns and stores 16 bytes or more.
// Blocks are computed as (q, p), so a lane holds four consecutive columns of one
// output row, one 16-byte unit. Each wave has its own part of LDS; unit u of row o
// lies at u ^ (o & 15), or u ^ (o & 7) where a row has 8. row_of(i) and col_of(j): first
// row and column of the wave's blocks (i, j) in the output; the rows of a run are
// consecutive.
template <int EPI, int LDS_BYTES, int WAVES, int FP, int FQ, typename Row, typename Col>
__device__ __forceinline__ void finish(const ProductArgs& g, int split, const v4f (&acc)[FP][FQ], uint16_t* lds, int wave,
                                       Row row_of, Col col_of) {
    static_assert(FQ >= 2 && FQ <= 4, "8 or 16 units a row; of 3 blocks with 4 left empty");
    constexpr int kBlocks = FQ == 2 ? 2 : 4;
    constexpr int kCols = 16 * kBlocks, kMask = 4 * kBlocks - 1, kLanes = 2 * kBlocks, kStep = 64 / kLanes;
    constexpr int kFit = LDS_BYTES / (WAVES * 16 * kCols * 4), kRun = kFit >= 4 ? 4 : kFit;
    static_assert(kRun >= 1 && FP % kRun == 0, "the runs cover a wave's rows");
    static_assert(16 * kRun % (4 * kStep) == 0, "whole groups of four rows a lane");
    const ProductDesc& d = g.d;
    const int lane = threadIdx.x & 63;
    const uint64_t off = d.drop.thr ? drop_offset(d.drop) : 0;
    float* const mine = reinterpret_cast<float*>(lds) + wave * kRun * 16 * kCols;
    // A split's sums go four columns to a lane, whole lines to a store instruction
    // (GPT-2 projection gradient 23.7 -> 22.9 us; f32 outputs, which read and compute as
    // well, are 5% faster with eight).
    const int c = g.part ? lane % (2 * kLanes) : lane % kLanes;
    const int64_t q = g.part ? col_of(c >> 2) + 4 * (c & 3) : col_of(c >> 1) + 8 * (c & 1);
    const bool some = (g.part ? c >> 2 : c >> 1) < FQ;
    const int n = !some ? 0 : d.Q - q >= 8 ? 8 : d.Q - q > 0 ? (int)(d.Q - q) : 0;
    float bias[8];
    epilogue_bias(d, q, g.part ? 0 : n, bias);
#pragma unroll
    for (int i0 = 0; i0 < FP; i0 += kRun) {
        EpilogueIn in[4];
        const auto load = [&](int o0) {
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int64_t p = row_of(i0) + o0 + kStep * u;
                if (p < d.P && n > 0) in[u].template load<EPI>(d, p, q, n);
            }
        };
        // four rows of each lane at a time, the first four before the sums go to LDS (GPT-2
        // projection with residual 17.4 -> 16.6 us; all eight at once spill the wide kernel)
        if (!g.part) load(lane / kLanes);
#pragma unroll
        for (int i = 0; i < kRun; ++i)
#pragma unroll
            for (int j = 0; j < FQ; ++j) {
                const int o = 16 * i + (lane & 15), u = 4 * j + (lane >> 4);
                *reinterpret_cast<v4f*>(mine + o * kCols + 4 * (u ^ (o & kMask))) = acc[i0 + i][j];
            }
        if (g.part) {
            // rows of ld_part, a multiple of 8, so a lane's columns all have a place
#pragma unroll 4
            for (int o = lane / (2 * kLanes); o < 16 * kRun; o += kStep / 2) {
                const int64_t p = row_of(i0) + o;
                const v4f v = *reinterpret_cast<const v4f*>(mine + o * kCols + 4 * (c ^ (o & kMask)));
                if (some && p < d.P && q < g.ld_part)
                    *reinterpret_cast<v4f*>(g.part + ((int64_t)split * d.P + p) * g.ld_part + q) = v;
            }
            continue;
        }
#pragma unroll 1
        for (int o0 = lane / kLanes; o0 < 16 * kRun; o0 += 4 * kStep) {
            if (o0 >= 4 * kStep) load(o0);
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int o = o0 + kStep * u;
                const int64_t p = row_of(i0) + o;
                const v4f lo = *reinterpret_cast<const v4f*>(mine + o * kCols + 4 * ((2 * c) ^ (o & kMask)));
                const v4f hi = *reinterpret_cast<const v4f*>(mine + o * kCols + 4 * ((2 * c + 1) ^ (o & kMask)));
                float v[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
                if (p >= d.P || n <= 0) continue;
                epilogue8<EPI>(d, off, p, q, v, in[u], bias, n);
            }
        }
    }
}

// The tile of 128 rows and COLS columns of a workgroup: of all of them, or (128 columns)
// of the quarters of wide tiles.
template <int COLS>
__device__ __forceinline__ SumTurn small_place(const ProductArgs& g, int* split, int64_t* p0, int64_t* q0) {
    const int id = tile_in_turn(g, split), np = g.np, nq = g.nq;
    int tp, tq;
    if (g.first_wide < 0) {
        tile_place(id, np, nq, &tp, &tq);
        *p0 = g.p0 + (int64_t)tp * 128;
        *q0 = g.q0 + (int64_t)tq * COLS;
        return g.sum_of == 1 ? SumTurn{tq, nq, true} : SumTurn{tp, np, g.sum_of == 2};
    }
    tile_place(g.first_wide + (id >> 2), np, nq, &tp, &tq);
    *p0 = (int64_t)tp * 256 + 128 * ((id >> 1) & 1);
    *q0 = (int64_t)tq * 256 + 128 * (id & 1);
    return g.sum_of == 1 ? SumTurn{tq, nq, (id & 1) == 0} : SumTurn{tp, np, g.sum_of == 2 && (id & 2) == 0};
}

// 128 x 128 outputs by four waves, 64 x 64 each (4 x 4 blocks), for outputs of more tiles
// than compute units but too few for the wide kernel, and for operands at any address:
// tiles of 64 reduction elements, two in LDS, the next one loading while one is
// multiplied. Two workgroups of 64 KB fit a compute unit and fill each other's waits. An
// operand goes straight to LDS where its rows allow it (DA, DB), through registers
// elsewhere: gradient by input of 1023 x 768 through 50,257 outputs, whose dz has odd
// rows, 101 us with its operands in the MALL, 780 TFLOP/s (113 with both operands through
// registers; 76 through 50,256 outputs, with neither, by the wide kernel). From memory it
// takes 131, aligned loads of the same rows 127: not the addresses bound it but the
// traffic of small tiles, each operand read from L2 twice as often as the wide kernel
// does, and the wait for the direct operand's loads, which takes in the register loads
// of the tile after it.
template <bool TA, bool TB, int EPI, bool DA, bool DB, bool SUM>
__global__ void __launch_bounds__(256, 2) k_product(const ProductArgs g) {
    constexpr int T = 256, B = 128, FP = 4, FQ = 4, kTile = B * kBR;
    __shared__ __attribute__((aligned(16))) uint16_t lds[2 * 2 * kTile];
    const ProductDesc& d = g.d;
    int split;
    int64_t p0, q0;
    SumTurn turn = small_place<B>(g, &split, &p0, &q0);
    if (g.first_wide >= 0 && (p0 >= d.P || q0 >= d.Q)) return;
    const int64_t r0 = (int64_t)split * g.r_per_split;
    const int64_t r1 = r0 + g.r_per_split < d.R ? r0 + g.r_per_split : d.R;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wp = (wave >> 1) * 64, wq = (wave & 1) * 64;

    v4f acc[FP][FQ];
#pragma unroll
    for (int i = 0; i < FP; ++i)
#pragma unroll
        for (int j = 0; j < FQ; ++j) acc[i][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    const Fragments<B, TA> ga(wp);
    const Fragments<B, TB> gb(wq);
    const uint32_t base = lds_address(lds);
    v4f sum[4] = {acc[0][0], acc[0][0], acc[0][0], acc[0][0]};
    const auto multiply = [&](uint32_t tile) {
        const bool now = SUM && turn.next();
#pragma unroll
        for (int s = 0; s < kBR / 32; ++s) {
            v8bf fa[FP], fb[FQ];
#pragma unroll
            for (int i = 0; i < FP; ++i) fa[i] = ga.get(tile, i, s);
#pragma unroll
            for (int j = 0; j < FQ; ++j) fb[j] = gb.get(tile + 2 * kTile, j, s);
#pragma unroll
            for (int i = 0; i < FP; ++i)
#pragma unroll
                for (int j = 0; j < FQ; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fb[j], fa[i], acc[i][j], 0, 0, 0);
            if constexpr (SUM)
                if (now) {
                    if (g.sum_of == 1) {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            sum[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ones8(), fa[i], sum[i], 0, 0, 0);
                    } else {
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            sum[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ones8(), fb[j], sum[j], 0, 0, 0);
                    }
                }
        }
    };

    if constexpr (DA && DB) {
        const int full = whole_steps(g, split);
        Direct<B, TA, T, 1> da;
        Direct<B, TB, T, 1> db;
        if (full > 0) {
            da.init(d.a, d.lda, p0, d.P, r0);
            db.init(d.b, d.ldb, q0, d.Q, r0);
            da.issue(0, da.base, base, wave, kAllRecords);
            db.issue(0, db.base, base + 2 * kTile, wave, kAllRecords);
        }
        for (int k = 0; k < full; ++k) {
            loads_landed<0>();
            meet_waves();
            const uint32_t tile = base + 4 * kTile * (k & 1), next = base + 4 * kTile * ((k + 1) & 1);
            if (k + 1 < full) {
                da.issue(0, da.base += da.step, next, wave, kAllRecords);
                db.issue(0, db.base += db.step, next + 2 * kTile, wave, kAllRecords);
            }
            multiply(tile);
        }
        if (r0 + (int64_t)full * kBR < r1) {
            // what is left of the reduction, with its end masked
            const int64_t r = r0 + (int64_t)full * kBR;
            uint16_t* const to = lds + 2 * kTile * (full & 1);
            stage_tail<B, TA, T>(to, d.a, d.lda, p0, d.P, r, r1);
            stage_tail<B, TB, T>(to + kTile, d.b, d.ldb, q0, d.Q, r, r1);
            meet_waves();
            multiply(base + 4 * kTile * (full & 1));
        }
    } else {
        // the next tile waits in registers while one is multiplied, or, of an operand
        // that can, is on its way to LDS
        const int full = whole_steps(g, split);
        std::conditional_t<DA, Direct<B, TA, T, 1>, Stage<B, TA, T>> sa;
        std::conditional_t<DB, Direct<B, TB, T, 1>, Stage<B, TB, T>> sb;
        const auto load = [&]() {
            if constexpr (!DA) sa.load(d.P);
            if constexpr (!DB) sb.load(d.Q);
        };
        const auto store = [&](int k) {
            uint16_t* const to = lds + 2 * kTile * (k & 1);
            if constexpr (!DA) sa.store(to);
            if constexpr (!DB) sb.store(to + kTile);
        };
        const auto issue = [&](int k) {
            const uint32_t to = base + 4 * kTile * (k & 1);
            if constexpr (DA) {
                sa.issue(0, sa.base, to, wave, kAllRecords);
                sa.base += sa.step;
            }
            if constexpr (DB) {
                sb.issue(0, sb.base, to + 2 * kTile, wave, kAllRecords);
                sb.base += sb.step;
            }
        };
        if (full > 0) {
            sa.init(d.a, d.lda, p0, d.P, r0);
            sb.init(d.b, d.ldb, q0, d.Q, r0);
            issue(0);
            load();
            store(0);
            if (full > 1) load();
        }
        for (int k = 0; k < full; ++k) {
            if constexpr (DA || DB) loads_landed<0>();
            meet_waves();
            if (k + 1 < full) {
                issue(k + 1);
                store(k + 1);
                if (k + 2 < full) load();
            }
            multiply(base + 4 * kTile * (k & 1));
        }
        if (r0 + (int64_t)full * kBR < r1) {
            const int64_t r = r0 + (int64_t)full * kBR;
            uint16_t* const to = lds + 2 * kTile * (full & 1);
            stage_tail<B, TA, T>(to, d.a, d.lda, p0, d.P, r, r1);
            stage_tail<B, TB, T>(to + kTile, d.b, d.ldb, q0, d.Q, r, r1);
            meet_waves();
            multiply(base + 4 * kTile * (full & 1));
        }
    }
    meet_waves();
    if constexpr (SUM)
        if (turn.on && (g.sum_of == 1 ? wq : wp) == 0)
#pragma unroll
            for (int i = 0; i < 4; ++i) put_sums(g, split, turn, (g.sum_of == 1 ? p0 + wp : q0 + wq) + 16 * i, sum[i]);
    finish<EPI, sizeof(lds), 4>(g, split, acc, lds, wave, [&](int i) { return p0 + wp + 16 * i; },
                                [&](int j) { return q0 + wq + 16 * j; });
}

// 128 x 64 FQ outputs (FQ 2 or 3) by eight waves, one workgroup to a compute unit: the
// wide kernel's turns with a whole tile of 64 reduction elements to a turn, in a ring of
// four. A wave has 64 rows and 16 columns of each run of 64. It reads the tile's operands
// and asks for the tile three ahead; then it multiplies; waves 4-7 are one barrier behind
// waves 0-3. A tile's place is asked for again one turn after it was read, two barriers or
// more after its last reads began; each turn ends when the next turn's tile is here, one
// barrier before anyone reads it. A turn takes 0.5 us, and what is around the turns 10: for
// the GPT-2 projection (8192 x 768 x 768 with dropout and residual, 256 tiles of 192
// columns) 18.2 to 20.0 us from memory, by the card, about 510 TFLOP/s, 5 of them its
// epilogue's memory and draws; gradient by input through the 2304 outputs of qkv 32 us,
// 905 TFLOP/s (28.9 with its operands in the MALL).
template <bool TA, bool TB, int EPI, bool SUM, int FQ>
__global__ void __launch_bounds__(512) k_product_mid(const ProductArgs g) {
    constexpr int T = 512, B = 128, FP = 4, kA = B * kBR, kB = 64 * kBR, kSlot = kA + FQ * kB, kSlots = 4;
    static_assert(!SUM || FQ == 2, "two waves share a block of b, and sum one each");
    __shared__ __attribute__((aligned(16))) uint16_t lds[kSlots * kSlot];
    const ProductDesc& d = g.d;
    int split;
    int64_t p0, q0;
    SumTurn turn = small_place<64 * FQ>(g, &split, &p0, &q0);
    if (g.first_wide >= 0 && (p0 >= d.P || q0 >= d.Q)) return;
    const int64_t r0 = (int64_t)split * g.r_per_split;
    const int64_t r1 = r0 + g.r_per_split < d.R ? r0 + g.r_per_split : d.R;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wp = (wave >> 2) * 64, wq = (wave & 3) * 16;

    v4f acc[FP][FQ], sum = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < FP; ++i)
#pragma unroll
        for (int j = 0; j < FQ; ++j) acc[i][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    const Fragments<B, TA> ga(wp);
    const Fragments<64, TB> gb(wq);
    const uint32_t base = lds_address(lds);
    v8bf fa[2][FP], fb[2][FQ];
    const auto read = [&](uint32_t tile) {
#pragma unroll
        for (int s = 0; s < 2; ++s) {
#pragma unroll
            for (int j = 0; j < FQ; ++j) fb[s][j] = gb.get(tile + 2 * (kA + j * kB), 0, s);
#pragma unroll
            for (int i = 0; i < FP; ++i) fa[s][i] = ga.get(tile, i, s);
        }
    };
    const auto multiply = [&]() {
        const bool now = SUM && turn.next();
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_setprio(1);
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int i = 0; i < FP; ++i)
#pragma unroll
                for (int j = 0; j < FQ; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fb[s][j], fa[s][i], acc[i][j], 0, 0, 0);
        __builtin_amdgcn_s_setprio(0);
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (SUM)
            if (now) {
                // waves with the same blocks of dz's operand sum one each
#pragma unroll
                for (int s = 0; s < 2; ++s) {
#pragma unroll
                    for (int i = 0; i < FP; ++i)
                        if (g.sum_of == 1 && (wave & 3) == i)
                            sum = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ones8(), fa[s][i], sum, 0, 0, 0);
#pragma unroll
                    for (int j = 0; j < FQ; ++j)
                        if (g.sum_of == 2 && (wave >> 2) == j)
                            sum = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ones8(), fb[s][j], sum, 0, 0, 0);
                }
            }
    };

    const int n = whole_steps(g, split);
    if (n > 0) {
        Direct<B, TA, T, 1> da;
        Direct<64, TB, T, FQ> db;
        constexpr int kLoads = Direct<B, TA, T, 1>::kLoads + FQ * Direct<64, TB, T, FQ>::kLoads;
        da.init(d.a, d.lda, p0, d.P, r0);
        db.init(d.b, d.ldb, q0, d.Q, r0);
        // loads of tiles behind the last are stopped by their buffer's range
        const auto load = [&](int k) {
            const int records = k < n ? kAllRecords : 0;
            const uint32_t to = base + 2 * kSlot * (k % kSlots);
            da.issue(0, da.base, to, wave, records);
            db.issue_all(db.base, to + 2 * kA, wave, records);
            da.base += da.step;
            db.base += db.step;
        };
#pragma unroll
        for (int k = 0; k < kSlots - 1; ++k) load(k);
        loads_landed<(kSlots - 2) * kLoads>();
        meet_waves();
        if (wave >= 4) meet_waves();
#pragma unroll 1
        for (int k = 0; k < n; ++k) {
            read(base + 2 * kSlot * (k % kSlots));
            load(k + kSlots - 1);
            loads_landed<(kSlots - 2) * kLoads>();
            meet_waves();
            multiply();
            meet_waves();
        }
        if (wave < 4) meet_waves();
        loads_landed<0>();
        meet_waves();
    }
    if (r0 + (int64_t)n * kBR < r1) {
        // what is left of the reduction, with its end masked
        const int64_t r = r0 + (int64_t)n * kBR;
        stage_tail<B, TA, T>(lds, d.a, d.lda, p0, d.P, r, r1);
#pragma unroll
        for (int j = 0; j < FQ; ++j) stage_tail<64, TB, T>(lds + kA + j * kB, d.b, d.ldb, q0 + 64 * j, d.Q, r, r1);
        meet_waves();
        read(base);
        multiply();
        meet_waves();
    }
    if constexpr (SUM)
        if (turn.on)
            put_sums(g, split, turn, g.sum_of == 1 ? p0 + wp + 16 * (wave & 3) : q0 + wq + 64 * (wave >> 2), sum);
    finish<EPI, sizeof(lds), 8>(g, split, acc, lds, wave, [&](int i) { return p0 + wp + 16 * i; },
                                [&](int j) { return q0 + wq + 64 * j; });
}

// 256 x 256 outputs by eight waves, one workgroup to a compute unit. With the 128 x 192
// tiles of its rest, 8192 x 4096 x 11008 (SiLU, pre-activation kept) takes 602 to 634 us
// from memory, by the card it runs on, 1.17-1.23 PFLOP/s; the down projection, two whole
// rounds, takes 526-546, 1.35-1.41 PFLOP/s, where a library's bare product takes 448-476.
// The matrix cores are busy 57-71% of the time at 1.9-2.0 GHz, without LDS bank conflicts;
// as that library has them busy 88% at 1.7 GHz, it is not power that holds the loop.
// Operand tiles of 64 reduction elements lie in LDS as halves of 128 outer indices, two tiles of four
// halves. A wave's outputs are 64 x 32 of each quarter (half of A, half of B), so a
// tile is four turns of 16 matrix instructions, and a turn has two parts that
// barriers divide: the wave reads what its quarter needs and no turn before it read,
// and asks for one half tile of the tiles to come; then it multiplies. Waves 4-7 are
// one barrier behind waves 0-3, which share their SIMDs, so that one wave of each
// pair multiplies while the other reads.
//
//   turn      reads            asks for           multiplies
//   4k        A0(k), B0(k)     A1(k + 1)          A0 B0
//   4k + 1    B1(k)            A0(k + 2)          A0 B1
//   4k + 2    A1(k)            B0(k + 2)          A1 B1
//   4k + 3    -                B1(k + 2)          A1 B0
//
// A half is read in one turn only, by all waves within the two barrier intervals that
// begin with that turn of waves 0-3, and asked for again one turn later or more: after
// them. What turn f reads was asked for in turn f - 6 or before, or in the prologue;
// turn f - 1 waits until at most the five latest turns' loads are under way, and its
// barrier comes before anyone's turn f. So a load has five turns to land.
template <bool TA, bool TB, int EPI, bool SUM>
__global__ void __launch_bounds__(512) k_product_wide(const ProductArgs g) {
    constexpr int T = 512, B = 256, H = 128, kHalf = H * kBR;
    __shared__ __attribute__((aligned(16))) uint16_t lds[2 * 4 * kHalf];
    const ProductDesc& d = g.d;
    int split, tp, tq;
    tile_place(tile_in_turn(g, &split), g.np, g.nq, &tp, &tq);
    SumTurn turn = g.sum_of == 1 ? SumTurn{tq, g.nq, true} : SumTurn{tp, g.np, g.sum_of == 2};
    const int64_t p0 = (int64_t)tp * B, q0 = (int64_t)tq * B;
    const int64_t r0 = (int64_t)split * g.r_per_split;
    const int64_t r1 = r0 + g.r_per_split < d.R ? r0 + g.r_per_split : d.R;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wp = (wave >> 2) * 64, wq = (wave & 3) * 32;

    // blocks (4 a + i, 2 b + j): block (i, j) of the quarter of halves a and b
    v4f acc[8][4];
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    const Fragments<H, TA> ga(wp);
    const Fragments<H, TB> gb(wq);
    v8bf fa[2][4], fb[2][2][2];     // [step][block], [half][step][block]
    // byte addresses of tile k's halves: A0, A1, B0, B1
    const uint32_t base = lds_address(lds);
    const auto half = [&](int k, int h) { return base + 2 * kHalf * (4 * (k & 1) + h); };
    const auto read_a = [&](uint32_t from) {
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int i = 0; i < 4; ++i) fa[s][i] = ga.get(from, i, s);
    };
    const auto read_b = [&](int h, uint32_t from) {
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int j = 0; j < 2; ++j) fb[h][s][j] = gb.get(from, j, s);
    };
    const auto multiply = [&](int a, int b) {
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_setprio(1);
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    acc[4 * a + i][2 * b + j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                        fb[b][s][j], fa[s][i], acc[4 * a + i][2 * b + j], 0, 0, 0);
        __builtin_amdgcn_s_setprio(0);
        __builtin_amdgcn_sched_barrier(0);
    };

    // Sums of dz's columns: where dz is operand a, the four waves of a row of waves
    // have the same blocks of a half, and each sums one; where it is b, the two waves
    // of a column of waves.
    v4f sum[2] = {acc[0][0], acc[0][0]};
    const auto sum_a = [&](int h) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if ((wave & 3) == i)
#pragma unroll
                for (int s = 0; s < 2; ++s)
                    sum[h] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ones8(), fa[s][i], sum[h], 0, 0, 0);
    };
    const auto sum_b = [&](int h) {
#pragma unroll
        for (int j = 0; j < 2; ++j)
            if ((wave >> 2) == j)
#pragma unroll
                for (int s = 0; s < 2; ++s)
                    sum[h] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ones8(), fb[h][s][j], sum[h], 0, 0, 0);
    };
    const auto sum_turn = [&](bool now, int turn_of_tile) {
        if constexpr (SUM)
            if (now) {
                if (g.sum_of == 1 && turn_of_tile != 1) sum_a(turn_of_tile / 2);
                if (g.sum_of == 2 && turn_of_tile != 2) sum_b(turn_of_tile);
            }
    };

    const int n = whole_steps(g, split);
    if (n > 0) {
        Direct<H, TA, T, 2> da;
        Direct<H, TB, T, 2> db;
        constexpr int kLoads = Direct<H, TA, T, 2>::kLoads;
        da.init(d.a, d.lda, p0, d.P, r0);
        db.init(d.b, d.ldb, q0, d.Q, r0);
        // loads of tiles behind the last are stopped by their buffer's range
        const auto there = [&](int k) { return k < n ? kAllRecords : 0; };
        da.issue(0, da.base, half(0, 0), wave, kAllRecords);
        db.issue(0, db.base, half(0, 2), wave, kAllRecords);
        db.issue(1, db.base, half(0, 3), wave, kAllRecords);
        da.issue(1, da.base, half(0, 1), wave, kAllRecords);
        da.issue(0, da.base + da.step, half(1, 0), wave, there(1));
        db.issue(0, db.base + db.step, half(1, 2), wave, there(1));
        db.issue(1, db.base + db.step, half(1, 3), wave, there(1));
        da.base += 2 * da.step;         // of tile k + 2
        db.base += 2 * db.step;
        loads_landed<5 * kLoads>();
        meet_waves();
        if (wave >= 4) meet_waves();
#pragma unroll 1
        for (int k = 0; k < n; ++k) {
            const int one = there(k + 1), two = there(k + 2);
            const bool now = SUM && turn.next();
            read_b(0, half(k, 2));
            read_a(half(k, 0));
            da.issue(1, da.base - da.step, half(k + 1, 1), wave, one);
            loads_landed<5 * kLoads>();
            meet_waves();
            multiply(0, 0);
            sum_turn(now, 0);
            meet_waves();
            read_b(1, half(k, 3));
            da.issue(0, da.base, half(k, 0), wave, two);
            loads_landed<5 * kLoads>();
            meet_waves();
            multiply(0, 1);
            sum_turn(now, 1);
            meet_waves();
            read_a(half(k, 1));
            db.issue(0, db.base, half(k, 2), wave, two);
            loads_landed<5 * kLoads>();
            meet_waves();
            multiply(1, 1);
            sum_turn(now, 2);
            meet_waves();
            db.issue(1, db.base, half(k, 3), wave, two);
            da.base += da.step;
            db.base += db.step;
            loads_landed<5 * kLoads>();
            meet_waves();
            multiply(1, 0);
            meet_waves();
        }
        if (wave < 4) meet_waves();
        loads_landed<0>();
        meet_waves();
    }
    if (r0 + (int64_t)n * kBR < r1) {
        // what is left of the reduction, with its end masked
        const int64_t r = r0 + (int64_t)n * kBR;
        stage_tail<H, TA, T>(lds, d.a, d.lda, p0, d.P, r, r1);
        stage_tail<H, TA, T>(lds + kHalf, d.a, d.lda, p0 + H, d.P, r, r1);
        stage_tail<H, TB, T>(lds + 2 * kHalf, d.b, d.ldb, q0, d.Q, r, r1);
        stage_tail<H, TB, T>(lds + 3 * kHalf, d.b, d.ldb, q0 + H, d.Q, r, r1);
        meet_waves();
        const bool now = SUM && turn.next();
        read_b(0, half(0, 2));
        read_b(1, half(0, 3));
        read_a(half(0, 0));
        multiply(0, 0);
        sum_turn(now, 0);
        multiply(0, 1);
        sum_turn(now, 1);
        read_a(half(0, 1));
        multiply(1, 1);
        sum_turn(now, 2);
        multiply(1, 0);
        meet_waves();
    }
    if constexpr (SUM)
        if (turn.on)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                put_sums(g, split, turn, (g.sum_of == 1 ? p0 + wp + 16 * (wave & 3) : q0 + wq + 16 * (wave >> 2)) + H * h,
                         sum[h]);
    finish<EPI, sizeof(lds), 8>(g, split, acc, lds, wave, [&](int i) { return p0 + H * (i >> 2) + wp + 16 * (i & 3); },
                                [&](int j) { return q0 + H * (j >> 1) + wq + 16 * (j & 1); });
}

// Products of at most 16 rows, bound by reading b once: a workgroup takes 16 columns
// (b's outer index in rows; 32 were slower, 21.9 against 17.4 us on one row of a
// Llama-7B shaped layer, with half the workgroups in flight) or 64 (reduced rows), its eight waves each an eighth of
// the reduction, and their sums are joined in LDS, so that one launch streams b with
// everything in flight and nothing goes through memory again. Waves do not wait for
// each other before that. Operand a is read straight into the matrix instruction's
// layout by every wave, and b too, where r is contiguous; reduced rows of b, and a
// with them, go through the wave's own part of LDS, two tiles of 64 in turn.
template <bool TB, int EPI>
__global__ void __launch_bounds__(512) k_product_few(const ProductArgs g) {
    constexpr int kWaves = 8, FQ = TB ? 4 : 1, kCols = 16 * FQ, kTile = (64 + 16) * kBR;
    __shared__ __attribute__((aligned(16))) uint16_t lds[TB ? kWaves * 2 * kTile : kWaves * 16 * kCols * 2];
    const ProductDesc& d = g.d;
    const int lane = threadIdx.x & 63, i = lane & 15, gr = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t q0 = (int64_t)blockIdx.x * kCols;
    // this wave's tiles of 64 reduction elements, the last of all perhaps partial
    const int tiles = (int)((d.R + kBR - 1) / kBR), whole = (int)(d.R / kBR);
    const int t0 = (int)((int64_t)tiles * wave / kWaves), t1 = (int)((int64_t)tiles * (wave + 1) / kWaves);
    const int tw = t1 < whole ? t1 : whole;
    const uint16_t* const arow = d.a + (i < d.P ? i : d.P - 1) * d.lda + 8 * gr;
    v4f acc[FQ];
#pragma unroll
    for (int j = 0; j < FQ; ++j) acc[j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    const auto mul = [&](v8bf b, v4u a, v4f c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(b, __builtin_bit_cast(v8bf, a), c, 0, 0, 0);
    };
    const auto left = [&](int64_t r) { return (int)(d.R - r < 0 ? 0 : d.R - r < 8 ? d.R - r : 8); };

    if constexpr (!TB) {
        const int64_t q = q0 + i;
        const uint16_t* const brow = d.b + (q < d.Q ? q : d.Q - 1) * d.ldb + 8 * gr;
        int t = t0;
        for (; t + 3 < tw; t += 4) {
            v4u a[8], b[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) b[k] = chunk_load(brow + (int64_t)t * kBR + 32 * k, 8);
#pragma unroll
            for (int k = 0; k < 8; ++k) a[k] = chunk_load(arow + (int64_t)t * kBR + 32 * k, 8);
#pragma unroll
            for (int k = 0; k < 8; ++k) acc[0] = mul(__builtin_bit_cast(v8bf, b[k]), a[k], acc[0]);
        }
        for (; t < t1; ++t) {
            const int64_t r = (int64_t)t * kBR;
            v4u a[2], b[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int n = left(r + 32 * k + 8 * gr);
                b[k] = n > 0 ? chunk_load(brow + r + 32 * k, n) : v4u{0, 0, 0, 0};
                a[k] = n > 0 ? chunk_load(arow + r + 32 * k, n) : v4u{0, 0, 0, 0};
            }
#pragma unroll
            for (int k = 0; k < 2; ++k) acc[0] = mul(__builtin_bit_cast(v8bf, b[k]), a[k], acc[0]);
        }
    } else {
        uint16_t* const mine = lds + wave * 2 * kTile;
        const uint32_t base = lds_address(mine);
        const Fragments<64, true> gb(0);
        const Fragments<16, false> ga(0);
        Direct<64, true, 64, 1> db;
        Direct<16, false, 64, 1> da;
        constexpr int kLoads = Direct<64, true, 64, 1>::kLoads + Direct<16, false, 64, 1>::kLoads;
        const auto load = [&](uint32_t tile) {
            db.issue(0, db.base, tile, 0, kAllRecords);
            da.issue(0, da.base, tile + 2 * 64 * kBR, 0, kAllRecords);
            db.base += db.step;
            da.base += da.step;
        };
        const auto multiply = [&](uint32_t tile) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const v4u a = __builtin_bit_cast(v4u, ga.get(tile + 2 * 64 * kBR, 0, k));
#pragma unroll
                for (int j = 0; j < FQ; ++j) acc[j] = mul(gb.get(tile, j, k), a, acc[j]);
            }
            // read, before the next turn's loads write here
            asm volatile("s_waitcnt lgkmcnt(0)" : : : "memory");
        };
        if (t0 < tw) {
            db.init(d.b, d.ldb, q0, d.Q, (int64_t)t0 * kBR);
            da.init(d.a, d.lda, 0, d.P, (int64_t)t0 * kBR);
            load(base);
        }
        for (int t = t0; t < tw; ++t) {
            if (t + 1 < tw) {
                load(base + 2 * kTile * ((t + 1 - t0) & 1));
                loads_landed<kLoads>();
            } else {
                loads_landed<0>();
            }
            multiply(base + 2 * kTile * ((t - t0) & 1));
        }
        if (tw < t1) {
            stage_tail<64, true, 64>(mine, d.b, d.ldb, q0, d.Q, (int64_t)tw * kBR, d.R);
            stage_tail<16, false, 64>(mine + 64 * kBR, d.a, d.lda, 0, d.P, (int64_t)tw * kBR, d.R);
            asm volatile("s_waitcnt lgkmcnt(0)" : : : "memory");
            multiply(base);
        }
        meet_waves();
    }

    // [wave][row p][column]: a lane holds columns 16 j + 4 gr .. + 3 of row i
    float* const sums = reinterpret_cast<float*>(lds);
#pragma unroll
    for (int j = 0; j < FQ; ++j)
        *reinterpret_cast<v4f*>(sums + (wave * 16 + i) * kCols + 16 * j + 4 * gr) = acc[j];
    __syncthreads();
    const int p = threadIdx.x / (kCols / 8), c = threadIdx.x % (kCols / 8);
    const int64_t q = q0 + 8 * c;
    if (p >= 16 || p >= d.P || q >= d.Q) return;
    const int n = d.Q - q < 8 ? (int)(d.Q - q) : 8;
    float v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = 0.0f;
#pragma unroll 2
    for (int w = 0; w < kWaves; ++w) {
        const v4f lo = *reinterpret_cast<const v4f*>(sums + (w * 16 + p) * kCols + 8 * c);
        const v4f hi = *reinterpret_cast<const v4f*>(sums + (w * 16 + p) * kCols + 8 * c + 4);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            v[k] += lo[k];
            v[4 + k] += hi[k];
        }
    }
    EpilogueIn in;
    in.template load<EPI>(d, p, q, n);
    float bias[8];
    epilogue_bias(d, q, n, bias);
    epilogue8<EPI>(d, d.drop.thr ? drop_offset(d.drop) : 0, p, q, v, in, bias, n);
}

// Joins the splits of a long reduction in their order, then the epilogue, eight
// columns of one row per thread (10 splits of 1023 x 768: 10.7 us, 3.1 TB/s); and, in the workgroups behind those, the rows of
// partial sums of the bias gradient, 64 columns to a workgroup, its four waves on
// every fourth row and then joined in order.
template <int EPI>
__global__ void __launch_bounds__(256) k_join(const ProductArgs g) {
    const ProductDesc& d = g.d;
    if (EPI == kEpiGradWeight && blockIdx.x >= g.join_blocks) {
        __shared__ float s[3][64];
        const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
        const int64_t j = (blockIdx.x - g.join_blocks) * 64 + lane;
        float v = 0.0f;
        if (j < g.sum_n) {
#pragma unroll 4
            for (int r = wave; r < g.sum_rows; r += 4) v += g.sums[r * g.ld_sums + j];
        }
        if (wave) s[wave - 1][lane] = v;
        __syncthreads();
        if (wave || j >= g.sum_n) return;
        v = ((v + s[0][lane]) + s[1][lane]) + s[2][lane];
        if (d.out_f32) {
            float* o = static_cast<float*>(d.bias_out) + j;
            *o = d.bias_add ? *o + v : v;
        } else {
            uint16_t* o = static_cast<uint16_t*>(d.bias_out) + j;
            *o = bf_one(d.bias_add ? bf_f(*o) + v : v);
        }
        return;
    }
    const int64_t groups = g.ld_part / 8, id = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t p = id / groups, q = 8 * (id % groups);
    if (p >= d.P) return;
    const int n = d.Q - q < 8 ? (int)(d.Q - q) : 8;
    EpilogueIn in;
    in.template load<EPI>(d, p, q, n);
    float v[8], t[8], bias[8];
    epilogue_bias(d, q, n, bias);
    load8_f(v, g.part + p * g.ld_part + q, 8);
#pragma unroll 4
    for (int s = 1; s < g.splits; ++s) {
        load8_f(t, g.part + ((int64_t)s * d.P + p) * g.ld_part + q, 8);
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] += t[k];
    }
    epilogue8<EPI>(d, d.drop.thr ? drop_offset(d.drop) : 0, p, q, v, in, bias, n);
}

// How a product of these sizes runs: the kind of tile, and into how many parts its
// reduction is split, by an estimate of the time in microseconds. Measured on
// products of 256 and more tiles: a 64-deep step of a 256 x 256 tile takes 1.5, one
// of two 128 x 128 tiles that share a compute unit 1.0 (1.5 through registers), of
// one alone 0.65; a tile's start and epilogue 7 and 3; a join 3 and its bytes at
// 4.5 TB/s. A step of a 128 x 192 tile takes 0.5 in a round of its own and 0.8 in two that
// follow the wide tiles' (which then run slower, all compute units being busy). 0.72
// stands for either behind whole rounds of wide tiles: it gives the Llama-7B shaped
// layer's 8192 x 4096 x 11008 five rounds of wide tiles and one of 128 x 192 (610 -> 601
// us), the head's weight gradient (50,256 x 768) one of them too (88.4 -> 84.2 us), and the
// f32 weight gradient, whose rest would be two, none (627 against 638). Of 24 random sizes
// that 0.5 or 0.8 by the number of rounds would plan otherwise, 0.72 is faster at 20, by
// 3% at the median and 20% at most, and slower at two, by 1 and 9%.
struct Plan {
    bool wide;
    int32_t splits;
    int64_t per;                    // reduction elements per split
    int64_t full;                   // wide tiles of whole rounds of the chip; the rest as quarters,
    int64_t rows, cols;             // or, where these many tiles down and across are wide, in tiles of
};                                  // 128 x 192
static double small_time(int64_t tiles, int64_t steps, bool direct) {
    const double two = direct ? 1.0 : 1.5, one = direct ? 0.65 : 1.0;
    const int64_t full = tiles / 512, rest = tiles % 512;
    return full * (two * steps + 3) + (rest == 0 ? 0 : rest <= 256 ? one * steps + 3 : two * steps + 3);
}
static int64_t over(int64_t n, int64_t by) { return n > 0 ? (n + by - 1) / by : 0; }
static Plan plan_of(int64_t P, int64_t Q, int64_t R, bool direct, bool sums) {
    // a bias gradient beside a weight of no elements still has its column of tiles
    if (P < 1) P = 1;
    if (Q < 1) Q = 1;
    const int64_t tiles = ((P + 127) / 128) * ((Q + 127) / 128), wide = ((P + 255) / 256) * ((Q + 255) / 256);
    const int64_t steps = (R + kBR - 1) / kBR;
    const int64_t down = over(P, 256), across = over(Q, 256);
    Plan best{false, 1, steps > 0 ? steps * kBR : kBR, 0, down, across};
    double least = 1e300;
    for (int64_t s = 1; s <= 64 && (s == 1 || (steps + s - 1) / s >= 2); ++s) {
        const int64_t each = steps > 0 ? (steps + s - 1) / s : 1, parts = steps > 0 ? (steps + each - 1) / each : 1;
        // one round and a bit is as fast without a split's traffic
        if (s > 1 && tiles * s > 2048) break;
        const double join = parts > 1 ? 3 + (double)parts * P * Q * 8 / 4.5e6 : 0;
        const double small = small_time(tiles * parts, each, direct) + join;
        if (small < least) {
            least = small;
            best = Plan{false, (int32_t)parts, each * kBR, 0, down, across};
        }
        if (!direct) continue;
        const int64_t rounds = wide * parts / 256, rest = wide * parts % 256;
        const double round = 1.5 * each + 7;
        double t = (rounds + (rest > 0)) * round + join;
        int64_t full = wide;
        if (parts == 1 && rounds > 0 && rest > 0) {
            const double quarters = rounds * round + 3 + small_time(4 * rest, each, true);
            if (quarters < t) t = quarters, full = rounds * 256;
        }
        if (t < least) {
            least = t;
            best = Plan{true, (int32_t)parts, each * kBR, full, down, across};
        }
        if (parts > 1 || sums || rounds == 0 || rest == 0) continue;
        // the whole rounds as a rectangle, whole columns of tiles or whole rows
        for (int k = 0; k < 2; ++k) {
            const int64_t rows = k ? rounds * 256 / across : down, cols = k ? across : rounds * 256 / down;
            if (rows < 1 || cols < 1) continue;
            const int64_t left = k ? over(P - 256 * rows, 128) * over(Q, 192) : over(P, 128) * over(Q - 256 * cols, 192);
            t = over(rows * cols, 256) * round + over(left, 256) * (0.72 * each + 7) + 3;
            if (t < least) {
                least = t;
                best = Plan{true, 1, each * kBR, rows * cols, rows, cols};
            }
        }
    }
    return best;
}

// Whether a product of few rows goes to k_product_few, or to tiles, splits and a join,
// whichever an estimate in microseconds says is done first.
// With b's outer index in rows, the eight waves of a workgroup take 1.1 ns for an element
// of the reduction and 3% of that more for each row of a: one row of GPT-2 qkv 3.3 us, in
// tiles 8.2; of a Llama-7B shaped layer 17.4 and 19.9; of 8192 through 64 to 768 columns
// 11.7-12.0 and 12.1-15.1; but of 16,384 through the same 21-24 and 13-19. More than 4 rows
// go there below 32 MB of b, as every workgroup reads all of a (16 rows of the Llama-7B
// shaped layer 23.6 and 20.5). Where rows are not on 16 bytes the loads take 3.1 ns an
// element, and more workgroups than compute units queue: one row of 4097 through 64
// columns 16.1 and 9.4, through 4096 17.2 and 20.9, through 11,008 43 and 36.
// With reduced rows, 64 columns to a workgroup: where its workgroups' share of memory
// (55 KB/us each) beats the join's launch and traffic; rows on 16 bytes only.
static bool few(int64_t P, int64_t Q, int64_t R, bool tb, bool direct) {
    if (P < 1 || P > 16 || Q < 1 || Q > (int64_t(1) << 26)) return false;   // 2^31 threads
    const double bytes = 2.0 * Q * R, groups = (double)((Q + 63) / 64);
    if (tb) return direct && bytes / ((groups < 256 ? groups : 256) * 55e3) < 5 + bytes / 6e6;
    if (P > 4 && bytes >= (32 << 20)) return false;
    if (direct) return R * (1.12e-3 + 3.5e-5 * P) < 11 + bytes / 13e6;
    const double queue = Q > 4096 ? Q / 4096.0 : 1.0;
    return R < 2048 || R * (3.1e-3 + 1.8e-4 * P) * queue < 6.5 + bytes / 3.3e6;
}

static int64_t up8(int64_t n) { return (n + 7) / 8 * 8; }
static size_t part_bytes(const Plan& pl, int64_t P, int64_t Q) {
    return pl.splits > 1 ? (size_t)pl.splits * (size_t)P * (size_t)up8(Q) * sizeof(float) : 0;
}
static int32_t sum_rows(const Plan& pl, int64_t other) {
    if (other < 1) other = 1;
    return pl.splits * (int32_t)((other + (pl.wide ? 255 : 127)) / (pl.wide ? 256 : 128));
}

size_t product_ws_bytes(int64_t P, int64_t Q, int64_t R, bool ta, bool tb) {
    size_t most = 0;
    for (int direct = 0; direct < 2; ++direct) {
        if (!ta && few(P, Q, R, tb, direct != 0)) continue;
        for (int sums = 0; sums < (ta && tb ? 2 : 1); ++sums) {
            const size_t b = part_bytes(plan_of(P, Q, R, direct != 0, sums != 0), P, Q);
            if (b > most) most = b;
        }
    }
    return most;
}
size_t sums_ws_bytes(int64_t P, int64_t Q, int64_t R, bool of_a) {
    size_t most = 0;
    for (int direct = 0; direct < 2; ++direct) {
        const Plan pl = plan_of(P, Q, R, direct != 0, true);
        const size_t b = (size_t)sum_rows(pl, of_a ? Q : P) * (size_t)up8(of_a ? P : Q) * sizeof(float);
        if (b > most) most = b;
    }
    return most;
}

// Rows on 16 bytes, and a tile's rows within the 2 GiB that its offsets reach.
static bool direct_ok(const uint16_t* p, int64_t ld, int64_t rows) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && (rows <= 1 || (ld % 8 == 0 && ld < (int64_t(1) << 21)));
}

size_t product_ws_needed(const uint16_t* a, int64_t lda, const uint16_t* b, int64_t ldb, int64_t P, int64_t Q,
                         int64_t R, bool tb) {
    return few(P, Q, R, tb, direct_ok(a, lda, P) && direct_ok(b, ldb, tb ? R : Q)) ? 0
                                                                                  : product_ws_bytes(P, Q, R, false, tb);
}

template <bool TA, bool TB, int EPI>
static hipError_t product(const ProductDesc& d, hipStream_t st) {
    const bool some = d.P > 0 && d.Q > 0;
    const bool da = some && direct_ok(d.a, d.lda, TA ? d.R : d.P), db = some && direct_ok(d.b, d.ldb, TB ? d.R : d.Q);
    const bool direct = da && db;
    if constexpr (!TA)
        if (few(d.P, d.Q, d.R, TB, direct)) {
            ProductArgs g{};
            g.d = d;
            const int cols = TB ? 64 : 16;
            hipLaunchKernelGGL((k_product_few<TB, EPI>), dim3((unsigned)((d.Q + cols - 1) / cols)), dim3(512), 0, st, g);
            return hipGetLastError();
        }
    if (!some && !d.bias_out) return hipSuccess;
    const Plan pl = plan_of(d.P, d.Q, d.R, direct, EPI == kEpiGradWeight && d.bias_out);
    const int64_t P = d.P > 0 ? d.P : 1, Q = d.Q > 0 ? d.Q : 1;     // a bias alone has tiles too
    const int64_t tiles = over(P, 128) * over(Q, 128), wide = pl.rows * pl.cols;
    const bool rectangle = pl.rows * 256 < P || pl.cols * 256 < Q;
    ProductArgs g{};
    g.d = d;
    g.splits = pl.splits;
    g.r_per_split = pl.per;
    g.ld_part = up8(d.Q);
    g.part = pl.splits > 1 ? d.ws : nullptr;
    if (EPI == kEpiGradWeight && d.bias_out) {
        g.sum_of = d.bias_of_a ? 1 : 2;
        g.sum_n = d.bias_of_a ? d.P : d.Q;
        g.ld_sums = up8(g.sum_n);
        g.sum_rows = sum_rows(pl, d.bias_of_a ? d.Q : d.P);
        g.sums = d.ws_sums;
    }
    const unsigned splits = (unsigned)pl.splits;
    constexpr bool kSums = EPI == kEpiGradWeight;
    hipError_t e = hipSuccess;
    if (pl.wide) {
        g.tiles = (int32_t)pl.full;
        g.np = (int32_t)pl.rows;
        g.nq = (int32_t)pl.cols;
        const auto k = kSums && g.sums ? k_product_wide<TA, TB, EPI, kSums> : k_product_wide<TA, TB, EPI, false>;
        hipLaunchKernelGGL(k, dim3((unsigned)pl.full * splits), dim3(512), 0, st, g);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    if (!pl.wide || pl.full < wide || rectangle) {
        const bool quarters = pl.wide && !rectangle;
        g.first_wide = quarters ? (int32_t)pl.full : -1;
        if (!quarters) {
            if (rectangle && pl.cols * 256 < Q) g.q0 = pl.cols * 256;
            else if (rectangle) g.p0 = pl.rows * 256;
            g.np = (int32_t)over(P - g.p0, 128);
            g.nq = (int32_t)over(Q - g.q0, 128);
        }
        g.tiles = (int32_t)(quarters ? 4 * (wide - pl.full) : tiles);
        // Tiles that get a compute unit each go to the eight-wave kernel (8192 x 768 x 2304
        // forward, whose quarters they are, 43.1 -> 40.4 us), more to the four-wave one, two
        // to a unit (with eight waves the GPT-2 projection 19.5 -> 23.1 us, its gradient by
        // input over 2304 outputs 34.6 -> 39.9); and where 192 columns a tile make them fit,
        // to the eight-wave kernel again (those two 19.1 -> 18.4 and 33.1 -> 28.9 us).
        const bool mid = direct && !rectangle && (int64_t)g.tiles * splits <= 256;
        const int64_t across3 = over(Q - g.q0, 192), tiles3 = g.np * across3;
        const bool three = rectangle || (direct && !mid && !pl.wide && splits == 1 && !g.sums && tiles3 <= 256);
        if (three) {
            g.nq = (int32_t)across3;
            g.tiles = (int32_t)tiles3;
        }
        const auto pick = [&](auto sums) {
            constexpr bool S = decltype(sums)::value;
            return mid ? k_product_mid<TA, TB, EPI, S, 2>
                       : da ? (db ? k_product<TA, TB, EPI, true, true, S> : k_product<TA, TB, EPI, true, false, S>)
                            : (db ? k_product<TA, TB, EPI, false, true, S> : k_product<TA, TB, EPI, false, false, S>);
        };
        const auto k = three ? k_product_mid<TA, TB, EPI, false, 3>
                             : kSums && g.sums ? pick(std::integral_constant<bool, kSums>{}) : pick(std::false_type{});
        hipLaunchKernelGGL(k, dim3((unsigned)g.tiles * splits), dim3(mid || three ? 512 : 256), 0, st, g);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    if (!g.part && !g.sums) return e;
    g.join_blocks = g.part ? (d.P * (g.ld_part / 8) + 255) / 256 : 0;
    const int64_t blocks = g.join_blocks + (g.sums ? (g.sum_n + 63) / 64 : 0);
    hipLaunchKernelGGL((k_join<EPI>), dim3((unsigned)blocks), dim3(256), 0, st, g);
    return hipGetLastError();
}

hipError_t launch_product(const ProductDesc& d, hipStream_t st) {
    if (d.epi == kEpiForward)
        return d.tb ? product<false, true, kEpiForward>(d, st) : product<false, false, kEpiForward>(d, st);
    if (d.epi == kEpiGradInput)
        return d.tb ? product<false, true, kEpiGradInput>(d, st) : product<false, false, kEpiGradInput>(d, st);
    return product<true, true, kEpiGradWeight>(d, st);
}

}  // namespace zk
