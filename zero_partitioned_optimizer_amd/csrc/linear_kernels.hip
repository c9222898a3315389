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

#include "layer_device.h"

namespace zk {

constexpr int kBR = 64;             // reduction elements per staged tile

struct ProductArgs {
    ProductDesc d;
    int64_t r_per_split;            // multiple of kBR
    int32_t splits;
    int64_t ld_part;                // row length of a split's partial products
    float* part;                    // [splits, P, ld_part], or nullptr: epilogue in place
};

// Staged tiles hold eight-element chunks (16 bytes), permuted within a row so that
// the lanes that read together meet different banks.
//   outer rows:   [rows][kBR], chunk c of row o at c ^ (o & 7): the 8 lanes of a
//                 16-byte read hold 8 rows at one c.
//   reduced rows: [kBR][cols], chunk c of row r at c ^ perm(r): a transposing read
//                 takes 4 rows x 32 bytes per 16 lanes, and two such groups 8 rows apart.
template <int COLS>
__device__ __forceinline__ int perm_reduced(int r) {
    return ((r & 3) << 1) | (COLS >= 128 ? ((r >> 3) & 1) << 3 : 0);
}

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

// A tile through registers into LDS: all of a thread's chunks loaded, then stored
// (Stage), or one at a time where registers are short (stage_tail).
template <int ROWS, bool T, int THREADS>
struct Stage {
    static constexpr int kChunks = ROWS * kBR / 8 / THREADS;
    v4u w[kChunks];
    __device__ __forceinline__ void load(const uint16_t* src, int64_t ld, int64_t o0, int64_t O, int64_t r0,
                                         int64_t r1) {
#pragma unroll
        for (int i = 0; i < kChunks; ++i)
            w[i] = tile_chunk<ROWS, T>(threadIdx.x + i * THREADS, src, ld, o0, O, r0, r1);
    }
    __device__ __forceinline__ void store(uint16_t* lds) const {
#pragma unroll
        for (int i = 0; i < kChunks; ++i) put_chunk<ROWS, T>(lds, threadIdx.x + i * THREADS, w[i]);
    }
};
template <int ROWS, bool T, int THREADS>
__device__ __forceinline__ void stage_tail(uint16_t* lds, const uint16_t* src, int64_t ld, int64_t o0, int64_t O,
                                           int64_t r0, int64_t r1) {
#pragma unroll 1
    for (int id = threadIdx.x; id < ROWS * kBR / 8; id += THREADS)
        put_chunk<ROWS, T>(lds, id, tile_chunk<ROWS, T>(id, src, ld, o0, O, r0, r1));
}

typedef __attribute__((address_space(3))) const uint16_t lds_u16;
typedef __attribute__((address_space(3))) const v8bf lds_v8bf;
typedef __attribute__((address_space(3))) v4bf lds_v4bf;
__device__ __forceinline__ uint32_t lds_address(const uint16_t* p) {
    return (uint32_t)reinterpret_cast<uintptr_t>((lds_u16*)p);
}

// The matrix instruction's operands from a staged tile: for block i, lane l holds
// outer index o0 + 16 i + (l & 15) and reduction elements 32 s + 8 (l >> 4) .. + 7.
// o0 is a multiple of the outer indices that the wave's blocks cover, a power of
// two, so one byte offset per lane serves all blocks: a constant is added to it,
// or, where a block's chunks lie under the permutation, exchanged into it.
template <int ROWS, bool T>
struct Fragments {
    uint32_t at;
    __device__ __forceinline__ explicit Fragments(int o0) {
        const int lane = threadIdx.x & 63, i = lane & 15, g = lane >> 4;
        if constexpr (T) {
            const int r = 8 * g + (i >> 2), chunk = (o0 >> 3) + ((i & 3) >> 1);
            at = 2 * (r * ROWS + 8 * (chunk ^ perm_reduced<ROWS>(r)) + 4 * (i & 1));
        } else {
            const int o = o0 + i;
            at = 2 * (o * kBR + 8 * (g ^ (o & 7)));
        }
    }
    __device__ __forceinline__ v8bf get(uint32_t tile, int i, int s) const {
        if constexpr (T) {
            // rows 32 further on have the same permutation
            const uint32_t p = tile + (at ^ (32u * i)) + 2 * 32 * ROWS * s;
            const v4bf lo = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_v4bf*)p);
            const v4bf hi = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_v4bf*)(p + 2 * 4 * ROWS));
            return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
        } else {
            return *(lds_v8bf*)(tile + (at ^ (64u * s)) + 2 * 16 * kBR * i);
        }
    }
};

// The epilogue of eight consecutive columns q .. of row p; n of them exist.
template <int EPI>
__device__ __forceinline__ void epilogue8(const ProductDesc& d, uint64_t off, int64_t p, int64_t q,
                                          float v[8], int n) {
    float t[8];
    if constexpr (EPI == kEpiForward) {
        if (d.bias) {
            load8_bf(t, d.bias + q, n);
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] += t[k];
        }
        if (d.z_out) store8_bf(d.z_out + p * d.ld_z + q, v, n);
        if (d.act != ZERO_ACT_NONE)
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = act_of(d.act, v[k]);
        if (d.drop.thr) drop8(v, d.drop, off, (uint32_t)p, (uint32_t)(q >> 3));
    }
    if constexpr (EPI == kEpiGradInput) {
        if (d.z_in) {
            load8_bf(t, d.z_in + p * d.ld_z + q, n);
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] *= act_slope(d.act, t[k]);
        }
        if (d.drop.thr) drop8(v, d.drop, off, (uint32_t)p, (uint32_t)(q >> 3));
    }
    if (d.res) {
        if (d.out_f32) load8_f(t, static_cast<const float*>(d.res) + p * d.ld_res + q, n);
        else load8_bf(t, static_cast<const uint16_t*>(d.res) + p * d.ld_res + q, n);
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] += t[k];
    }
    if (d.out_f32) store8_f(static_cast<float*>(d.out) + p * d.ld_out + q, v, n);
    else store8_bf(static_cast<uint16_t*>(d.out) + p * d.ld_out + q, v, n);
}

typedef int v4i __attribute__((ext_vector_type(4)));

// 16 bytes a lane from the buffer's byte `at` to LDS, lane l of the wave to byte
// 16 l behind `to` (the same in all lanes). Written in assembly because the
// compiler, which sees in its own builtin a store to LDS of unknown extent, waits
// for it before the next LDS read of any tile. It has no output register; what
// reads the tile waits with loads_landed first.
__device__ __forceinline__ void lds_load(v4i rsrc, uint32_t at, uint32_t to) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
                 :
                 : "s"(to), "v"(at), "s"(rsrc)
                 : "memory");
}
// Until at most N of this wave's loads are under way.
template <int N>
__device__ __forceinline__ void loads_landed() {
    asm volatile("s_waitcnt vmcnt(%0)" : : "n"(N) : "memory");
}
// All waves have come here and their LDS reads and writes are done.
__device__ __forceinline__ void meet_waves() {
    asm volatile("" : : : "memory");
    __builtin_amdgcn_s_waitcnt(0xC07F);         // lgkmcnt(0), where the compiler counts it too
    asm volatile("s_barrier" : : : "memory");
}

// One operand's tiles from memory straight into LDS: 16 bytes a lane, lane l of a
// wave to byte 16 l behind the wave's LDS address, so the chunk permutation is
// applied to the address that a lane reads. Rows and chunks outside the operand
// read its last ones instead: they only reach outputs that do not exist. Used
// where rows start on 16 bytes and a whole tile of the reduction is left.
template <int ROWS, bool T, int THREADS>
struct Direct {
    static constexpr int kLoads = ROWS * kBR / 8 / THREADS;
    uint32_t at[kLoads];            // byte offsets from `base`
    const char* base;
    int64_t step;
    __device__ __forceinline__ void init(const uint16_t* src, int64_t ld, int64_t o0, int64_t O, int64_t r0) {
        if (o0 >= O) o0 = (O - 1) & ~int64_t(7);        // a half tile with nothing in it
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int id = threadIdx.x + i * THREADS;
            if constexpr (T) {
                const int r = id / (ROWS / 8);
                int64_t c = 8 * ((id % (ROWS / 8)) ^ perm_reduced<ROWS>(r));
                if (o0 + c >= O) c = (O - 1 - o0) & ~int64_t(7);
                at[i] = (uint32_t)((r * ld + c) * 2);
            } else {
                int64_t o = id / (kBR / 8);
                const int c = 8 * ((id % (kBR / 8)) ^ (int)(o & 7));
                if (o0 + o >= O) o = O - 1 - o0;
                at[i] = (uint32_t)((o * ld + c) * 2);
            }
        }
        base = reinterpret_cast<const char*>(src + (T ? r0 * ld + o0 : o0 * ld + r0));
        step = (T ? kBR * ld : kBR) * 2;
    }
    // The tile's loads to LDS byte address `tile`; `wave` is the same in all lanes.
    // With `records` 0 the buffer's range check stops them (they still count as loads).
    __device__ __forceinline__ void issue(uint32_t tile, int wave, int records) {
        const v4i rsrc = {(int)(uint32_t)reinterpret_cast<uintptr_t>(base),
                          (int)(uint32_t)(reinterpret_cast<uintptr_t>(base) >> 32), records, 0x00020000};
#pragma unroll
        for (int i = 0; i < kLoads; ++i) lds_load(rsrc, at[i], tile + 16 * (i * THREADS + 64 * wave));
        base += step;
    }
};

// The output tile of a workgroup. Workgroups go to the 8 XCDs in turn, each with an
// L2 of its own, so each XCD gets a run of consecutive tiles; runs walk down blocks
// of kTileRows rows of tiles, column by column, so that the 32 workgroups that an
// XCD runs at a time share few operand rows.
// (Llama-7B shaped products: 8 rows 5% faster than tiles in order, 4 or 16 rows 2%
// behind 8 on the deepest reductions.)
constexpr int kTileRows = 8;
__device__ __forceinline__ void tile_of(int id, int tiles, int np, int nq, int* tp, int* tq) {
    const int xcd = id & 7, slot = id >> 3, each = tiles >> 3, more = tiles & 7;
    const int t = xcd * each + (xcd < more ? xcd : more) + slot;
    const int block = t / (kTileRows * nq), in = t - block * kTileRows * nq;
    const int rows = np - block * kTileRows < kTileRows ? np - block * kTileRows : kTileRows;
    *tq = in / rows;
    *tp = block * kTileRows + in - *tq * rows;
}

// The epilogue of a workgroup's tile, through LDS: kRun rows of a wave's blocks at a
// time, so that a lane gets eight consecutive columns and stores 16 bytes or more.
// Blocks are computed as (q, p), so a lane holds four consecutive columns of one
// output row, one 16-byte unit. Each wave has its own part of LDS; unit u of row o
// lies at u ^ (o & 15). row_of(i) and col_of(j): first row and column of the wave's
// blocks (i, j) in the output; the rows of a run are consecutive.
template <int EPI, int LDS_BYTES, int WAVES, int FP, int FQ, typename Row, typename Col>
__device__ __forceinline__ void finish(const ProductArgs& g, const v4f (&acc)[FP][FQ], uint16_t* lds, int wave,
                                       Row row_of, Col col_of) {
    static_assert(FQ == 4, "16 units a row");
    constexpr int kFit = LDS_BYTES / (WAVES * 16 * 64 * 4), kRun = kFit >= 4 ? 4 : kFit;
    static_assert(kRun >= 1 && FP % kRun == 0, "the runs cover a wave's rows");
    const ProductDesc& d = g.d;
    const int lane = threadIdx.x & 63;
    const uint64_t off = d.drop.thr ? drop_offset(d.drop) : 0;
    float* const mine = reinterpret_cast<float*>(lds) + wave * kRun * 16 * 64;
#pragma unroll
    for (int i0 = 0; i0 < FP; i0 += kRun) {
#pragma unroll
        for (int i = 0; i < kRun; ++i)
#pragma unroll
            for (int j = 0; j < FQ; ++j) {
                const int o = 16 * i + (lane & 15), u = 4 * j + (lane >> 4);
                *reinterpret_cast<v4f*>(mine + o * 64 + 4 * (u ^ (o & 15))) = acc[i0 + i][j];
            }
        const int c = lane & 7;
        const int64_t q = col_of(c >> 1) + 8 * (c & 1);
#pragma unroll 1
        for (int o = lane >> 3; o < 16 * kRun; o += 8) {
            const v4f lo = *reinterpret_cast<const v4f*>(mine + o * 64 + 4 * ((2 * c) ^ (o & 15)));
            const v4f hi = *reinterpret_cast<const v4f*>(mine + o * 64 + 4 * ((2 * c + 1) ^ (o & 15)));
            float v[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
            const int64_t p = row_of(i0) + o;
            if (p >= d.P || q >= d.Q) continue;
            const int n = d.Q - q < 8 ? (int)(d.Q - q) : 8;
            if (g.part) store8_f(g.part + ((int64_t)blockIdx.y * d.P + p) * g.ld_part + q, v, 8);
            else epilogue8<EPI>(d, off, p, q, v, n);
        }
    }
}

// 128 x 128 outputs by four waves, 64 x 64 each (4 x 4 blocks), for outputs of few
// tiles and, without DIRECT, for operands at any address: tiles of 64 reduction
// elements, two in LDS, the next one loading while one is multiplied. Two
// workgroups of 64 KB fit a compute unit and fill each other's waits.
template <bool TA, bool TB, int EPI, bool DIRECT>
__global__ void __launch_bounds__(256) k_product(const ProductArgs g) {
    constexpr int T = 256, B = 128, FP = 4, FQ = 4, kTile = B * kBR;
    constexpr int kBufs = DIRECT ? 2 : 1;
    __shared__ __attribute__((aligned(16))) uint16_t lds[kBufs * 2 * kTile];
    const ProductDesc& d = g.d;
    int tp, tq;
    tile_of(blockIdx.x, gridDim.x, (int)((d.P + B - 1) / B), (int)((d.Q + B - 1) / B), &tp, &tq);
    const int64_t p0 = (int64_t)tp * B, q0 = (int64_t)tq * B;
    const int64_t r0 = (int64_t)blockIdx.y * g.r_per_split;
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
    const auto multiply = [&](uint32_t tile) {
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
        }
    };

    if constexpr (DIRECT) {
        const int full = (int)((r1 - r0) / kBR);
        Direct<B, TA, T> da;
        Direct<B, TB, T> db;
        if (full > 0) {
            da.init(d.a, d.lda, p0, d.P, r0);
            db.init(d.b, d.ldb, q0, d.Q, r0);
            da.issue(base, wave, -1);
            db.issue(base + 2 * kTile, wave, -1);
        }
        for (int k = 0; k < full; ++k) {
            loads_landed<0>();
            meet_waves();
            const uint32_t tile = base + 4 * kTile * (k & 1), next = base + 4 * kTile * ((k + 1) & 1);
            if (k + 1 < full) {
                da.issue(next, wave, -1);
                db.issue(next + 2 * kTile, wave, -1);
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
        Stage<B, TA, T> sa;
        Stage<B, TB, T> sb;
        if (r0 < r1) {
            sa.load(d.a, d.lda, p0, d.P, r0, r1);
            sb.load(d.b, d.ldb, q0, d.Q, r0, r1);
        }
        for (int64_t r = r0; r < r1; r += kBR) {
            __syncthreads();
            sa.store(lds);
            sb.store(lds + kTile);
            __syncthreads();
            if (r + kBR < r1) {
                sa.load(d.a, d.lda, p0, d.P, r + kBR, r1);
                sb.load(d.b, d.ldb, q0, d.Q, r + kBR, r1);
            }
            multiply(base);
        }
    }
    meet_waves();
    finish<EPI, sizeof(lds), 4>(g, acc, lds, wave, [&](int i) { return p0 + wp + 16 * i; },
                                [&](int j) { return q0 + wq + 16 * j; });
}

// 256 x 256 outputs by eight waves, one workgroup to a compute unit. Operand tiles of
// 64 reduction elements lie in LDS as halves of 128 outer indices, two tiles of four
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
template <bool TA, bool TB, int EPI>
__global__ void __launch_bounds__(512) k_product_wide(const ProductArgs g) {
    constexpr int T = 512, B = 256, H = 128, kHalf = H * kBR;
    __shared__ __attribute__((aligned(16))) uint16_t lds[2 * 4 * kHalf];
    const ProductDesc& d = g.d;
    int tp, tq;
    tile_of(blockIdx.x, gridDim.x, (int)((d.P + B - 1) / B), (int)((d.Q + B - 1) / B), &tp, &tq);
    const int64_t p0 = (int64_t)tp * B, q0 = (int64_t)tq * B;
    const int64_t r0 = (int64_t)blockIdx.y * g.r_per_split;
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

    const int n = (int)((r1 - r0) / kBR);
    if (n > 0) {
        Direct<H, TA, T> a0, a1;
        Direct<H, TB, T> b0, b1;
        constexpr int kLoads = Direct<H, TA, T>::kLoads;
        a0.init(d.a, d.lda, p0, d.P, r0);
        a1.init(d.a, d.lda, p0 + H, d.P, r0);
        b0.init(d.b, d.ldb, q0, d.Q, r0);
        b1.init(d.b, d.ldb, q0 + H, d.Q, r0);
        // loads of tiles behind the last are stopped by their buffer's range
        const auto there = [&](int k) { return __builtin_amdgcn_readfirstlane(k < n ? -1 : 0); };
        a0.issue(half(0, 0), wave, -1);
        b0.issue(half(0, 2), wave, -1);
        b1.issue(half(0, 3), wave, -1);
        a1.issue(half(0, 1), wave, -1);
        a0.issue(half(1, 0), wave, there(1));
        b0.issue(half(1, 2), wave, there(1));
        b1.issue(half(1, 3), wave, there(1));
        loads_landed<5 * kLoads>();
        meet_waves();
        if (wave >= 4) meet_waves();
#pragma unroll 1
        for (int k = 0; k < n; ++k) {
            const int one = there(k + 1), two = there(k + 2);
            read_b(0, half(k, 2));
            read_a(half(k, 0));
            a1.issue(half(k + 1, 1), wave, one);
            loads_landed<5 * kLoads>();
            meet_waves();
            multiply(0, 0);
            meet_waves();
            read_b(1, half(k, 3));
            a0.issue(half(k, 0), wave, two);
            loads_landed<5 * kLoads>();
            meet_waves();
            multiply(0, 1);
            meet_waves();
            read_a(half(k, 1));
            b0.issue(half(k, 2), wave, two);
            loads_landed<5 * kLoads>();
            meet_waves();
            multiply(1, 1);
            meet_waves();
            b1.issue(half(k, 3), wave, two);
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
        read_b(0, half(0, 2));
        read_b(1, half(0, 3));
        read_a(half(0, 0));
        multiply(0, 0);
        multiply(0, 1);
        read_a(half(0, 1));
        multiply(1, 1);
        multiply(1, 0);
        meet_waves();
    }
    finish<EPI, sizeof(lds), 8>(g, acc, lds, wave, [&](int i) { return p0 + H * (i >> 2) + wp + 16 * (i & 3); },
                                [&](int j) { return q0 + H * (j >> 1) + wq + 16 * (j & 1); });
}

// Joins the splits of a long reduction in their order, then the epilogue: eight
// columns of one row per thread.
template <int EPI>
__global__ void __launch_bounds__(256) k_join(const ProductArgs g) {
    const ProductDesc& d = g.d;
    const int64_t groups = g.ld_part / 8, id = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t p = id / groups, q = 8 * (id % groups);
    if (p >= d.P) return;
    float v[8], t[8];
    load8_f(v, g.part + p * g.ld_part + q, 8);
    for (int s = 1; s < g.splits; ++s) {
        load8_f(t, g.part + ((int64_t)s * d.P + p) * g.ld_part + q, 8);
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] += t[k];
    }
    const int n = d.Q - q < 8 ? (int)(d.Q - q) : 8;
    epilogue8<EPI>(d, d.drop.thr ? drop_offset(d.drop) : 0, p, q, v, n);
}

// How the reduction of a product of these sizes is split.
struct Split {
    int32_t splits;
    int64_t per;
};
static Split split_of(int64_t P, int64_t Q, int64_t R) {
    const int64_t tiles = ((P + 127) / 128) * ((Q + 127) / 128), steps = (R + kBR - 1) / kBR;
    int64_t s = tiles > 0 && tiles < 256 ? 512 / tiles : 1;
    if (s > steps / 4) s = steps / 4;
    if (s < 1) s = 1;
    const int64_t per = (steps + s - 1) / s * kBR;
    return Split{(int32_t)(per > 0 ? (R + per - 1) / per : 1), per > 0 ? per : kBR};
}

size_t product_ws_bytes(int64_t P, int64_t Q, int64_t R) {
    const Split s = split_of(P, Q, R);
    return s.splits > 1 ? (size_t)s.splits * (size_t)P * (size_t)((Q + 7) / 8 * 8) * sizeof(float) : 0;
}

// Rows on 16 bytes, and a tile's rows within the 2 GiB that its offsets reach.
static bool direct_ok(const uint16_t* p, int64_t ld, int64_t rows) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && (rows <= 1 || (ld % 8 == 0 && ld < (int64_t(1) << 21)));
}

template <bool TA, bool TB, int EPI>
static hipError_t product(ProductArgs& g, hipStream_t st) {
    const ProductDesc& d = g.d;
    if (d.P <= 0 || d.Q <= 0) return hipSuccess;
    const bool direct = direct_ok(d.a, d.lda, TA ? d.R : d.P) && direct_ok(d.b, d.ldb, TB ? d.R : d.Q);
    const int64_t wide = ((d.P + 255) / 256) * ((d.Q + 255) / 256), tiles = ((d.P + 127) / 128) * ((d.Q + 127) / 128);
    if (tiles > INT32_MAX) return hipErrorInvalidValue;
    const unsigned splits = (unsigned)g.splits;
    if (direct && wide >= 256)
        hipLaunchKernelGGL((k_product_wide<TA, TB, EPI>), dim3((unsigned)wide, splits), dim3(512), 0, st, g);
    else if (direct)
        hipLaunchKernelGGL((k_product<TA, TB, EPI, true>), dim3((unsigned)tiles, splits), dim3(256), 0, st, g);
    else
        hipLaunchKernelGGL((k_product<TA, TB, EPI, false>), dim3((unsigned)tiles, splits), dim3(256), 0, st, g);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || !g.part) return e;
    const int64_t blocks = (d.P * (g.ld_part / 8) + 255) / 256;
    hipLaunchKernelGGL((k_join<EPI>), dim3((unsigned)blocks), dim3(256), 0, st, g);
    return hipGetLastError();
}

hipError_t launch_product(const ProductDesc& d, hipStream_t st) {
    const Split s = split_of(d.P, d.Q, d.R);
    ProductArgs g{};
    g.d = d;
    g.splits = s.splits;
    g.r_per_split = s.per;
    g.ld_part = (d.Q + 7) / 8 * 8;
    g.part = s.splits > 1 ? d.ws : nullptr;
    if (d.epi == kEpiForward)
        return d.tb ? product<false, true, kEpiForward>(g, st) : product<false, false, kEpiForward>(g, st);
    if (d.epi == kEpiGradInput)
        return d.tb ? product<false, true, kEpiGradInput>(g, st) : product<false, false, kEpiGradInput>(g, st);
    return product<true, true, kEpiGradWeight>(g, st);
}

// Column sums of dz: each workgroup sums a run of rows for 512 columns (eight
// columns to a thread, four waves on alternate rows, joined in LDS), and a second
// kernel adds the runs in their order.
constexpr int kSumCols = 512;
static int64_t sum_runs(int64_t M, int64_t N) {
    const int64_t cols = (N + kSumCols - 1) / kSumCols;
    int64_t runs = cols > 0 ? 512 / cols : 1;
    const int64_t most = (M + 31) / 32;
    if (runs > most) runs = most;
    return runs < 1 ? 1 : runs;
}

size_t colsum_ws_bytes(int64_t M, int64_t N) {
    return (size_t)sum_runs(M, N) * (size_t)((N + 7) / 8 * 8) * sizeof(float);
}

__global__ void __launch_bounds__(256) k_colsum(const uint16_t* dz, int64_t ld, int64_t M, int64_t N,
                                                int64_t rows, float* part) {
    __shared__ float s[3][kSumCols];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int64_t j = (int64_t)blockIdx.x * kSumCols + 8 * lane;
    const int64_t m0 = (int64_t)blockIdx.y * rows, m1 = m0 + rows < M ? m0 + rows : M;
    const int n = N - j >= 8 ? 8 : N - j > 0 ? (int)(N - j) : 0;
    float v[8], t[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = 0.0f;
    if (n > 0)
        for (int64_t m = m0 + wave; m < m1; m += 4) {
            load8_bf(t, dz + m * ld + j, n);
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] += t[k];
        }
    if (wave)
#pragma unroll
        for (int k = 0; k < 8; ++k) s[wave - 1][8 * lane + k] = v[k];
    __syncthreads();
    if (wave == 0 && n > 0) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            v[k] = ((v[k] + s[0][8 * lane + k]) + s[1][8 * lane + k]) + s[2][8 * lane + k];
        store8_f(part + (int64_t)blockIdx.y * ((N + 7) / 8 * 8) + j, v, 8);
    }
}

__global__ void __launch_bounds__(256) k_colsum_join(const float* part, int64_t N, int runs, void* out, bool f32,
                                                     bool accumulate) {
    const int64_t j = (int64_t)blockIdx.x * 256 + threadIdx.x, ld = (N + 7) / 8 * 8;
    if (j >= N) return;
    float v = 0.0f;
    for (int s = 0; s < runs; ++s) v += part[s * ld + j];
    if (f32) {
        float* o = static_cast<float*>(out) + j;
        *o = accumulate ? *o + v : v;
    } else {
        uint16_t* o = static_cast<uint16_t*>(out) + j;
        *o = bf_one(accumulate ? bf_f(*o) + v : v);
    }
}

hipError_t launch_colsum(const uint16_t* dz, int64_t ld, int64_t M, int64_t N, void* out, bool out_f32,
                         bool accumulate, float* ws, hipStream_t st) {
    if (N <= 0) return hipSuccess;
    const int64_t runs = sum_runs(M, N), rows = (M + runs - 1) / runs;
    hipLaunchKernelGGL(k_colsum, dim3((unsigned)((N + kSumCols - 1) / kSumCols), (unsigned)runs), dim3(256), 0,
                       st, dz, ld, M, N, rows, ws);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(k_colsum_join, dim3((unsigned)((N + 255) / 256)), dim3(256), 0, st, ws, N, (int)runs, out,
                       out_f32, accumulate);
    return hipGetLastError();
}

}  // namespace zk
