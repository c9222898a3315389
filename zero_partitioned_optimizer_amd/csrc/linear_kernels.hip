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

typedef __attribute__((address_space(3))) uint16_t lds_u16;

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

// The matrix instruction's operand for 16 outer indices from o0 and reduction
// elements 32 * s .. 32 * s + 31 of a staged tile: lane l holds outer index
// o0 + (l & 15) and elements 8 * (l >> 4) .. + 7.
template <int ROWS, bool T>
__device__ __forceinline__ v8bf fragment(const uint16_t* lds, int o0, int s) {
    const int lane = threadIdx.x & 63, i = lane & 15, g = lane >> 4;
    if constexpr (T) {
        const int r = 32 * s + 8 * g + (i >> 2), col = o0 + 4 * (i & 3);
        const int at = r * ROWS + 8 * ((col >> 3) ^ perm_reduced<ROWS>(r)) + (col & 7);
        typedef __attribute__((address_space(3))) v4bf lds_v4bf;
        const v4bf lo = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_v4bf*)(lds + at));
        const v4bf hi = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_v4bf*)(lds + at + 4 * ROWS));
        return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    } else {
        const int o = o0 + i, c = 4 * s + g;
        return *reinterpret_cast<const v8bf*>(lds + o * kBR + 8 * (c ^ (o & 7)));
    }
}

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
__device__ __forceinline__ void lds_load(v4i rsrc, uint32_t at, const uint16_t* to) {
    const uint32_t m0 = __builtin_amdgcn_readfirstlane(
        (uint32_t)reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) const void*)to));
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
                 :
                 : "s"(m0), "v"(at), "s"(rsrc)
                 : "memory");
}
// Until at most N of this wave's loads are under way.
template <int N>
__device__ __forceinline__ void loads_landed() {
    asm volatile("s_waitcnt vmcnt(%0)" : : "n"(N) : "memory");
}
// All waves have come here and their LDS reads and writes are done.
__device__ __forceinline__ void meet_waves() {
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" : : : "memory");
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
    __device__ __forceinline__ void issue(uint16_t* lds) {
        const v4i rsrc = {(int)(uint32_t)reinterpret_cast<uintptr_t>(base),
                          (int)(uint32_t)(reinterpret_cast<uintptr_t>(base) >> 32), -1, 0x00020000};
#pragma unroll
        for (int i = 0; i < kLoads; ++i) lds_load(rsrc, at[i], lds + 8 * (i * THREADS + (threadIdx.x & ~63)));
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

// NWP x NWQ waves, each with FP x FQ blocks of 16 x 16 outputs. The blocks are
// computed as (q, p), so a lane holds four consecutive columns of one output row;
// and so 16 bytes of the tile that the epilogue takes through LDS.
template <int NWP, int NWQ, int FP, int FQ, bool TA, bool TB, int EPI, bool DIRECT>
__global__ void __launch_bounds__(64 * NWP * NWQ) k_product(const ProductArgs g) {
    constexpr int T = 64 * NWP * NWQ, BP = 16 * FP * NWP, BQ = 16 * FQ * NWQ;
    constexpr int kBufs = DIRECT ? 2 : 1;
    __shared__ __attribute__((aligned(16))) uint16_t lds[kBufs * (BP + BQ) * kBR];
    const auto la = [&](int k) { return lds + k * (BP + BQ) * kBR; };
    const auto lb = [&](int k) { return lds + k * (BP + BQ) * kBR + BP * kBR; };
    const ProductDesc& d = g.d;
    int tp, tq;
    tile_of(blockIdx.x, gridDim.x, (int)((d.P + BP - 1) / BP), (int)((d.Q + BQ - 1) / BQ), &tp, &tq);
    const int64_t p0 = (int64_t)tp * BP, q0 = (int64_t)tq * BQ;
    const int64_t r0 = (int64_t)blockIdx.y * g.r_per_split;
    const int64_t r1 = r0 + g.r_per_split < d.R ? r0 + g.r_per_split : d.R;
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int wp = (wave / NWQ) * 16 * FP, wq = (wave % NWQ) * 16 * FQ;

    v4f acc[FP][FQ];
#pragma unroll
    for (int i = 0; i < FP; ++i)
#pragma unroll
        for (int j = 0; j < FQ; ++j) acc[i][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};

    const auto multiply = [&](const uint16_t* ta, const uint16_t* tb) {
#pragma unroll
        for (int s = 0; s < kBR / 32; ++s) {
            v8bf fa[FP], fb[FQ];
#pragma unroll
            for (int i = 0; i < FP; ++i) fa[i] = fragment<BP, TA>(ta, wp + 16 * i, s);
#pragma unroll
            for (int j = 0; j < FQ; ++j) fb[j] = fragment<BQ, TB>(tb, wq + 16 * j, s);
#pragma unroll
            for (int i = 0; i < FP; ++i)
#pragma unroll
                for (int j = 0; j < FQ; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fb[j], fa[i], acc[i][j], 0, 0, 0);
        }
    };

    if constexpr (DIRECT) {
        const int full = (int)((r1 - r0) / kBR);
        Direct<BP, TA, T> da;
        Direct<BQ, TB, T> db;
        if (full > 0) {
            da.init(d.a, d.lda, p0, d.P, r0);
            db.init(d.b, d.ldb, q0, d.Q, r0);
            da.issue(la(0));
            db.issue(lb(0));
        }
        for (int k = 0; k < full; ++k) {
            loads_landed<0>();
            meet_waves();
            if (k + 1 < full) {
                da.issue(la((k + 1) & 1));
                db.issue(lb((k + 1) & 1));
            }
            multiply(la(k & 1), lb(k & 1));
        }
        if (r0 + (int64_t)full * kBR < r1) {
            const int64_t r = r0 + (int64_t)full * kBR;
            stage_tail<BP, TA, T>(la(full & 1), d.a, d.lda, p0, d.P, r, r1);
            stage_tail<BQ, TB, T>(lb(full & 1), d.b, d.ldb, q0, d.Q, r, r1);
            __syncthreads();
            multiply(la(full & 1), lb(full & 1));
        }
    } else {
        Stage<BP, TA, T> sa;
        Stage<BQ, TB, T> sb;
        if (r0 < r1) {
            sa.load(d.a, d.lda, p0, d.P, r0, r1);
            sb.load(d.b, d.ldb, q0, d.Q, r0, r1);
        }
        for (int64_t r = r0; r < r1; r += kBR) {
            __syncthreads();
            sa.store(la(0));
            sb.store(lb(0));
            __syncthreads();
            if (r + kBR < r1) {
                sa.load(d.a, d.lda, p0, d.P, r + kBR, r1);
                sb.load(d.b, d.ldb, q0, d.Q, r + kBR, r1);
            }
            multiply(la(0), lb(0));
        }
    }

    // Epilogue through LDS, a run of kRows of each wave's rows at a time, so that a
    // lane gets eight consecutive columns and a wave stores whole 128-byte lines.
    // Each wave has its own part: 16-byte units, unit u of row o at u ^ (o & 15).
    constexpr int kCols = 16 * FQ;
    constexpr int kFit = (int)(sizeof(lds) / sizeof(float)) / (NWP * NWQ * kCols) / 16 * 16;
    constexpr int kRows = kFit < 16 * FP ? kFit : 16 * FP, kRun = kRows / 16;
    static_assert(kRun >= 1 && FP % kRun == 0, "the runs cover a wave's rows");
    static_assert(kCols % 64 == 0, "units are permuted within 64 columns");
    const uint64_t off = d.drop.thr ? drop_offset(d.drop) : 0;
    float* const mine = reinterpret_cast<float*>(lds) + wave * kRows * kCols;
    meet_waves();
#pragma unroll
    for (int i0 = 0; i0 < FP; i0 += kRun) {
#pragma unroll
        for (int i = 0; i < kRun; ++i)
#pragma unroll
            for (int j = 0; j < FQ; ++j) {
                const int o = 16 * i + (lane & 15), u = 4 * j + (lane >> 4);
                *reinterpret_cast<v4f*>(mine + o * kCols + 4 * (u ^ (o & 15))) = acc[i0 + i][j];
            }
        constexpr int kGroups = kCols / 8;
#pragma unroll 1
        for (int at = lane; at < kRows * kGroups; at += 64) {
            const int o = at / kGroups, c = at % kGroups;
            const v4f lo = *reinterpret_cast<const v4f*>(mine + o * kCols + 4 * ((2 * c) ^ (o & 15)));
            const v4f hi = *reinterpret_cast<const v4f*>(mine + o * kCols + 4 * ((2 * c + 1) ^ (o & 15)));
            float v[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
            const int64_t p = p0 + wp + 16 * i0 + o, q = q0 + wq + 8 * c;
            if (p >= d.P || q >= d.Q) continue;
            const int n = d.Q - q < 8 ? (int)(d.Q - q) : 8;
            if (g.part) store8_f(g.part + ((int64_t)blockIdx.y * d.P + p) * g.ld_part + q, v, 8);
            else epilogue8<EPI>(d, off, p, q, v, n);
        }
    }
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

template <int NWP, int NWQ, int FP, int FQ, bool TA, bool TB, int EPI, bool DIRECT>
static hipError_t tiles_launch(const ProductArgs& g, hipStream_t st) {
    constexpr int BP = 16 * FP * NWP, BQ = 16 * FQ * NWQ;
    const int64_t tiles = ((g.d.P + BP - 1) / BP) * ((g.d.Q + BQ - 1) / BQ);
    if (tiles > INT32_MAX) return hipErrorInvalidValue;
    hipLaunchKernelGGL((k_product<NWP, NWQ, FP, FQ, TA, TB, EPI, DIRECT>), dim3((unsigned)tiles, (unsigned)g.splits),
                       dim3(64 * NWP * NWQ), 0, st, g);
    return hipGetLastError();
}

template <bool TA, bool TB, int EPI>
static hipError_t product(ProductArgs& g, hipStream_t st) {
    const ProductDesc& d = g.d;
    if (d.P <= 0 || d.Q <= 0) return hipSuccess;
    const bool direct = direct_ok(d.a, d.lda, TA ? d.R : d.P) && direct_ok(d.b, d.ldb, TB ? d.R : d.Q);
    const int64_t big = ((d.P + 255) / 256) * ((d.Q + 255) / 256);
    hipError_t e = !direct ? tiles_launch<2, 2, 4, 4, TA, TB, EPI, false>(g, st)
                   : big >= 256 ? tiles_launch<2, 4, 8, 4, TA, TB, EPI, true>(g, st)
                                : tiles_launch<2, 2, 4, 4, TA, TB, EPI, true>(g, st);
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
