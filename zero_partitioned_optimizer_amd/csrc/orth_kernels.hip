// orth_kernels.hip -- orthogonalisation of whole matrices by Newton-Schulz products:
//   X = x / (|x| + eps);  X <- a X + (b A + c A A) X, A = X X^T, `steps` times;  o = scale X
// with A on the smaller side: a matrix that is taller than wide takes A = X^T X and
// X <- a X + X (b A + c A A) instead, so that nothing is transposed in memory.
//
// A step is three products on the matrix cores: the Gram product A, whose two triangles
// are equal, the square's, likewise, and the update's. Their operands are fp16, their sums
// fp32. What is rounded to 16 bits, and what is not:
//   X        kept as two fp16 numbers, hi + lo / 2048, about 22 bits; hi is the operand. The
//            update adds a X from both. A step multiplies directions that X does not hold
//            by a, 485 times in five steps: rounding noise of X in both its missing rows
//            and columns grows by that (X in fp16 alone leaves a rank-8 matrix 4% off, in
//            bf16 33%), while the noise of an operand lies in rows or columns that X holds.
//   A        off its diagonal. The diagonal, near 1 once X is nearly orthogonal and then
//            most of A, stays in fp32, in a vector.
//   b A + c A A   likewise. Its diagonal multiplies hi and lo in the last three steps, hi alone
//            before: with lo it is closer where it is most of the product, but puts a little
//            of hi's noise where X holds nothing, which later steps grow.
// What that leaves, against the formula in 64 bits and before o is rounded (which is 1.7e-3),
// on a CPU model of these roundings: 0.5 to 1e-3 of the result's norm for normal numbers,
// rank 1, rank 4 and falling spectra at 32 x 32 to 512 x 2048 (up to 1.6e-3 there, 2.5e-3
// at 8 x 8); with the diagonals in fp16 1.0 to 2.4e-3; with lo in every step 0.4 to 1.0e-3 on
// normal numbers but 4e-3 on rank 1 at 64 x 256, in none 1.1 to 1.6e-3 on normal numbers.
// fp16 holds X, A and b A + c A A times 1024: a 4096 x 11008 X starts with elements of 1.5e-4,
// and none of the three has elements above 10 with the default coefficients.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "layer_device.h"
#include "muon_internal.h"

namespace zk {

typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef short s4 __attribute__((ext_vector_type(4)));
typedef int v4i __attribute__((ext_vector_type(4)));

constexpr int kBR = 64;                     // reduction elements per staged tile
constexpr int kSide = 128;                  // all sides are padded to this, with zeros
constexpr float kScale = 1024.0f, kLow = 2048.0f;
constexpr int kSquareParts = 256;           // partial sums of squares of a matrix, at most

enum OrthOp { kGram, kSquare, kUpdate };

// C[p, q] = sum_r A(p, r) B(q, r) for each matrix of a group.
struct OrthArgs {
    const _Float16* a;
    const _Float16* b;
    int64_t lda, ldb, step_a, step_b;       // row lengths, and from one matrix to the next
    int64_t P, Q;                           // multiples of kSide
    int32_t turns;                          // reduction tiles of kBR
    int32_t np, nq, tiles, all;             // output tiles: down, across, of a matrix, of all
    const _Float16* in;                     // square: A, update: X hi; of C's shape
    int64_t ld_in, step_in;
    const float* diag_in;                   // square: of A, update: of b A + c A A
    _Float16* out;                          // update: X hi of the next step, or nullptr after the last
    int64_t ld_out, step_out;
    float* diag_out;
    int64_t step_diag;
    _Float16* lo;                           // update: X lo, in place, laid out as `in`
    float ca, cb, cc;
    float low;                              // update: what of lo the diagonal meets, 1 / kLow or 0
    bool by_column;                         // update: the diagonal goes by column
    uint16_t* o;                            // the last update's output and its size
    int64_t ld_o, step_o, rows, cols;
    float scale;
};

// ---------------------------------------------------------------------------
// tiles in LDS
// ---------------------------------------------------------------------------

// A staged tile has 128 outer indices and kBR reduction elements in chunks of eight (16
// bytes), permuted so that lanes that read together meet different banks: with the outer
// index in rows chunk c of row o lies at c ^ (o & 7); with the reduction in rows (T), chunk
// c of row r at c ^ perm(r), as a transposing read takes 4 rows x 32 bytes per 16 lanes,
// two such groups 8 rows apart.
__device__ __forceinline__ int perm_rows(int r) { return (r & 3) << 1 | (r >> 3 & 1) << 3; }

typedef __attribute__((address_space(3))) const _Float16 lds_f16;
typedef __attribute__((address_space(3))) const h8 lds_h8;
typedef __attribute__((address_space(3))) s4 lds_s4;
__device__ __forceinline__ uint32_t lds_address(const _Float16* p) {
    return (uint32_t)reinterpret_cast<uintptr_t>((lds_f16*)p);
}

// Two loads of 16 bytes a lane from the buffer's bytes at0, at1 to LDS, lane l of the wave
// to byte 16 l behind `to` and `to` + STEP. In assembly because the compiler, which sees in
// its own builtin a store to LDS of unknown extent, waits for it before the next LDS read of
// any tile. It has no output register; what reads the tile waits with loads_landed first.
// The descriptor comes from v_readfirstlane, and a scalar register that a vector instruction
// wrote takes five wait states until a memory instruction may read it, which the compiler
// does not see to inside assembly: the first load's move and four of s_nop are those five.
// m0 itself needs one.
template <int STEP>
__device__ __forceinline__ void lds_loads(v4i rsrc, uint32_t at0, uint32_t at1, uint32_t to) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 3\n\tbuffer_load_dwordx4 %3, %1, 0 offen lds\n\t"
                 "s_add_u32 m0, %0, %2\n\ts_nop 0\n\tbuffer_load_dwordx4 %4, %1, 0 offen lds"
                 :
                 : "s"(to), "s"(rsrc), "n"(STEP), "v"(at0), "v"(at1)
                 : "memory", "m0", "scc");
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

// PARTS runs of 128 outer indices from memory to LDS, a thread's chunks at byte offsets
// from `base` that every tile of the reduction shares. A run that lies outside the operand
// reads its last one instead, which reaches no output.
template <bool T, int THREADS, int PARTS>
struct Loader {
    static constexpr int kLoads = kSide * kBR / 8 / THREADS;
    static_assert(kLoads % 2 == 0, "pairs of loads");
    uint32_t at[PARTS][kLoads];
    const char* base;
    int64_t step;
    __device__ __forceinline__ void init(const _Float16* src, int64_t ld, int64_t o0, int64_t O) {
#pragma unroll
        for (int h = 0; h < PARTS; ++h) {
            const int64_t run = o0 + kSide * h < O ? kSide * h : O - kSide - o0;
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                const int id = threadIdx.x + i * THREADS;
                if constexpr (T) {
                    const int r = id / (kSide / 8), c = 8 * ((id % (kSide / 8)) ^ perm_rows(r));
                    at[h][i] = (uint32_t)((r * ld + run + c) * 2);
                } else {
                    const int o = id / (kBR / 8), c = 8 * ((id % (kBR / 8)) ^ (o & 7));
                    at[h][i] = (uint32_t)(((run + o) * ld + c) * 2);
                }
            }
        }
        base = reinterpret_cast<const char*>(src + (T ? o0 : o0 * ld));
        step = (T ? kBR * ld : kBR) * 2;
    }
    // Run h of the tile at `from` to LDS byte address `tile`; `wave` is the same in all
    // lanes. With `records` 0 the buffer's range check stops the loads (which still count).
    __device__ __forceinline__ void issue(int h, const char* from, uint32_t tile, int wave, int records) const {
        const uintptr_t b = reinterpret_cast<uintptr_t>(from);
        const v4i rsrc = {__builtin_amdgcn_readfirstlane((int)(uint32_t)b),
                          __builtin_amdgcn_readfirstlane((int)(uint32_t)(b >> 32)), records, 0x00020000};
#pragma unroll
        for (int i = 0; i < kLoads; i += 2)
            lds_loads<16 * THREADS>(rsrc, at[h][i], at[h][i + 1], tile + 16 * 64 * wave + 16 * THREADS * i);
    }
};
constexpr int kAllRecords = 0x7FFFFFFF;

// The matrix instruction's operands: for block i, lane l holds outer index o0 + 16 i + (l & 15)
// and reduction elements 32 s + 8 (l >> 4) .. + 7. o0 is a multiple of 32.
template <bool T>
struct Fragments {
    uint32_t at;
    __device__ __forceinline__ explicit Fragments(int o0) {
        const int lane = threadIdx.x & 63, i = lane & 15, g = lane >> 4;
        if constexpr (T) {
            const int r = 8 * g + (i >> 2), chunk = (o0 >> 3) + ((i & 3) >> 1);
            at = 2 * (r * kSide + 8 * (chunk ^ perm_rows(r)) + 4 * (i & 1));
        } else {
            const int o = o0 + i;
            at = 2 * (o * kBR + 8 * (g ^ (o & 7)));
        }
    }
    __device__ __forceinline__ h8 get(uint32_t tile, int i, int s) const {
        if constexpr (T) {
            // rows 32 further on have the same permutation
            const uint32_t p = tile + (at ^ (32u * i)) + 2 * 32 * kSide * s;
            const s4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4*)p);
            const s4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4*)(p + 2 * 4 * kSide));
            return __builtin_bit_cast(h8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
        } else {
            return *(lds_h8*)(tile + (at ^ (64u * s)) + 2 * 16 * kBR * i);
        }
    }
};

// Workgroup `id` of `all` goes to XCD id % 8, each with an L2 of its own: each XCD gets a run
// of consecutive tiles.
__device__ __forceinline__ int in_turn(int all) {
    const int id = blockIdx.x, xcd = id & 7, each = all >> 3, more = all & 7;
    return xcd * each + (xcd < more ? xcd : more) + (id >> 3);
}
// The matrix and the tile of a workgroup: of a symmetric product those on and below the
// diagonal, row by row, else down blocks of eight rows of tiles, column by column, so that
// the tiles that run at a time share operand rows.
template <bool SYM>
__device__ __forceinline__ int place(const OrthArgs& g, int* tp, int* tq) {
    const int t = in_turn(g.all), m = t / g.tiles, in = t - m * g.tiles;
    int p, q;
    if constexpr (SYM) {
        p = (int)((__builtin_sqrtf(8.0f * (float)in + 1.0f) - 1.0f) * 0.5f);
        while (p * (p + 1) / 2 > in) --p;
        while ((p + 1) * (p + 2) / 2 <= in) ++p;
        q = in - p * (p + 1) / 2;
    } else {
        const int block = in / (8 * g.nq), left = in - block * 8 * g.nq;
        const int rows = g.np - 8 * block < 8 ? g.np - 8 * block : 8;
        q = left / rows;
        p = 8 * block + left - q * rows;
    }
    // the same in all lanes, which the divisions hide from the compiler
    *tp = __builtin_amdgcn_readfirstlane(p);
    *tq = __builtin_amdgcn_readfirstlane(q);
    return __builtin_amdgcn_readfirstlane(m);
}

// ---------------------------------------------------------------------------
// epilogues
// ---------------------------------------------------------------------------

__device__ __forceinline__ void put_h8(_Float16* p, const float v[8]) {
    h8 t;
#pragma unroll
    for (int k = 0; k < 8; ++k) t[k] = (_Float16)v[k];
    *reinterpret_cast<h8*>(p) = t;
}

// Columns q .. q + 7 of row p of matrix m, from their sums v.
template <int OP>
__device__ __forceinline__ void epilogue8(const OrthArgs& g, int64_t m, int64_t p, int64_t q, float v[8]) {
    constexpr float kOnce = 1.0f / kScale, kTwice = kOnce * kOnce;
    if constexpr (OP == kGram) {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            if (p == q + k) {
                g.diag_out[m * g.step_diag + p] = v[k] * kTwice;
                v[k] = 0.0f;
            }
            v[k] *= kOnce;
        }
        put_h8(g.out + m * g.step_out + p * g.ld_out + q, v);
    } else if constexpr (OP == kSquare) {
        // A = D + F, its diagonal and the rest: A A = F F + D F + F D + D D
        const h8 f = *reinterpret_cast<const h8*>(g.in + m * g.step_in + p * g.ld_in + q);
        const float* const d = g.diag_in + m * g.step_diag;
        const float dp = d[p];
        float dq[8];
        load8_f(dq, d + q, 8);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float fk = (float)f[k], ff = v[k] * kOnce;
            v[k] = fmaf(g.cc, fmaf(dp + dq[k], fk, ff), g.cb * fk);
            if (p == q + k) {
                g.diag_out[m * g.step_diag + p] = fmaf(g.cc, fmaf(dp, dp, ff * kOnce), g.cb * dp);
                v[k] = 0.0f;
            }
        }
        put_h8(g.out + m * g.step_out + p * g.ld_out + q, v);
    } else {
        const int64_t at = m * g.step_in + p * g.ld_in + q;
        const h8 hi = *reinterpret_cast<const h8*>(g.in + at), lo = *reinterpret_cast<const h8*>(g.lo + at);
        const float* const e = g.diag_in + m * g.step_diag;
        float eq[8];
        if (g.by_column) load8_f(eq, e + q, 8);
        const float ep = e[g.by_column ? 0 : p];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float h = (float)hi[k], l = (float)lo[k];
            v[k] = fmaf(g.ca, fmaf(l, 1.0f / kLow, h), fmaf(g.by_column ? eq[k] : ep, fmaf(l, g.low, h), v[k] * kOnce));
        }
        if (g.out) {
            h8 h, l;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                h[k] = (_Float16)v[k];
                l[k] = (_Float16)((v[k] - (float)h[k]) * kLow);
            }
            *reinterpret_cast<h8*>(g.out + at) = h;
            *reinterpret_cast<h8*>(g.lo + at) = l;
        } else if (p < g.rows && q < g.cols) {
            const int n = g.cols - q < 8 ? (int)(g.cols - q) : 8;
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] *= g.scale * kOnce;
            store8_bf(g.o + m * g.step_o + p * g.ld_o + q, v, n);
        }
    }
}

// A wave's blocks, (FP 16) x 64 outputs, through its 16 KB of LDS, 64 rows at a time, so that
// a lane has eight consecutive columns. Blocks are computed as (q, p): a lane holds four
// consecutive columns of a row, a 16-byte unit, unit u of row o at u ^ (o & 15). Below the
// diagonal of a symmetric product the same outputs go to their mirrored places too, eight
// consecutive rows to a lane.
template <int OP, int FP, typename Row, typename Col>
__device__ __forceinline__ void finish(const OrthArgs& g, int64_t m, const v4f (&acc)[FP][4], float* mine, bool mirror,
                                       Row row_of, Col col_of) {
    const int lane = threadIdx.x & 63, c = lane & 7;
#pragma unroll
    for (int i0 = 0; i0 < FP; i0 += 4) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int o = 16 * i + (lane & 15), u = 4 * j + (lane >> 4);
                *reinterpret_cast<v4f*>(mine + 64 * o + 4 * (u ^ (o & 15))) = acc[i0 + i][j];
            }
        const int64_t p0 = row_of(i0), q = col_of(c >> 1) + 8 * (c & 1);
        if (p0 < g.P && q < g.Q) {
#pragma unroll 2
            for (int o = lane >> 3; o < 64; o += 8) {
                const v4f lo = *reinterpret_cast<const v4f*>(mine + 64 * o + 4 * ((2 * c) ^ (o & 15)));
                const v4f hi = *reinterpret_cast<const v4f*>(mine + 64 * o + 4 * ((2 * c + 1) ^ (o & 15)));
                float v[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
                epilogue8<OP>(g, m, p0 + o, q, v);
            }
        }
        if (OP != kUpdate && mirror && p0 < g.P) {
#pragma unroll 2
            for (int j = lane >> 3; j < 64; j += 8) {
                const int64_t row = col_of(j >> 4) + (j & 15);
                if (row >= g.Q) continue;
                float v[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const int o = 8 * c + k;
                    v[k] = mine[64 * o + 4 * ((j >> 2) ^ (o & 15)) + (j & 3)];
                }
                epilogue8<OP>(g, m, row, p0 + 8 * c, v);
            }
        }
    }
}

// ---------------------------------------------------------------------------
// products
// ---------------------------------------------------------------------------

__device__ __forceinline__ v4f mul(h8 a, h8 b, v4f c) { return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0); }

// 128 x 128 outputs by four waves, 64 x 64 each; two tiles of the reduction in LDS, the next
// one loading while one is multiplied. Two workgroups fit a compute unit.
template <int OP, bool TA, bool TB>
__global__ void __launch_bounds__(256, 2) k_orth(const OrthArgs g) {
    constexpr bool SYM = OP != kUpdate;
    constexpr int kTile = kSide * kBR;
    __shared__ __attribute__((aligned(16))) _Float16 lds[4 * kTile];
    int tp, tq;
    const int64_t m = place<SYM>(g, &tp, &tq), p0 = (int64_t)tp * kSide, q0 = (int64_t)tq * kSide;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wp = (wave >> 1) * 64, wq = (wave & 1) * 64;
    v4f acc[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    const Fragments<TA> ga(wp);
    const Fragments<TB> gb(wq);
    const uint32_t base = lds_address(lds);
    Loader<TA, 256, 1> la;
    Loader<TB, 256, 1> lb;
    la.init(g.a + m * g.step_a, g.lda, p0, g.P);
    lb.init(g.b + m * g.step_b, g.ldb, q0, g.Q);
    la.issue(0, la.base, base, wave, kAllRecords);
    lb.issue(0, lb.base, base + 2 * kTile, wave, kAllRecords);
#pragma unroll 1
    for (int k = 0; k < g.turns; ++k) {
        loads_landed<0>();
        meet_waves();
        const uint32_t tile = base + 4 * kTile * (k & 1), next = base + 4 * kTile * ((k + 1) & 1);
        if (k + 1 < g.turns) {
            la.issue(0, la.base += la.step, next, wave, kAllRecords);
            lb.issue(0, lb.base += lb.step, next + 2 * kTile, wave, kAllRecords);
        }
#pragma unroll
        for (int s = 0; s < kBR / 32; ++s) {
            h8 fa[4], fb[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) fa[i] = ga.get(tile, i, s);
#pragma unroll
            for (int j = 0; j < 4; ++j) fb[j] = gb.get(tile + 2 * kTile, j, s);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = mul(fb[j], fa[i], acc[i][j]);
        }
    }
    meet_waves();
    finish<OP, 4>(g, m, acc, reinterpret_cast<float*>(lds) + wave * 64 * 64, tp != tq, [&](int i) { return p0 + wp + 16 * i; },
                  [&](int j) { return q0 + wq + 16 * j; });
}

// ---------------------------------------------------------------------------
// before the first step
// ---------------------------------------------------------------------------

struct StartArgs {
    const void* x;
    int64_t ld_x, step_x, rows, cols;
    int64_t Rp, Cp;
    _Float16* hi;
    _Float16* lo;
    double* parts;                  // [matrix][kSquareParts]
    int32_t n_parts;
    double eps;
};

__device__ __forceinline__ double block_sum(double v) {
    __shared__ double s[4];
#pragma unroll
    for (int k = 32; k > 0; k >>= 1) v += __shfl_xor(v, k);
    if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
    __syncthreads();
    return (s[0] + s[1]) + (s[2] + s[3]);
}
template <bool XF>
__device__ __forceinline__ void load_x8(float v[8], const StartArgs& g, int64_t m, int64_t row, int64_t j) {
    const int n = row >= g.rows || j >= g.cols ? 0 : g.cols - j < 8 ? (int)(g.cols - j) : 8;
    const int64_t at = m * g.step_x + row * g.ld_x + j;
    if constexpr (XF) load8_f(v, static_cast<const float*>(g.x) + at, n);
    else load8_bf(v, static_cast<const uint16_t*>(g.x) + at, n);
}
// Row and chunk `c` of eight columns of a matrix's chunk `id`, by a reciprocal that is then
// corrected (ids stay below 2^51).
__device__ __forceinline__ int64_t row_of_chunk(int64_t id, int64_t chunks, double inv, int64_t* c) {
    int64_t row = (int64_t)((double)id * inv);
    if (row * chunks > id) --row;
    else if ((row + 1) * chunks <= id) ++row;
    *c = id - row * chunks;
    return row;
}

// Sums of squares in 64 bits (no scale overflows them), a workgroup's each to its place.
template <bool XF>
__global__ void __launch_bounds__(256) k_orth_squares(const StartArgs g) {
    const int64_t m = blockIdx.y, chunks = (g.cols + 7) / 8, all = g.rows * chunks;
    const double inv = 1.0 / (double)chunks;
    double sum = 0.0;
#pragma unroll 4
    for (int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x; id < all; id += (int64_t)g.n_parts * 256) {
        int64_t c;
        const int64_t row = row_of_chunk(id, chunks, inv, &c);
        float v[8];
        load_x8<XF>(v, g, m, row, 8 * c);
#pragma unroll
        for (int k = 0; k < 8; ++k) sum = fma((double)v[k], (double)v[k], sum);
    }
    sum = block_sum(sum);
    if (threadIdx.x == 0) g.parts[m * kSquareParts + blockIdx.x] = sum;
}

// X hi and lo with their padding. A norm that is not finite makes all of them NaN.
template <bool XF>
__global__ void __launch_bounds__(256) k_orth_start(const StartArgs g) {
    const int64_t m = blockIdx.y, chunks = g.Cp / 8, all = g.Rp * chunks;
    const double square = block_sum((int)threadIdx.x < g.n_parts ? g.parts[m * kSquareParts + threadIdx.x] : 0.0);
    const double norm = sqrt(square), inv = 1.0 / (double)chunks;
    const double by = norm < INFINITY ? (double)kScale / (norm + g.eps) : (double)NAN;
#pragma unroll 2
    for (int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x; id < all; id += (int64_t)gridDim.x * 256) {
        int64_t c;
        const int64_t row = row_of_chunk(id, chunks, inv, &c);
        float v[8];
        load_x8<XF>(v, g, m, row, 8 * c);
        h8 h, l;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float x = (float)((double)v[k] * by);
            h[k] = (_Float16)x;
            l[k] = (_Float16)((x - (float)h[k]) * kLow);
        }
        const int64_t at = m * g.Rp * g.Cp + row * g.Cp + 8 * c;
        *reinterpret_cast<h8*>(g.hi + at) = h;
        *reinterpret_cast<h8*>(g.lo + at) = l;
    }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

static int64_t padded(int64_t n) { return (n + kSide - 1) / kSide * kSide; }

// What a group of matrices has in the workspace, in this order: X hi twice and lo, A and
// b A + c A A, their diagonals, the partial sums of squares.
struct OrthShape {
    int64_t Rp, Cp, m;              // padded sides, the smaller one
    int64_t x, a;                   // elements
    size_t each;                    // bytes of a matrix
    int64_t group;                  // matrices at a time
};
static OrthShape shape_of(int64_t batch, int64_t rows, int64_t cols) {
    OrthShape s{};
    s.Rp = padded(rows);
    s.Cp = padded(cols);
    s.m = s.Rp < s.Cp ? s.Rp : s.Cp;
    s.x = s.Rp * s.Cp;
    s.a = s.m * s.m;
    s.each = (size_t)(6 * s.x + 4 * s.a + 8 * s.m) + kSquareParts * sizeof(double);
    const int64_t most = (int64_t)((size_t(4) << 30) / s.each);
    s.group = most < 1 ? 1 : most > 16384 ? 16384 : most;
    if (s.group > batch) s.group = batch;
    return s;
}

size_t orth_ws_bytes(int64_t batch, int64_t rows, int64_t cols) {
    if (batch < 1 || rows < 1 || cols < 1) return 0;
    const OrthShape s = shape_of(batch, rows, cols);
    return (size_t)s.group * s.each;
}

template <int OP, bool TA, bool TB>
static hipError_t product(OrthArgs g, int64_t n, hipStream_t st) {
    g.np = (int32_t)(g.P / kSide);
    g.nq = (int32_t)(g.Q / kSide);
    g.tiles = OP == kUpdate ? g.np * g.nq : g.np * (g.np + 1) / 2;
    // as many matrices to a launch as its 2^31 threads hold
    const int64_t most = (int64_t(1) << 23) / g.tiles, first_launch = most < 1 ? 1 : most;
    for (int64_t done = 0; done < n; done += first_launch) {
        const int64_t some = n - done < first_launch ? n - done : first_launch;
        g.all = (int32_t)(g.tiles * some);
        hipLaunchKernelGGL((k_orth<OP, TA, TB>), dim3((unsigned)g.all), dim3(256), 0, st, g);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        g.a += some * g.step_a;
        g.b += some * g.step_b;
        if (g.in) g.in += some * g.step_in;
        if (g.lo) g.lo += some * g.step_in;
        if (g.out) g.out += some * g.step_out;
        if (g.diag_in) g.diag_in += some * g.step_diag;
        if (g.diag_out) g.diag_out += some * g.step_diag;
        if (g.o) g.o += some * g.step_o;
    }
    return hipSuccess;
}

static hipError_t orthogonalize(const OrthDesc& d, const OrthShape& s, int64_t first, int64_t n, hipStream_t st) {
    const int64_t x_all = s.group * s.x, a_all = s.group * s.a;
    _Float16* hi[2] = {static_cast<_Float16*>(d.ws), static_cast<_Float16*>(d.ws) + x_all};
    _Float16* const lo = hi[1] + x_all;
    _Float16* const A = lo + x_all;
    _Float16* const B = A + a_all;
    float* const da = reinterpret_cast<float*>(B + a_all);
    float* const db = da + s.group * s.m;
    double* const parts = reinterpret_cast<double*>(db + s.group * s.m);
    const bool tall = d.rows > d.cols;

    StartArgs b{};
    const int64_t skip = first * d.stride_x;
    b.x = d.x_f32 ? static_cast<const void*>(static_cast<const float*>(d.x) + skip)
                  : static_cast<const void*>(static_cast<const uint16_t*>(d.x) + skip);
    b.ld_x = d.ld_x;
    b.step_x = d.stride_x;
    b.rows = d.rows;
    b.cols = d.cols;
    b.Rp = s.Rp;
    b.Cp = s.Cp;
    b.hi = hi[0];
    b.lo = lo;
    b.parts = parts;
    b.eps = d.eps;
    const int64_t chunks = (d.rows * ((d.cols + 7) / 8) + 1023) / 1024, whole = (s.x / 8 + 511) / 512;
    b.n_parts = (int32_t)(chunks < kSquareParts ? chunks : kSquareParts);
    const unsigned blocks = (unsigned)(whole < 2048 ? whole : 2048);
    hipLaunchKernelGGL(d.x_f32 ? k_orth_squares<true> : k_orth_squares<false>, dim3((unsigned)b.n_parts, (unsigned)n),
                       dim3(256), 0, st, b);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(d.x_f32 ? k_orth_start<true> : k_orth_start<false>, dim3(blocks, (unsigned)n), dim3(256), 0, st, b);
    if ((e = hipGetLastError()) != hipSuccess) return e;

    for (int k = 0; k < d.steps; ++k) {
        const _Float16* const X = hi[k & 1];
        OrthArgs g{};
        g.ca = (float)d.coefficients[3 * k];
        g.cb = (float)d.coefficients[3 * k + 1];
        g.cc = (float)d.coefficients[3 * k + 2];
        g.step_diag = s.m;
        // A
        OrthArgs p = g;
        p.a = p.b = X;
        p.lda = p.ldb = s.Cp;
        p.step_a = p.step_b = s.x;
        p.P = p.Q = s.m;
        p.turns = (int32_t)((tall ? s.Rp : s.Cp) / kBR);
        p.out = A;
        p.ld_out = s.m;
        p.step_out = s.a;
        p.diag_out = da;
        e = tall ? product<kGram, true, true>(p, n, st) : product<kGram, false, false>(p, n, st);
        if (e != hipSuccess) return e;
        // b A + c A A
        p = g;
        p.a = p.b = p.in = A;
        p.lda = p.ldb = p.ld_in = p.ld_out = s.m;
        p.step_a = p.step_b = p.step_in = p.step_out = s.a;
        p.P = p.Q = s.m;
        p.turns = (int32_t)(s.m / kBR);
        p.diag_in = da;
        p.out = B;
        p.diag_out = db;
        if ((e = product<kSquare, false, false>(p, n, st)) != hipSuccess) return e;
        // X; b A + c A A is symmetric, and so an operand with its outer index in rows on either side
        p = g;
        p.a = tall ? X : B;
        p.b = tall ? B : X;
        p.lda = tall ? s.Cp : s.m;
        p.ldb = tall ? s.m : s.Cp;
        p.step_a = tall ? s.x : s.a;
        p.step_b = tall ? s.a : s.x;
        p.P = s.Rp;
        p.Q = s.Cp;
        p.turns = (int32_t)(s.m / kBR);
        p.in = X;
        p.ld_in = p.ld_out = s.Cp;
        p.step_in = p.step_out = s.x;
        p.lo = lo;
        p.diag_in = db;
        p.by_column = tall;
        p.low = d.steps - 1 - k <= 2 ? 1.0f / kLow : 0.0f;
        if (k + 1 < d.steps) {
            p.out = hi[(k + 1) & 1];
        } else {
            p.o = d.o + first * d.stride_o;
            p.ld_o = d.ld_o;
            p.step_o = d.stride_o;
            p.rows = d.rows;
            p.cols = d.cols;
            p.scale = d.scale;
        }
        e = tall ? product<kUpdate, false, false>(p, n, st) : product<kUpdate, false, true>(p, n, st);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

hipError_t launch_orthogonalize(const OrthDesc& d, hipStream_t st) {
    const OrthShape s = shape_of(d.batch, d.rows, d.cols);
    for (int64_t first = 0; first < d.batch; first += s.group) {
        const int64_t n = d.batch - first < s.group ? d.batch - first : s.group;
        const hipError_t e = orthogonalize(d, s, first, n, st);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace zk
