// orth_kernels.hip -- orthogonalisation of whole matrices by Newton-Schulz products:
//   X = x / (|x| + eps);  X <- a X + (b A + c A A) X, A = X X^T, `steps` times;  o = scale X
// with A on the smaller side: a matrix that is taller than wide takes A = X^T X and
// X <- a X + X (b A + c A A) instead, so that nothing is transposed in memory.
//
// A step is three products on the matrix cores: the Gram product A, whose two triangles
// are equal, the square's, likewise, and the update's, with fp32 sums. A step multiplies
// directions that X does not hold by a, 485 times in five steps, and any rounding puts some
// noise there: with operands and X in fp16 alone a rank-8 matrix comes out 4% off, in bf16
// 33%, and with fp16 operands and 18 bits of X one of 64 equal singular values 0.4%, where
// fp32 is 8e-6 off. So all of X, A and b A + c A A are pairs of fp16 numbers, hi the value
// rounded and lo what that leaves, rounded: 22 bits and a sign, 32 in all. A product of two pairs
// is three of fp16 operands into the same fp32 sums,
//   hi hi + hi lo + lo hi,
// and leaves out lo lo, 2^-22 of it at most. Of A and b A + c A A the diagonal, near 1 once X is
// nearly orthogonal and then most of them, is kept beside in fp32 and meets X in fp32.
// What that leaves, against the formula in 64 bits and before o is rounded (which is 1.7e-3 of
// the norm), on a CPU model of these roundings: 1e-6 for normal numbers, 1e-5 for rank 32 to
// 66, 2e-4 for rank 1, each up to 2.4 times what operations in fp32 leave. As it grows with
// each a, the product of the a's is bounded.
// fp16 holds A and b A + c A A times 1024 and X times 4096, of which a 4096 x 11008 one starts
// with elements of 1.5e-4; with the default coefficients no element of them passes 3. Below
// 6e-5 fp16's numbers are 6e-8 apart, so lo is known to 1.5e-11 of X's norm and 6e-11 of A's at
// the least.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "layer_device.h"
#include "muon_internal.h"
#include "orth_plan.h"
#include "tile_device.h"

namespace zk {

typedef _Float16 h8 __attribute__((ext_vector_type(8)));

constexpr float kScale = 1024.0f, kScaleX = 4096.0f;

enum OrthOp { kGram, kSquare, kUpdate, kUpdateTall };        // of a matrix that is taller than wide

// C[p, q] = sum_r A(p, r) B(q, r) for each matrix of a group, of pairs hi and lo.
struct OrthArgs {
    const _Float16* a;                      // hi
    const _Float16* b;
    int64_t low_a, low_b;                   // from an element's hi to its lo
    int64_t lda, ldb, step_a, step_b;       // row lengths, and from one matrix to the next
    int64_t P, Q;                           // multiples of kSide
    int32_t turns;                          // kTerms for each reduction tile of kBR
    int32_t np, nq, tiles;                  // output tiles: down, across, of a matrix
    int32_t first, all;                     // the launch's first one, of all matrices', and how many
    const _Float16* in;                     // square: A, update: X, hi; of C's shape
    int64_t low_in, ld_in, step_in;
    const float* diag_in;                   // square: of A, update: of b A + c A A
    _Float16* out;                          // update: X of the next step, or nullptr after the last
    int64_t low_out, ld_out, step_out;
    float* diag_out;
    int64_t step_diag;
    float ca, cb, cc;
    uint16_t* o;                            // the last update's output and its size
    int64_t ld_o, step_o, rows, cols;
    float scale;
    float* part;                            // split tiles' partial sums
};

// ---------------------------------------------------------------------------
// tiles in LDS
// ---------------------------------------------------------------------------

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

// PARTS runs of ROWS outer indices from memory to LDS, a thread's chunks at byte offsets
// from turn(k) that every turn shares; THREADS consecutive threads load a run. A run that
// lies outside the operand reads its last one instead, which reaches no output. Turns take
// a reduction tile's three terms one after another, operand A as hi, hi, lo and operand B (LOW
// 1) as hi, lo, hi: what a turn reads again is still in the caches.
template <int ROWS, bool T, int THREADS, int PARTS, int LOW>
struct Loader {
    static constexpr int kLoads = ROWS * kBR / 8 / THREADS;
    static_assert(kLoads % 2 == 0, "pairs of loads");
    uint32_t at[PARTS][kLoads];
    const char* base;
    int64_t step, low;
    __device__ __forceinline__ void init(const _Float16* src, int64_t to_low, int64_t ld, int64_t o0, int64_t O) {
#pragma unroll
        for (int h = 0; h < PARTS; ++h) {
            const int64_t run = o0 + ROWS * h < O ? ROWS * h : O - ROWS - o0;
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                const int id = threadIdx.x % THREADS + i * THREADS;
                if constexpr (T) {
                    const int r = id / (ROWS / 8), c = 8 * ((id % (ROWS / 8)) ^ perm_reduced<ROWS>(r));
                    at[h][i] = (uint32_t)((r * ld + run + c) * 2);
                } else {
                    const int o = id / (kBR / 8), c = 8 * ((id % (kBR / 8)) ^ (o & 7));
                    at[h][i] = (uint32_t)(((run + o) * ld + c) * 2);
                }
            }
        }
        base = reinterpret_cast<const char*>(src + (T ? o0 : o0 * ld));
        step = (T ? kBR * ld : kBR) * 2;
        low = to_low * 2;
    }
    __device__ __forceinline__ const char* turn(int k) const {
        const uint32_t tile = (uint32_t)k / kTerms, term = (uint32_t)k - kTerms * tile;
        return base + tile * step + (term == LOW ? low : 0);
    }
    // Run h of what lies at `from` to LDS byte address `tile`; `wave` (of those that load the
    // run) is the same in all lanes. `records`: kAllRecords, or 0 for no load.
    __device__ __forceinline__ void issue(int h, const char* from, uint32_t tile, int wave, int records) const {
        const v4i rsrc = descriptor(from, records);
#pragma unroll
        for (int i = 0; i < kLoads; i += 2)
            lds_loads<16 * THREADS>(rsrc, at[h][i], at[h][i + 1], tile + 16 * 64 * wave + 16 * THREADS * i);
    }
};
template <int ROWS, bool T, int THREADS, int PARTS>
using LoaderA = Loader<ROWS, T, THREADS, PARTS, 2>;
template <int ROWS, bool T, int THREADS, int PARTS>
using LoaderB = Loader<ROWS, T, THREADS, PARTS, 1>;

template <int ROWS, bool T>
using Fragments = TileFragments<ROWS, T, kBR, h8>;

// Workgroup `id` of `all` goes to XCD id % 8, each with an L2 of its own: each XCD gets a run
// of consecutive tiles.
__device__ __forceinline__ int in_turn(int all) {
    const int id = blockIdx.x, xcd = id & 7, each = all >> 3, more = all & 7;
    return xcd * each + (xcd < more ? xcd : more) + (id >> 3);
}
// The matrix and the place of tile t of all: of a symmetric product those on and below the
// diagonal, row by row, else down blocks of eight rows of tiles, column by column, so that
// the tiles that run at a time share operand rows.
template <bool SYM>
__device__ __forceinline__ int place(const OrthArgs& g, int t, int* tp, int* tq) {
    const int m = t / g.tiles, in = t - m * g.tiles;
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

// Eight values as pairs, lo `low` elements behind hi. A value beyond fp16's largest has an
// infinity in both, of either sign, so that what it reaches is NaN.
struct Pair8 {
    h8 hi, lo;
    __device__ __forceinline__ void load(const _Float16* p, int64_t low) {
        hi = *reinterpret_cast<const h8*>(p);
        lo = *reinterpret_cast<const h8*>(p + low);
    }
    __device__ __forceinline__ float get(int k) const { return (float)hi[k] + (float)lo[k]; }
};
__device__ __forceinline__ void put_pairs(_Float16* p, int64_t low, const float v[8]) {
    h8 hi, lo;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        hi[k] = (_Float16)v[k];
        lo[k] = (_Float16)(v[k] - (float)hi[k]);
    }
    *reinterpret_cast<h8*>(p) = hi;
    *reinterpret_cast<h8*>(p + low) = lo;
}

// What a product makes of its sums, for a lane's eight columns q + s .. q + s + 7 of matrix m (s:
// a run's distance from the first one): what the columns need is loaded once a run (columns),
// what a row needs ahead of its use (In, load), so that many rows' loads are under way.
template <int OP>
struct OrthEpilogue;

// A: F off the diagonal, the diagonal in fp32.
template <>
struct OrthEpilogue<kGram> {
    static constexpr float kOff = kScale / (kScaleX * kScaleX);
    struct In {};
    struct Columns {};
    const OrthArgs& g;
    _Float16* out;
    float* diag;
    const int64_t q;
    __device__ __forceinline__ OrthEpilogue(const OrthArgs& a, int64_t m, int64_t col)
        : g(a), out(a.out + m * a.step_out + col), diag(a.diag_out + m * a.step_diag), q(col) {}
    __device__ __forceinline__ void columns(Columns&, int) const {}
    __device__ __forceinline__ void load(In&, int64_t, int) const {}
    // v: in, the sums; out, what the matrix holds, here and, of a symmetric one, at the mirrored place
    __device__ __forceinline__ void put(const In&, const Columns&, int64_t p, int s, float v[8]) const {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            v[k] *= kOff;
            if (p == q + s + k) {
                diag[p] = v[k] * (1.0f / kScale);
                v[k] = 0.0f;
            }
        }
        put_pairs(out + p * g.ld_out + s, g.low_out, v);
    }
};

// b A + c A A, where A = D + F: A A = F F + D F + F D + D D.
template <>
struct OrthEpilogue<kSquare> {
    static constexpr float kOnce = 1.0f / kScale;
    struct In {
        Pair8 f;
        float d;
    };
    struct Columns {
        float d[8];
    };
    const OrthArgs& g;
    const _Float16* in;
    const float* from;
    _Float16* out;
    float* diag;
    const int64_t q;
    __device__ __forceinline__ OrthEpilogue(const OrthArgs& a, int64_t m, int64_t col)
        : g(a), in(a.in + m * a.step_in + col), from(a.diag_in + m * a.step_diag), out(a.out + m * a.step_out + col),
          diag(a.diag_out + m * a.step_diag), q(col) {}
    __device__ __forceinline__ void columns(Columns& c, int s) const { load8_f(c.d, from + q + s, 8); }
    __device__ __forceinline__ void load(In& r, int64_t p, int s) const {
        r.f.load(in + p * g.ld_in + s, g.low_in);
        r.d = from[p];
    }
    __device__ __forceinline__ void put(const In& r, const Columns& c, int64_t p, int s, float v[8]) const {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float f = r.f.get(k), ff = v[k] * kOnce;
            v[k] = fmaf(g.cc, fmaf(r.d + c.d[k], f, ff), g.cb * f);
            if (p == q + s + k) {
                diag[p] = fmaf(g.cc, fmaf(r.d, r.d, ff * kOnce), g.cb * r.d);
                v[k] = 0.0f;
            }
        }
        put_pairs(out + p * g.ld_out + s, g.low_out, v);
    }
};

// a X + (b A + c A A) X, the diagonal by row; or X on the left of it, by column.
template <bool TALL>
struct UpdateEpilogue {
    static constexpr float kOnce = 1.0f / kScale;
    struct In {
        Pair8 x;
        float d;
    };
    struct Columns {
        float d[8];
    };
    const OrthArgs& g;
    const int64_t at;
    const float* from;
    uint16_t* o;
    const int64_t q;
    __device__ __forceinline__ UpdateEpilogue(const OrthArgs& a, int64_t m, int64_t col)
        : g(a), at(m * a.step_in + col), from(a.diag_in + m * a.step_diag), o(a.o + m * a.step_o + col), q(col) {}
    __device__ __forceinline__ void columns(Columns& c, int s) const {
        if constexpr (TALL) load8_f(c.d, from + q + s, 8);
    }
    __device__ __forceinline__ void load(In& r, int64_t p, int s) const {
        r.x.load(g.in + at + p * g.ld_in + s, g.low_in);
        if constexpr (!TALL) r.d = from[p];
    }
    __device__ __forceinline__ void put(const In& r, const Columns& c, int64_t p, int s, float v[8]) const {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            v[k] = fmaf(g.ca + (TALL ? c.d[k] : r.d), r.x.get(k), v[k] * kOnce);
        }
        if (g.out) {
            put_pairs(g.out + at + p * g.ld_in + s, g.low_out, v);
        } else if (p < g.rows && q + s < g.cols) {
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] *= g.scale * (1.0f / kScaleX);
            store8_bf(o + p * g.ld_o + s, v, g.cols - q - s >= 8 ? 8 : (int)(g.cols - q - s));
        }
    }
};
template <>
struct OrthEpilogue<kUpdate> : UpdateEpilogue<false> {
    using UpdateEpilogue<false>::UpdateEpilogue;
};
template <>
struct OrthEpilogue<kUpdateTall> : UpdateEpilogue<true> {
    using UpdateEpilogue<true>::UpdateEpilogue;
};
constexpr bool symmetric(int op) { return op < kUpdate; }

// What lanes of a wave have written to LDS, other lanes of it may read: LDS operations of a wave
// are done in their order, and the compiler keeps them in it.
__device__ __forceinline__ void meet_lanes() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
    __builtin_amdgcn_wave_barrier();
}

// A wave's blocks, four times FQ at a time, through its part of LDS (64 rows of 16 FQ floats),
// so that a lane has eight consecutive columns, the same in all its rows of a run. Blocks are
// computed as (q, p): a lane holds four consecutive columns of a row, a 16-byte unit, unit u
// of row o at u ^ (o & mask). What a lane's rows need is asked for kAhead rows ahead, and (ask) of
// the first ones together: before the reduction by k_orth_mid, behind it by the others, which
// gain nothing from it or lose (12 updates of 768 x 2304 55 to 59 us). Below the diagonal of a
// symmetric product the results go back to LDS, and from there to their mirrored places,
// eight consecutive rows to a lane. row_of(i): first row of block i, an even one's before the
// next's; col_of(run): first of its columns.
template <int OP, int FQ, int RUNS, typename Row, typename Col>
struct Finish {
    static constexpr int kCols = 16 * FQ, kMask = 4 * FQ - 1, kGroups = 2 * FQ, kStep = 64 / kGroups, kRows = 64 / kStep;
    const OrthArgs& g;
    const int64_t m;
    const Row row_of;
    const Col col_of;
    const int lane, c, o0;
    const OrthEpilogue<OP> epi;
    // a run's rows, or half of them where all, beside two runs' sums, would not fit the registers
    static constexpr int kAhead = OP == kSquare && RUNS == 2 ? kRows / 2 : kRows;
    typename OrthEpilogue<OP>::In in[kAhead];

    __device__ __forceinline__ Finish(const OrthArgs& a, int64_t matrix, Row rows, Col cols)
        : g(a), m(matrix), row_of(rows), col_of(cols), lane(threadIdx.x & 63), c(lane % kGroups), o0(lane / kGroups),
          epi(a, m, cols(0) + 8 * c) {}
    __device__ __forceinline__ int64_t row(int o) const { return row_of(o >> 4) + (o & 15); }
    __device__ __forceinline__ int64_t column(int run) const { return col_of(run) + 8 * c; }
    __device__ __forceinline__ int shift(int run) const { return (int)(col_of(run) - col_of(0)); }
    // what row `at` of all runs' needs
    __device__ __forceinline__ void load(int at) {
        const int run = at / kRows;
        const int64_t p = row(o0 + kStep * (at % kRows));
        if (at < RUNS * kRows && column(run) < g.Q && p < g.P) epi.load(in[at % kAhead], p, shift(run));
    }
    __device__ __forceinline__ void ask() {
#pragma unroll
        for (int u = 0; u < kAhead; ++u) load(u);
    }
    __device__ __forceinline__ void operator()(const v4f (&acc)[4][FQ * RUNS], float* mine, bool mirror) {
        const int r = lane & 7;
#pragma unroll
        for (int run = 0; run < RUNS; ++run) {
            typename OrthEpilogue<OP>::Columns col;
            if (column(run) < g.Q) epi.columns(col, shift(run));
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < FQ; ++j) {
                    const int o = 16 * i + (lane & 15), u = 4 * j + (lane >> 4);
                    *reinterpret_cast<v4f*>(mine + kCols * o + 4 * (u ^ (o & kMask))) = acc[i][FQ * run + j];
                }
            meet_lanes();
#pragma unroll
            for (int u = 0; u < kRows; ++u) {
                const int o = o0 + kStep * u;
                v4f* const lo = reinterpret_cast<v4f*>(mine + kCols * o + 4 * ((2 * c) ^ (o & kMask)));
                v4f* const hi = reinterpret_cast<v4f*>(mine + kCols * o + 4 * ((2 * c + 1) ^ (o & kMask)));
                float v[8] = {(*lo)[0], (*lo)[1], (*lo)[2], (*lo)[3], (*hi)[0], (*hi)[1], (*hi)[2], (*hi)[3]};
                if (column(run) < g.Q && row(o) < g.P) epi.put(in[u % kAhead], col, row(o), shift(run), v);
                if (symmetric(OP) && mirror) {
                    *lo = v4f{v[0], v[1], v[2], v[3]};
                    *hi = v4f{v[4], v[5], v[6], v[7]};
                }
                load(run * kRows + u + kAhead);
            }
            if (symmetric(OP) && mirror) meet_lanes();
            if (symmetric(OP) && mirror && row(8 * r) < g.P) {
#pragma unroll 2
                for (int j = lane >> 3; j < kCols; j += 8) {
                    float v[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const int o = 8 * r + k;
                        v[k] = mine[kCols * o + 4 * ((j >> 2) ^ (o & kMask)) + (j & 3)];
                    }
                    const int64_t q = col_of(run) + j;
                    if (q < g.Q) put_pairs(g.out + m * g.step_out + q * g.ld_out + row(8 * r), g.low_out, v);
                }
            }
            if (run + 1 < RUNS) meet_lanes();
        }
    }
};
template <int OP, int FQ, int RUNS, typename Row, typename Col>
__device__ __forceinline__ Finish<OP, FQ, RUNS, Row, Col> finish(const OrthArgs& g, int64_t m, Row row_of, Col col_of) {
    return Finish<OP, FQ, RUNS, Row, Col>(g, m, row_of, col_of);
}

// ---------------------------------------------------------------------------
// products
// ---------------------------------------------------------------------------

__device__ __forceinline__ v4f mul(h8 a, h8 b, v4f c) { return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0); }
template <int FP, int FQ>
__device__ __forceinline__ void clear(v4f (&acc)[FP][FQ]) {
#pragma unroll
    for (int i = 0; i < FP; ++i)
#pragma unroll
        for (int j = 0; j < FQ; ++j) acc[i][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
}

// 64 x 64 outputs by eight waves, for outputs of few tiles: two groups of four waves take
// every other turn, each with a ring of four in LDS, and their sums are joined there. A wave
// has 32 x 32. A product of 768 x 768 takes 11 to 13 us, of which its 36 turns are about 7 and what
// surrounds them the rest.
template <int OP, bool TA, bool TB>
__global__ void __launch_bounds__(512) k_orth_few(const OrthArgs g) {
    constexpr bool SYM = symmetric(OP);
    constexpr int H = 64, kTile = H * kBR, kSlot = 2 * kTile, kSlots = 4;
    __shared__ __attribute__((aligned(16))) _Float16 lds[2 * kSlots * kSlot];
    int tp, tq;
    const int64_t m = place<SYM>(g, g.first + in_turn(g.all), &tp, &tq), p0 = (int64_t)tp * H, q0 = (int64_t)tq * H;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), half = wave >> 2;
    const int wp = (wave >> 1 & 1) * 32, wq = (wave & 1) * 32;
    v4f acc[2][2];
    clear(acc);
    const Fragments<H, TA> ga(wp);
    const Fragments<H, TB> gb(wq);
    const uint32_t base = lds_address(lds) + 2 * kSlots * kSlot * half;
    LoaderA<H, TA, 256, 1> la;
    LoaderB<H, TB, 256, 1> lb;
    constexpr int kLoads = 2 * decltype(la)::kLoads;
    la.init(g.a + m * g.step_a, g.low_a, g.lda, p0, g.P);
    lb.init(g.b + m * g.step_b, g.low_b, g.ldb, q0, g.Q);
    const int n = g.turns / 2;              // sides are padded to 128: an even number
    // loads of turns behind the last are stopped by their buffer's range
    const auto load = [&](int k) {
        const int records = k < n ? kAllRecords : 0;
        const uint32_t to = base + 2 * kSlot * (k % kSlots);
        la.issue(0, la.turn(2 * k + half), to, wave & 3, records);
        lb.issue(0, lb.turn(2 * k + half), to + 2 * kTile, wave & 3, records);
    };
#pragma unroll
    for (int k = 0; k < kSlots - 1; ++k) load(k);
#pragma unroll 1
    for (int k = 0; k < n; ++k) {
        loads_landed<(kSlots - 2) * kLoads>();
        meet_waves();
        load(k + kSlots - 1);
        const uint32_t tile = base + 2 * kSlot * (k % kSlots);
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            h8 fa[2], fb[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                fa[i] = ga.get(tile, i, s);
                fb[i] = gb.get(tile + 2 * kTile, i, s);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j) acc[i][j] = mul(fb[j], fa[i], acc[i][j]);
        }
    }
    loads_landed<0>();
    const OrthEpilogue<OP> epi(g, m, q0 + 8 * (threadIdx.x & 7));
    typename OrthEpilogue<OP>::In in;
    typename OrthEpilogue<OP>::Columns col;
    epi.columns(col, 0);
    epi.load(in, p0 + (threadIdx.x >> 3), 0);
    meet_waves();
    // [64][64] floats, unit u of row o at u ^ (o & 15)
    float* const sums = reinterpret_cast<float*>(lds);
#pragma unroll
    for (int turn = 1; turn >= 0; --turn) {
        if (half == turn)
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int o = wp + 16 * i + ((int)threadIdx.x & 15), u = (wq >> 2) + 4 * j + ((int)threadIdx.x >> 4 & 3);
                    v4f* const at = reinterpret_cast<v4f*>(sums + 64 * o + 4 * (u ^ (o & 15)));
                    if (turn) *at = acc[i][j];
                    else *at = acc[i][j] + *at;
                }
        meet_waves();
    }
    const int o = threadIdx.x >> 3, c = threadIdx.x & 7;
    v4f* const lo = reinterpret_cast<v4f*>(sums + 64 * o + 4 * ((2 * c) ^ (o & 15)));
    v4f* const hi = reinterpret_cast<v4f*>(sums + 64 * o + 4 * ((2 * c + 1) ^ (o & 15)));
    float v[8] = {(*lo)[0], (*lo)[1], (*lo)[2], (*lo)[3], (*hi)[0], (*hi)[1], (*hi)[2], (*hi)[3]};
    epi.put(in, col, p0 + o, 0, v);
    if (SYM && tp != tq) {
        *lo = v4f{v[0], v[1], v[2], v[3]};
        *hi = v4f{v[4], v[5], v[6], v[7]};
        meet_waves();
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int row = 8 * c + k;
            v[k] = sums[64 * row + 4 * ((o >> 2) ^ (row & 15)) + (o & 3)];
        }
        put_pairs(g.out + m * g.step_out + (q0 + o) * g.ld_out + p0 + 8 * c, g.low_out, v);
    }
}

// 128 x 128 outputs by four waves, 64 x 64 each; two turns' tiles in LDS, the next one
// loading while one is multiplied. Two workgroups fit a compute unit, and one's epilogue
// runs beside the other's products: the update of twelve of 768 x 2304 124 to 138 us, 97.8 GFLOP
// in three terms, 0.7 to 0.8 PFLOP/s.
template <int OP, bool TA, bool TB>
__global__ void __launch_bounds__(256, 2) k_orth(const OrthArgs g) {
    constexpr bool SYM = symmetric(OP);
    constexpr int H = 128, kTile = H * kBR;
    __shared__ __attribute__((aligned(16))) _Float16 lds[4 * kTile];
    int tp, tq;
    const int64_t m = place<SYM>(g, g.first + in_turn(g.all), &tp, &tq), p0 = (int64_t)tp * H, q0 = (int64_t)tq * H;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wp = (wave >> 1) * 64, wq = (wave & 1) * 64;
    v4f acc[4][4];
    clear(acc);
    const Fragments<H, TA> ga(wp);
    const Fragments<H, TB> gb(wq);
    const uint32_t base = lds_address(lds);
    LoaderA<H, TA, 256, 1> la;
    LoaderB<H, TB, 256, 1> lb;
    la.init(g.a + m * g.step_a, g.low_a, g.lda, p0, g.P);
    lb.init(g.b + m * g.step_b, g.low_b, g.ldb, q0, g.Q);
    la.issue(0, la.turn(0), base, wave, kAllRecords);
    lb.issue(0, lb.turn(0), base + 2 * kTile, wave, kAllRecords);
#pragma unroll 1
    for (int k = 0; k < g.turns; ++k) {
        loads_landed<0>();
        meet_waves();
        const uint32_t tile = base + 4 * kTile * (k & 1), next = base + 4 * kTile * ((k + 1) & 1);
        if (k + 1 < g.turns) {
            la.issue(0, la.turn(k + 1), next, wave, kAllRecords);
            lb.issue(0, lb.turn(k + 1), next + 2 * kTile, wave, kAllRecords);
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
    auto end = finish<OP, 4, 1>(g, m, [&](int i) { return p0 + wp + 16 * i; }, [&](int) { return q0 + wq; });
    end.ask();
    end(acc, reinterpret_cast<float*>(lds) + wave * 64 * 64, tp != tq);
}

// 128 x 128 outputs by eight waves, 64 x 32 each, one workgroup to a compute unit: a ring of
// four turns' tiles, in turns that barriers divide into two parts. A wave reads the
// turn's operands and asks for the tile three ahead; then it multiplies; waves 4-7 are one
// barrier behind waves 0-3, which share their SIMDs, so that one wave of each pair
// multiplies while the other reads. A tile's place is asked for again one turn after it was
// read, two barriers or more after its last reads began; each turn ends when the next turn's
// tile is here, one barrier before anyone reads it. The 252 tiles of twelve of 768 x 2304 take
// 67 to 73 us for the Gram product and 31 to 34 for the square.
template <int OP, bool TA, bool TB>
__global__ void __launch_bounds__(512) k_orth_mid(const OrthArgs g) {
    constexpr bool SYM = symmetric(OP);
    constexpr int H = 128, kTile = H * kBR, kSlot = 2 * kTile, kSlots = 4;
    __shared__ __attribute__((aligned(16))) _Float16 lds[kSlots * kSlot];
    int tp, tq;
    const int64_t m = place<SYM>(g, g.first + in_turn(g.all), &tp, &tq), p0 = (int64_t)tp * H, q0 = (int64_t)tq * H;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wp = (wave >> 2) * 64, wq = (wave & 3) * 32;
    v4f acc[4][2];
    clear(acc);
    const Fragments<H, TA> ga(wp);
    const Fragments<H, TB> gb(wq);
    const uint32_t base = lds_address(lds);
    LoaderA<H, TA, 512, 1> la;
    LoaderB<H, TB, 512, 1> lb;
    constexpr int kLoads = 2 * decltype(la)::kLoads;
    la.init(g.a + m * g.step_a, g.low_a, g.lda, p0, g.P);
    lb.init(g.b + m * g.step_b, g.low_b, g.ldb, q0, g.Q);
    const int n = g.turns;
    const auto load = [&](int k) {
        const int records = k < n ? kAllRecords : 0;
        const uint32_t to = base + 2 * kSlot * (k % kSlots);
        la.issue(0, la.turn(k), to, wave, records);
        lb.issue(0, lb.turn(k), to + 2 * kTile, wave, records);
    };
    auto end = finish<OP, 2, 1>(g, m, [&](int i) { return p0 + wp + 16 * i; }, [&](int) { return q0 + wq; });
    end.ask();
#pragma unroll
    for (int k = 0; k < kSlots - 1; ++k) load(k);
    loads_landed<(kSlots - 2) * kLoads>();
    meet_waves();
    if (wave >= 4) meet_waves();
#pragma unroll 1
    for (int k = 0; k < n; ++k) {
        const uint32_t tile = base + 2 * kSlot * (k % kSlots);
        h8 fa[2][4], fb[2][2];
#pragma unroll
        for (int s = 0; s < 2; ++s) {
#pragma unroll
            for (int j = 0; j < 2; ++j) fb[s][j] = gb.get(tile + 2 * kTile, j, s);
#pragma unroll
            for (int i = 0; i < 4; ++i) fa[s][i] = ga.get(tile, i, s);
        }
        load(k + kSlots - 1);
        loads_landed<(kSlots - 2) * kLoads>();
        meet_waves();
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_setprio(1);
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j) acc[i][j] = mul(fb[s][j], fa[s][i], acc[i][j]);
        __builtin_amdgcn_s_setprio(0);
        __builtin_amdgcn_sched_barrier(0);
        meet_waves();
    }
    if (wave < 4) meet_waves();
    loads_landed<0>();
    meet_waves();
    end(acc, reinterpret_cast<float*>(lds) + wave * 64 * 32, tp != tq);
}

// 256 x 256 outputs by eight waves, one workgroup to a compute unit. Reduction tiles lie in
// LDS as halves of 128 outer indices, two tiles of four halves. A wave's outputs are 32 x 64
// of each quarter (half of A, half of B), so that it stores whole lines. A tile (a term of 64
// reduction elements: a turn of OrthArgs) is two turns of 32 matrix instructions here, and such a
// turn has two parts that barriers divide: the wave reads
// what its turn needs and no turn before it read, and asks for halves of the tiles to come;
// then it multiplies. Waves 4-7 are one barrier behind waves 0-3, so that one wave of each
// pair multiplies while the other reads.
//
//   turn      reads                asks for                        multiplies
//   2k        A0(k) A1(k) B0(k)    B1(k + 1)                       A0 B0, A1 B0
//   2k + 1    B1(k)                A0(k + 2) A1(k + 2) B0(k + 2)   A0 B1, A1 B1
//
// A half is read in one turn only, by all waves within the two barrier intervals that begin
// with that turn of waves 0-3, and asked for again one turn later: after them. What turn f
// reads was asked for in turn f - 3, or before, or in the prologue; turn f - 1 waits until at
// most the four halves of the two latest turns are under way, and its barrier comes before
// anyone's turn f.
// (With one term a product: four turns of 16 instructions, eight barriers a tile in place of
// four, made the Gram product of 4096 x 11008 take 242 us in place of 200; half of the first
// turn's reads a turn ahead, 12 KB in every turn in place of 16 and 8, 208 us there, and the
// update's 340 in place of 348; the 32 x 32 matrix instruction, with four turns, 5-8% more.) The
// 688 tiles of the update of 11008 x 4096 take 813 us, 1.36 PFLOP/s in three terms.
//
// The workgroup takes reduction tiles first .. last of output tile `t`: WHOLE, or a part,
// whose sums go to memory for k_orth_join, a wave's as they lie in its registers.
template <int OP, bool TA, bool TB, bool WHOLE>
__device__ __forceinline__ void wide_tile(const OrthArgs& g, int t, int first, int last, _Float16* lds, float* part) {
    constexpr bool SYM = symmetric(OP);
    constexpr int H = 128, B = 256, kHalf = H * kBR;
    int tp, tq;
    const int64_t m = place<SYM>(g, t, &tp, &tq), p0 = (int64_t)tp * B, q0 = (int64_t)tq * B;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wp = (wave & 3) * 32, wq = (wave >> 2) * 64;
    v4f acc[4][8];                          // blocks (2 a + i, 4 b + j): block (i, j) of the quarter of halves a and b
    clear(acc);
    const Fragments<H, TA> ga(wp);
    const Fragments<H, TB> gb(wq);
    h8 fa[2][2][2], fb[2][4];               // [half][step][block], [step][block]
    const uint32_t base = lds_address(lds);
    const auto half = [&](int k, int h) { return base + 2 * kHalf * (4 * (k & 1) + h); };   // A0, A1, B0, B1 of tile k
    const auto read_a = [&](int h, uint32_t from) {
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int i = 0; i < 2; ++i) fa[h][s][i] = ga.get(from, i, s);
    };
    const auto read_b = [&](uint32_t from) {
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int j = 0; j < 4; ++j) fb[s][j] = gb.get(from, j, s);
    };
    const auto multiply = [&](int b) {
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_setprio(1);
#pragma unroll
        for (int a = 0; a < 2; ++a)
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) acc[2 * a + i][4 * b + j] = mul(fb[s][j], fa[a][s][i], acc[2 * a + i][4 * b + j]);
        __builtin_amdgcn_s_setprio(0);
        __builtin_amdgcn_sched_barrier(0);
    };
    LoaderA<H, TA, 512, 2> la;
    LoaderB<H, TB, 512, 2> lb;
    constexpr int kLoads = decltype(la)::kLoads;
    la.init(g.a + m * g.step_a, g.low_a, g.lda, p0, g.P);
    lb.init(g.b + m * g.step_b, g.low_b, g.ldb, q0, g.Q);
    const int n = last - first;
    // loads of tiles behind the last are stopped by their buffer's range
    const auto there = [&](int k) { return k < n ? kAllRecords : 0; };
    const char *a0 = la.turn(first), *b0 = lb.turn(first), *a1 = la.turn(first + 1), *b1 = lb.turn(first + 1);
    la.issue(0, a0, half(0, 0), wave, kAllRecords);
    la.issue(1, a0, half(0, 1), wave, kAllRecords);
    lb.issue(0, b0, half(0, 2), wave, kAllRecords);
    lb.issue(1, b0, half(0, 3), wave, kAllRecords);
    la.issue(0, a1, half(1, 0), wave, there(1));
    la.issue(1, a1, half(1, 1), wave, there(1));
    lb.issue(0, b1, half(1, 2), wave, there(1));
    loads_landed<4 * kLoads>();
    meet_waves();
    if (wave >= 4) meet_waves();
#pragma unroll 1
    for (int k = 0; k < n; ++k) {
        const int one = there(k + 1), two = there(k + 2);
        read_a(0, half(k, 0));
        read_b(half(k, 2));
        read_a(1, half(k, 1));
        lb.issue(1, b1, half(k + 1, 3), wave, one);
        loads_landed<4 * kLoads>();
        meet_waves();
        multiply(0);
        meet_waves();
        read_b(half(k, 3));
        a1 = la.turn(first + k + 2);
        b1 = lb.turn(first + k + 2);
        la.issue(0, a1, half(k, 0), wave, two);
        la.issue(1, a1, half(k, 1), wave, two);
        lb.issue(0, b1, half(k, 2), wave, two);
        loads_landed<4 * kLoads>();
        meet_waves();
        multiply(1);
        meet_waves();
    }
    if (wave < 4) meet_waves();
    loads_landed<0>();
    meet_waves();
    if constexpr (WHOLE) {
        auto end = finish<OP, 4, 2>(g, m, [&](int i) { return p0 + H * (i >> 1) + wp + 16 * (i & 1); },
                                    [&](int run) { return q0 + H * run + wq; });
        end.ask();
        end(acc, reinterpret_cast<float*>(lds) + wave * 64 * 64, SYM && tp != tq);
    } else {
        float* const to = part + wave * (64 * 128) + 4 * ((int)threadIdx.x & 63);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) *reinterpret_cast<v4f*>(to + 256 * (16 * (j >> 2) + 4 * i + (j & 3))) = acc[i][j];
    }
}
template <int OP, bool TA, bool TB>
__global__ void __launch_bounds__(512) k_orth_wide(const OrthArgs g) {
    __shared__ __attribute__((aligned(16))) _Float16 lds[2 * 4 * kSide * kBR];
    wide_tile<OP, TA, TB, true>(g, g.first + in_turn(g.all), 0, g.turns, lds, nullptr);
}

// Fewer tiles than kSplit, shared by kSplit workgroups (Slices), all of them at the same place of the
// reduction as those that share operand rows with them: workgroup w < a s takes slice w / a of
// s of tile w % a; the r tiles that are left over are cut likewise, into t slices, for a
// second part of each workgroup's work. k_orth_join puts the parts together, in order.
// (Runs of consecutive turns, whatever tile they are of, share no operand rows in the caches:
// with one term a product, the Gram product of 4096 x 11008 took 240 us in place of 180.) As it
// is the Gram product of 11008 x 4096 takes 477 to 512 us and its join 44 to 46, by the 128 MB of
// sums between them; the square 180 to 192 and 42 to 44.
template <int OP, bool TA, bool TB>
__global__ void __launch_bounds__(512) k_orth_split(const OrthArgs g) {
    __shared__ __attribute__((aligned(16))) _Float16 lds[2 * 4 * kSide * kBR];
    const int w = in_turn(kSplit);
    const Slices c = slices_of(g.all);
#pragma unroll 1
    for (int part = 0; part < 2; ++part) {
        const int tiles = part ? c.r : c.a, n = part ? c.t : c.s;
        if (w >= tiles * n) continue;
        // the same in all lanes, which the divisions hide from the compiler
        const int slice = __builtin_amdgcn_readfirstlane(w / tiles);
        const int first = __builtin_amdgcn_readfirstlane(g.turns * slice / n);
        const int last = __builtin_amdgcn_readfirstlane(g.turns * (slice + 1) / n);
        wide_tile<OP, TA, TB, false>(g, g.first + (part ? c.a : 0) + w - slice * tiles, first, last, lds,
                                     g.part + (kSplit * part + w) * kPartFloats);
    }
}
// A wave to half of what one of the waves that computed it had of a tile, a workgroup each.
template <int OP>
__global__ void __launch_bounds__(64) k_orth_join(const OrthArgs g) {
    __shared__ __attribute__((aligned(16))) float lds[64 * 64];
    constexpr bool SYM = symmetric(OP);
    constexpr int H = 128, B = 256;
    const int t = blockIdx.x >> 4, wave = blockIdx.x >> 1 & 7, half = blockIdx.x & 1;
    const int wp = (wave & 3) * 32, wq = (wave >> 2) * 64;
    const Slices c = slices_of(g.all);
    const int tiles = t < c.a ? c.a : c.r, n = t < c.a ? c.s : c.t;
    const float* from = g.part + (t < c.a ? t : kSplit + t - c.a) * kPartFloats + wave * (64 * 128) + half * (64 * 64) +
                        4 * threadIdx.x;
    v4f acc[4][4];
    clear(acc);
#pragma unroll 2
    for (int k = 0; k < n; ++k, from += tiles * kPartFloats)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][j] += *reinterpret_cast<const v4f*>(from + 256 * (4 * i + j));
    int tp, tq;
    const int64_t m = place<SYM>(g, g.first + t, &tp, &tq), p0 = (int64_t)tp * B, q0 = (int64_t)tq * B;
    auto end = finish<OP, 4, 1>(g, m, [&](int i) { return p0 + H * (i >> 1) + wp + 16 * (i & 1); },
                                [&](int) { return q0 + H * half + wq; });
    end.ask();
    end(acc, lds, SYM && tp != tq);
}

// ---------------------------------------------------------------------------
// before the first step
// ---------------------------------------------------------------------------

struct StartArgs {
    const void* x;
    int64_t ld_x, step_x, rows, cols;
    int64_t Rp, Cp;
    _Float16* hi;
    int64_t low;
    double* parts;                  // [matrix][kSquareParts]
    int32_t n_parts;
    double eps;
};

template <int WAVES>
__device__ __forceinline__ double block_sum(double v) {
    __shared__ double s[WAVES];
#pragma unroll
    for (int k = 32; k > 0; k >>= 1) v += __shfl_xor(v, k);
    if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
    __syncthreads();
    v = s[0];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) v += s[w];
    return v;
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

// Sums of squares in 64 bits (no scale overflows them), a workgroup's each to its place:
// sixteen waves of it, as a matrix has at most one to a compute unit.
constexpr int kSquareBlock = 1024;
template <bool XF>
__global__ void __launch_bounds__(kSquareBlock) k_orth_squares(const StartArgs g) {
    const int64_t m = blockIdx.y, chunks = (g.cols + 7) / 8, all = g.rows * chunks;
    const double inv = 1.0 / (double)chunks;
    double sum = 0.0;
#pragma unroll 4
    for (int64_t id = (int64_t)blockIdx.x * kSquareBlock + threadIdx.x; id < all; id += (int64_t)g.n_parts * kSquareBlock) {
        int64_t c;
        const int64_t row = row_of_chunk(id, chunks, inv, &c);
        float v[8];
        load_x8<XF>(v, g, m, row, 8 * c);
#pragma unroll
        for (int k = 0; k < 8; ++k) sum = fma((double)v[k], (double)v[k], sum);
    }
    sum = block_sum<kSquareBlock / 64>(sum);
    if (threadIdx.x == 0) g.parts[m * kSquareParts + blockIdx.x] = sum;
}

// X with its padding, 11008 x 4096 from bf16 in 44 to 50 us (5.4 to 6.1 TB/s). A norm that is not finite makes all of them NaN.
template <bool XF>
__global__ void __launch_bounds__(256) k_orth_start(const StartArgs g) {
    const int64_t m = blockIdx.y, chunks = g.Cp / 8, all = g.Rp * chunks;
    const double square = block_sum<4>((int)threadIdx.x < g.n_parts ? g.parts[m * kSquareParts + threadIdx.x] : 0.0);
    const double norm = sqrt(square), inv = 1.0 / (double)chunks;
    const double by = (double)kScaleX / (norm + g.eps);
    const bool fine = norm < INFINITY;
#pragma unroll 2
    for (int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x; id < all; id += (int64_t)gridDim.x * 256) {
        int64_t c;
        const int64_t row = row_of_chunk(id, chunks, inv, &c);
        float v[8];
        load_x8<XF>(v, g, m, row, 8 * c);
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = fine ? (float)((double)v[k] * by) : NAN;
        put_pairs(g.hi + m * g.Rp * g.Cp + row * g.Cp + 8 * c, g.low, v);
    }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

size_t orth_ws_bytes(int64_t batch, int64_t rows, int64_t cols) {
    if (batch < 1 || rows < 1 || cols < 1) return 0;
    const OrthShape s = shape_of(batch, rows, cols);
    return (size_t)s.group * s.each + s.part;
}

template <int OP, bool TA, bool TB>
static hipError_t run(const OrthPlan& plan, OrthArgs g, int64_t n, hipStream_t st) {
    constexpr bool SYM = symmetric(OP);
    const OrthKind kind = plan.kind;
    const int side = kind == kFew ? 64 : kind == kWide ? 256 : 128, threads = kind == kTwo ? 256 : 512;
    g.np = (int32_t)over(g.P, side);
    g.nq = (int32_t)over(g.Q, side);
    g.tiles = (int32_t)tiles_of(g.P, g.Q, side, SYM);
    const auto k = kind == kFew ? k_orth_few<OP, TA, TB> : kind == kMid ? k_orth_mid<OP, TA, TB>
                   : kind == kTwo ? k_orth<OP, TA, TB> : k_orth_wide<OP, TA, TB>;
    // a launch holds 2^31 threads
    const int64_t whole = n * g.tiles - plan.split, most = int64_t(1) << 22;
    for (int64_t done = 0; done < whole; done += most) {
        g.first = (int32_t)done;
        g.all = (int32_t)(whole - done < most ? whole - done : most);
        hipLaunchKernelGGL(k, dim3((unsigned)g.all), dim3(threads), 0, st, g);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if (plan.split == 0) return hipSuccess;
    g.first = (int32_t)whole;
    g.all = (int32_t)plan.split;
    hipLaunchKernelGGL((k_orth_split<OP, TA, TB>), dim3(kSplit), dim3(512), 0, st, g);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((k_orth_join<OP>), dim3(16 * (unsigned)g.all), dim3(64), 0, st, g);
    return hipGetLastError();
}
template <int OP, bool TA, bool TB>
static hipError_t product(const OrthArgs& g, int64_t n, bool may_split, hipStream_t st) {
    return run<OP, TA, TB>(plan_of(n, g.P, g.Q, g.turns, symmetric(OP), may_split), g, n, st);
}

static hipError_t orthogonalize(const OrthDesc& d, const OrthShape& s, int64_t first, int64_t n, hipStream_t st) {
    const int64_t x_all = s.group * s.x, a_all = s.group * s.a;
    _Float16* const xs[2] = {static_cast<_Float16*>(d.ws), static_cast<_Float16*>(d.ws) + 2 * x_all};
    _Float16* const A = xs[1] + 2 * x_all;
    _Float16* const B = A + 2 * a_all;
    float* const da = reinterpret_cast<float*>(B + 2 * a_all);
    float* const db = da + s.group * s.m;
    double* const parts = reinterpret_cast<double*>(db + s.group * s.m);
    float* const part = reinterpret_cast<float*>(parts + s.group * kSquareParts);
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
    b.hi = xs[0];
    b.low = x_all;
    b.parts = parts;
    b.eps = d.eps;
    // a chunk to a thread while all workgroups run at once, else four (768 x 768 4.2 us in place
    // of 6.2; twelve of 768 x 2304 13.5 in place of 19.7)
    const int64_t squares = over(d.rows * over(d.cols, 8), kSquareBlock), whole = (s.x / 8 + 511) / 512;
    const int64_t squares_at = n * squares <= 256 ? squares : over(squares, 4);
    b.n_parts = (int32_t)(squares_at < kSquareParts ? squares_at : kSquareParts);
    const unsigned blocks = (unsigned)(whole < 2048 ? whole : 2048);
    hipLaunchKernelGGL(d.x_f32 ? k_orth_squares<true> : k_orth_squares<false>, dim3((unsigned)b.n_parts, (unsigned)n),
                       dim3(kSquareBlock), 0, st, b);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(d.x_f32 ? k_orth_start<true> : k_orth_start<false>, dim3(blocks, (unsigned)n), dim3(256), 0, st, b);
    if ((e = hipGetLastError()) != hipSuccess) return e;

    for (int k = 0; k < d.steps; ++k) {
        const _Float16* const X = xs[k & 1];
        OrthArgs g{};
        g.ca = (float)d.coefficients[3 * k];
        g.cb = (float)d.coefficients[3 * k + 1];
        g.cc = (float)d.coefficients[3 * k + 2];
        g.step_diag = s.m;
        g.part = part;
        // A
        OrthArgs p = g;
        p.a = p.b = X;
        p.low_a = p.low_b = x_all;
        p.lda = p.ldb = s.Cp;
        p.step_a = p.step_b = s.x;
        p.P = p.Q = s.m;
        p.turns = (int32_t)turns_of(tall ? s.Rp : s.Cp);
        p.out = A;
        p.low_out = a_all;
        p.ld_out = s.m;
        p.step_out = s.a;
        p.diag_out = da;
        e = tall ? product<kGram, true, true>(p, n, s.may_split, st) : product<kGram, false, false>(p, n, s.may_split, st);
        if (e != hipSuccess) return e;
        // b A + c A A
        p = g;
        p.a = p.b = p.in = A;
        p.low_a = p.low_b = p.low_in = p.low_out = a_all;
        p.lda = p.ldb = p.ld_in = p.ld_out = s.m;
        p.step_a = p.step_b = p.step_in = p.step_out = s.a;
        p.P = p.Q = s.m;
        p.turns = (int32_t)turns_of(s.m);
        p.diag_in = da;
        p.out = B;
        p.diag_out = db;
        if ((e = product<kSquare, false, false>(p, n, s.may_split, st)) != hipSuccess) return e;
        // X; b A + c A A is symmetric, and so an operand with its outer index in rows on either side
        p = g;
        p.a = tall ? X : B;
        p.b = tall ? B : X;
        p.low_a = tall ? x_all : a_all;
        p.low_b = tall ? a_all : x_all;
        p.lda = tall ? s.Cp : s.m;
        p.ldb = tall ? s.m : s.Cp;
        p.step_a = tall ? s.x : s.a;
        p.step_b = tall ? s.a : s.x;
        p.P = s.Rp;
        p.Q = s.Cp;
        p.turns = (int32_t)turns_of(s.m);
        p.in = X;
        p.low_in = p.low_out = x_all;
        p.ld_in = p.ld_out = s.Cp;
        p.step_in = p.step_out = s.x;
        p.diag_in = db;
        if (k + 1 < d.steps) {
            p.out = xs[(k + 1) & 1];
        } else {
            p.o = d.o + first * d.stride_o;
            p.ld_o = d.ld_o;
            p.step_o = d.stride_o;
            p.rows = d.rows;
            p.cols = d.cols;
            p.scale = d.scale;
        }
        e = tall ? product<kUpdateTall, false, false>(p, n, s.may_split, st) : product<kUpdate, false, true>(p, n, s.may_split, st);
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
