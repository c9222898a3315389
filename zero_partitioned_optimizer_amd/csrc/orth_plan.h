// orth_plan.h -- how the products of an orthogonalisation are cut into tiles, and what lies in
// its workspace (orth_kernels.hip runs them). Plain C++, without device code.
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace zk {

constexpr int kBR = 64;                     // reduction elements per staged tile
constexpr int kTerms = 3;                   // of a product of pairs: hi hi, hi lo, lo hi
constexpr int kSide = 128;                  // all sides are padded to this, with zeros
constexpr int kSquareParts = 256;           // partial sums of squares of a matrix, at most

// Fewer tiles than kSplit, shared by kSplit workgroups (k_orth_split): s slices of each of the
// first a tiles, t of each of the r that are left over.
constexpr int kSplit = 256;
constexpr int64_t kPartFloats = 256 * 256;
struct Slices {
    int32_t s, a, r, t;
};
constexpr Slices slices_of(int32_t tiles) {
    Slices c{};
    c.s = (kSplit + tiles - 1) / tiles;
    c.a = kSplit / c.s;
    c.r = tiles - c.a;
    c.t = c.r > 0 ? kSplit / c.r : 0;
    return c;
}

inline int64_t padded(int64_t n) { return (n + kSide - 1) / kSide * kSide; }
inline int64_t turns_of(int64_t R) { return kTerms * R / kBR; }

inline int64_t over(int64_t n, int64_t by) { return (n + by - 1) / by; }
inline int64_t tiles_of(int64_t P, int64_t Q, int64_t side, bool sym) {
    const int64_t p = over(P, side), q = over(Q, side);
    return sym ? p * (p + 1) / 2 : p * q;
}

// How a product of n matrices runs, by an estimate of its time in microseconds.
enum OrthKind { kFew, kMid, kTwo, kWide };
struct OrthPlan {
    OrthKind kind;
    int64_t split;                  // kWide: of all tiles, the last ones that are split
};
inline OrthPlan plan_of(int64_t n, int64_t P, int64_t Q, int64_t turns, bool sym, bool may_split) {
    const int64_t few = n * tiles_of(P, Q, 64, sym), mid = n * tiles_of(P, Q, 128, sym), wide = n * tiles_of(P, Q, 256, sym);
    OrthPlan best{kTwo, 0};
    double least = 1e300;
    const auto offer = [&](OrthKind k, int64_t split, double time) {
        if (time < least) {
            least = time;
            best = OrthPlan{k, split};
        }
    };
    // us for a turn and for a tile's start and end, in a round of the chip, as measured with 1 to 2,752
    // tiles of 64 to 5,632 columns and 6 to 516 turns; of 54 such products the estimate took the
    // fastest kind for 48 and ones 1 to 6% slower for the others. A wide tile's turn takes 1.45 in a round of
    // 256 and 1.1 with half of the compute units idle (128 tiles 1.06 to 1.18, 180 1.21, 216 1.32).
    const int64_t rest = mid % 512;
    offer(kTwo, 0, mid / 512 * (0.9 * turns + 9) + (rest == 0 ? 0 : rest <= 256 ? 0.65 * turns + 8.5 : 0.9 * turns + 9));
    offer(kFew, 0, over(few, 256) * (0.185 * turns + 3.4));
    // a compute unit to each: at 171 to 252 tiles 15 to 31% faster than two a unit, at 273 to 960 from
    // 2% faster to 24% slower
    if (mid <= 256) offer(kMid, 0, 0.49 * turns + 8.5);
    const int64_t left = wide % kSplit;
    const double ends = sym ? 12 : 18, rounds = wide / 256 * (1.45 * turns + ends);
    const double turn = left <= 128 ? 1.1 : 1.1 + 0.35 * (left - 128) / 128;
    offer(kWide, 0, rounds + (left == 0 ? 0 : turn * turns + ends));
    if (left > 0 && may_split) {
        const Slices c = slices_of((int32_t)left);
        const double each = (double)turns / c.s + (c.r > 0 ? (double)turns / c.t : 0);
        // the join: by all parts, or by those that one wave adds up
        const double all = 0.088 * (c.a * c.s + c.r * c.t), one = 0.33 * c.s;
        if (turns >= 2 * c.s && turns >= c.t)       // two turns to a slice, one to the others
            offer(kWide, left, rounds + 1.5 * each + 25 + (all > one ? all : one));
    }
    return best;
}

// What a group of matrices has in the workspace, in this order: X twice, A and b A + c A A, hi
// and then lo of each, the diagonals, the partial sums of squares, those of split tiles.
struct OrthShape {
    int64_t Rp, Cp, m;              // padded sides, the smaller one
    int64_t x, a;                   // elements
    size_t each;                    // bytes of a matrix
    int64_t group;                  // matrices at a time
    bool may_split;
    size_t part;                    // bytes of split tiles' partial sums
};
inline OrthShape shape_of(int64_t batch, int64_t rows, int64_t cols) {
    OrthShape s{};
    s.Rp = padded(rows);
    s.Cp = padded(cols);
    s.m = s.Rp < s.Cp ? s.Rp : s.Cp;
    s.x = s.Rp * s.Cp;
    s.a = s.m * s.m;
    s.each = (size_t)(8 * s.x + 8 * s.a + 8 * s.m) + kSquareParts * sizeof(double);
    const int64_t most = (int64_t)((size_t(4) << 30) / s.each);
    s.group = most < 1 ? 1 : most > 16384 ? 16384 : most;     // a grid's y
    if (s.group > batch) s.group = batch;
    // Groups of a longer stack are 4 GiB of matrices, whose tiles go round the chip many times: what
    // a split would save of the last round is little, and its partial sums are 128 MB.
    s.may_split = s.group == batch || s.group == 1;
    const int64_t gram = turns_of(rows > cols ? s.Rp : s.Cp), square = turns_of(s.m), n = s.group;
    const bool split = plan_of(n, s.m, s.m, gram, true, s.may_split).split ||
                       plan_of(n, s.m, s.m, square, true, s.may_split).split ||
                       plan_of(n, s.Rp, s.Cp, square, false, s.may_split).split;
    s.part = split ? 2 * kSplit * kPartFloats * sizeof(float) : 0;
    return s;
}

}  // namespace zk
