// norm_kernels.hip -- the norm of a block's rows and its gradient:
//   forward   s = residual + x; y = (s - mean) rstd w + b
//   gradient  h = (x - mean) rstd, g = dy w: dx = residual_grad + rstd (g - mean(g) - h mean(g h)),
//             dw = [dw +] sum of dy h over the rows, db = [db +] sum of dy
// The mean is taken in two parts, m from the sum of the differences to one of the row's elements
// and delta from that of the differences to m: a row of one value has differences of exactly 0
// however its mean would round, and where the mean is large beside sigma delta is what m lacks.
// The variance is the mean of the squared differences to m, less delta^2.
// Bound by HBM where rows are long: each matrix is read or written once. A row stays in
// registers between its sums and its outputs, eight columns to a lane and 16 bytes to a load.
// 8192 x 4096, bf16 rows added to an f32 stream, RMS: 77 us, 5.2 TB/s; back through it with the
// stream's gradient in bf16 61 us, 5.5 TB/s, 4.8 of them the second launch. Rows of 768 in bf16
// are bound by their instructions as much: 8192 of them forward 11.6 to 12 us, 4.2 to 4.3 TB/s (0.3
// of it the mean in two parts), back 16.0 and 3.2 (12.1 and 4 the two launches). Divisions, masks of columns that do not exist and 64-bit
// products of addresses out of the loops were 3 of 19 us there, and of 45 at 2304 columns 7.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "layer_device.h"

namespace zk {

template <bool F>
__device__ __forceinline__ void load8(float v[8], const void* p, int64_t at, int n) {
    if constexpr (F) load8_f(v, static_cast<const float*>(p) + at, n);
    else load8_bf(v, static_cast<const uint16_t*>(p) + at, n);
}
__device__ __forceinline__ v4u load_once(const void* p) {
    return __builtin_nontemporal_load(static_cast<const v4u_any*>(p));
}
template <bool F>
__device__ __forceinline__ void store8(void* p, int64_t at, const float v[8], int n) {
    if constexpr (F) store8_f(static_cast<float*>(p) + at, v, n);
    else store8_bf(static_cast<uint16_t*>(p) + at, v, n);
}
__device__ __forceinline__ int valid8(int64_t N, int64_t j) {
    return N - j >= 8 ? 8 : N > j ? (int)(N - j) : 0;
}
// Eight of a norm's weights, or ones.
__device__ __forceinline__ void weights8(float v[8], const uint16_t* w, int64_t j, int n) {
    if (w && n > 0) {
        load8_bf(v, w + j, n);
        return;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = 1.0f;
}

// Eight elements of a row as they lie in memory: asked for ahead of their use, converted then.
// Inputs are read once and do not stay in the caches.
template <bool F>
struct Raw {
    v4u lo, hi;
    __device__ __forceinline__ void load(const void* base, int64_t at, int n) {
        // zeros first: written behind a load of other lanes they would wait for it
        lo = hi = v4u{0, 0, 0, 0};
        if constexpr (F) {
            const float* const p = static_cast<const float*>(base) + at;
            if (n >= 8) {
                lo = load_once(p);
                hi = load_once(p + 4);
            } else if (n > 0) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    if (k < n) lo[k] = __float_as_uint(p[k]);
                    if (4 + k < n) hi[k] = __float_as_uint(p[4 + k]);
                }
            }
        } else {
            const uint16_t* const p = static_cast<const uint16_t*>(base) + at;
            if (n >= 8) {
                lo = load_once(p);
            } else if (n > 0) {
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (k < n) lo[k >> 1] |= (uint32_t)p[k] << (16 * (k & 1));
            }
        }
    }
    __device__ __forceinline__ void set(const float v[8]) {
        if constexpr (F) {
            lo = v4u{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])};
            hi = v4u{__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7])};
        } else {
            lo = v4u{bf_pack(v[0], v[1]), bf_pack(v[2], v[3]), bf_pack(v[4], v[5]), bf_pack(v[6], v[7])};
        }
    }
    __device__ __forceinline__ void store(void* base, int64_t at, int n) const {
        if constexpr (F) {
            float* const p = static_cast<float*>(base) + at;
            if (n >= 8) {
                *reinterpret_cast<v4u_any*>(p) = lo;
                *reinterpret_cast<v4u_any*>(p + 4) = hi;
            } else if (n > 0) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    if (k < n) p[k] = __uint_as_float(lo[k]);
                    if (4 + k < n) p[4 + k] = __uint_as_float(hi[k]);
                }
            }
        } else {
            uint16_t* const p = static_cast<uint16_t*>(base) + at;
            if (n >= 8) {
                *reinterpret_cast<v4u_any*>(p) = lo;
            } else if (n > 0) {
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (k < n) p[k] = (uint16_t)(lo[k >> 1] >> (16 * (k & 1)));
            }
        }
    }
    // What is made of it from here on is made anew.
    __device__ __forceinline__ void keep() {
        asm volatile("" : "+v"(lo));
        if constexpr (F) asm volatile("" : "+v"(hi));
    }
    __device__ __forceinline__ void get(float v[8]) const {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            v[F ? k : 2 * k] = F ? __uint_as_float(lo[k]) : bf_lo(lo[k]);
            v[F ? 4 + k : 2 * k + 1] = F ? __uint_as_float(hi[k]) : bf_hi(lo[k]);
        }
    }
};
// Eight of a norm's bf16 weights (`none`: what their halves are without any), kept as they are.
struct RawWeights {
    v4u w;
    __device__ __forceinline__ void load(const uint16_t* p, int64_t j, int n, uint32_t none) {
        w = v4u{none, none, none, none};
        if (!p || n <= 0) return;
        if (n >= 8) {
            w = *reinterpret_cast<const v4u_any*>(p + j);
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (k < n) w[k >> 1] = (w[k >> 1] & (k & 1 ? 0xFFFFu : 0xFFFF0000u)) | (uint32_t)p[j + k] << (16 * (k & 1));
        }
    }
    __device__ __forceinline__ float get(int k) const { return k & 1 ? bf_hi(w[k >> 1]) : bf_lo(w[k >> 1]); }
};
constexpr uint32_t kOnes = 0x3F803F80u;

template <int CONTROL>
__device__ __forceinline__ float add_across(float v) {
    return v + __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(v), CONTROL, 0xF, 0xF, true));
}
__device__ __forceinline__ float lane_of(float v, int lane) {
    return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), lane));
}
// The same in all lanes: 16 lanes' sums by exchanges within them, then the four.
__device__ __forceinline__ float wave_sum(float v) {
    v = add_across<0xB1>(v);            // lanes 1, 0, 3, 2 of four
    v = add_across<0x4E>(v);            // 2, 3, 0, 1
    v = add_across<0x141>(v);           // mirrored in eight
    v = add_across<0x140>(v);           // and in sixteen
    return (lane_of(v, 0) + lane_of(v, 16)) + (lane_of(v, 32) + lane_of(v, 48));
}
// Sums over the W waves that share a row; `part` is W floats of LDS that nothing else has
// used since the last barrier but one.
template <int W>
__device__ __forceinline__ float row_sum(float v, float* part) {
    v = wave_sum(v);
    if constexpr (W > 1) {
        if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
        __syncthreads();
        v = part[0];
#pragma unroll
        for (int w = 1; w < W; ++w) v += part[w];
    }
    return v;
}

// Two sums at a time; `part` likewise, of pairs.
template <int W>
__device__ __forceinline__ void row_sums(float& a, float& b, float (*part)[2]) {
    a = wave_sum(a);
    b = wave_sum(b);
    if constexpr (W > 1) {
        if ((threadIdx.x & 63) == 0) {
            part[threadIdx.x >> 6][0] = a;
            part[threadIdx.x >> 6][1] = b;
        }
        __syncthreads();
        a = part[0][0];
        b = part[0][1];
#pragma unroll
        for (int w = 1; w < W; ++w) {
            a += part[w][0];
            b += part[w][1];
        }
    }
}
// The mean of a row from the sums that its waves have of the differences to an element of theirs:
// wave w has columns 512 (w + W i) .. + 511, i < C, that are below N.
template <int W, int C>
__device__ __forceinline__ float row_mean(float sum, float one, int N, float (*part)[2]) {
    sum = wave_sum(sum);
    if constexpr (W > 1) {
        if ((threadIdx.x & 63) == 0) {
            part[threadIdx.x >> 6][0] = sum;
            part[threadIdx.x >> 6][1] = one;
        }
        __syncthreads();
        sum = part[0][0];
        one = part[0][1];
#pragma unroll
        for (int w = 1; w < W; ++w) {
            int n = 0;
#pragma unroll
            for (int i = 0; i < C; ++i) {
                const int left = N - 512 * (w + W * i);
                n += left > 512 ? 512 : left > 0 ? left : 0;
            }
            sum += fmaf((float)n, part[w][1] - one, part[w][0]);
        }
    }
    return one + sum / (float)N;
}
// rstd, from the mean of the squares of a row's differences to m and delta, their own mean.
__device__ __forceinline__ float row_rstd(float square, float delta, float eps) {
    const float var = fmaf(-delta, delta, square);
    return 1.0f / sqrtf((var < 0.0f ? 0.0f : var) + eps);       // a NaN stays one
}

constexpr int kNormBlock = 256;

// s of eight columns, rounded to its own type and stored, where there is a residual; x
// itself otherwise.
template <bool XF, bool SF>
__device__ __forceinline__ void sum8(float v[8], const NormDesc& d, int64_t row, int64_t j, int n) {
    load8<XF>(v, d.x, row * d.ld_x + j, n);
    if (!d.res) return;
    float r[8];
    load8<SF>(r, d.res, row * d.ld_res + j, n);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        v[k] += r[k];
        if constexpr (!SF) v[k] = bf_f(bf_one(v[k]));
    }
    store8<SF>(d.sum, row * d.ld_sum + j, v, n);
}
template <bool YF>
__device__ __forceinline__ void norm8(const float v[8], const NormDesc& d, float m, float rstd, float shift, int64_t row,
                                      int64_t j, int n) {
    float w[8], b[8], y[8];
    weights8(w, d.w, j, n);
#pragma unroll
    for (int k = 0; k < 8; ++k) b[k] = 0.0f;
    if (d.b) load8_bf(b, d.b + j, n);
#pragma unroll
    for (int k = 0; k < 8; ++k) y[k] = fmaf(v[k] - m, rstd, shift) * w[k] + b[k];
    store8<YF>(d.y, row * d.ld_y + j, y, n);
}

// W waves to a row of at most 512 W C columns, held in registers; one or (W = 1) four rows to a
// workgroup at a time, which takes every `stride`-th group of them and asks for the next row
// before it works on one. Loads that stay in the caches: 8192 x 2304 33.6 in place of 29.2 us.
template <bool XF, bool SF, bool YF, int W, int C>
__global__ void __launch_bounds__(W > 4 ? 512 : kNormBlock) k_norm(const NormDesc d, int64_t stride) {
    constexpr int G = W == 1 ? 4 : 1;
    __shared__ float part[2][2][W][2];
    const int t = W == 1 ? threadIdx.x & 63 : threadIdx.x;
    int64_t row = (int64_t)blockIdx.x * G + (W == 1 ? threadIdx.x >> 6 : 0);
    if (row >= d.M) return;
    int j[C], n[C];
    RawWeights w[C], b[C];
    Raw<XF> x[C];
    Raw<SF> r[C];
    const auto ask = [&](int64_t at) {
#pragma unroll
        for (int i = 0; i < C; ++i) {
            x[i].load(d.x, at * d.ld_x + j[i], n[i]);
            if (d.res) r[i].load(d.res, at * d.ld_res + j[i], n[i]);
        }
    };
#pragma unroll
    for (int i = 0; i < C; ++i) {
        j[i] = 8 * (t + 64 * W * i);
        n[i] = valid8(d.N, j[i]);
    }
    ask(row);
#pragma unroll
    for (int i = 0; i < C; ++i) {
        w[i].load(d.w, j[i], n[i], kOnes);
        b[i].load(d.b, j[i], n[i], 0);
    }
    int turn = 0;
#pragma unroll 1
    for (;; turn ^= 1) {
        float v[C][8], sq = 0.0f, delta = 0.0f, m = 0.0f;
        Raw<SF> s[C];
#pragma unroll
        for (int i = 0; i < C; ++i) {
            x[i].get(v[i]);
            if (d.res) {
                float add[8];
                r[i].get(add);
#pragma unroll
                for (int k = 0; k < 8; ++k) v[i][k] += add[k];
                s[i].set(v[i]);
                if constexpr (!SF) s[i].get(v[i]);          // what is stored is what is normed
            }
        }
        const int64_t next = row + stride * G;
        if (next < d.M) ask(next);
        if (d.res)
#pragma unroll
            for (int i = 0; i < C; ++i) s[i].store(d.sum, row * d.ld_sum + j[i], n[i]);
        // the differences of a chunk to `by`; of no column: zeros, and 0 to the sums
        const auto less = [&](float to[8], int i, float by) {
            const float b = n[i] > 0 ? by : 0.0f;
#pragma unroll
            for (int k = 0; k < 8; ++k) to[k] = v[i][k] - b;
            if (n[i] > 0 && n[i] < 8)
#pragma unroll
                for (int k = 1; k < 8; ++k)
                    if (k >= n[i]) to[k] = 0.0f;
        };
        if (!d.rms) {
            const float one = lane_of(v[0][0], 0);
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < C; ++i) {
                float e[8];
                less(e, i, one);
#pragma unroll
                for (int k = 0; k < 8; ++k) sum += e[k];
            }
            m = row_mean<W, C>(sum, one, (int)d.N, part[turn][0]);
        }
#pragma unroll
        for (int i = 0; i < C; ++i) {
            less(v[i], i, m);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                sq = fmaf(v[i][k], v[i][k], sq);
                delta += v[i][k];
            }
        }
        row_sums<W>(sq, delta, part[turn][1]);
        delta = d.rms ? 0.0f : delta / (float)d.N;
        const float rstd = row_rstd(sq / (float)d.N, delta, d.eps), shift = d.rms ? 0.0f : -delta * rstd;
        if (d.stats && t == 0) {
            d.stats[2 * row] = m + delta;
            d.stats[2 * row + 1] = rstd;
        }
#pragma unroll
        for (int i = 0; i < C; ++i) {
#pragma unroll
            for (int k = 0; k < 8; ++k) v[i][k] = fmaf(v[i][k], rstd, shift) * w[i].get(k) + b[i].get(k);
            Raw<YF> y;
            y.set(v[i]);
            y.store(d.y, row * d.ld_y + j[i], n[i]);
        }
        if (next >= d.M) return;
        row = next;
    }
}

// Rows of any length, read again for each sum (from the caches, up to some length).
template <bool XF, bool SF, bool YF>
__global__ void __launch_bounds__(kNormBlock) k_norm_long(const NormDesc d, int64_t first) {
    __shared__ float part[4];
    __shared__ float parts[4][2];
    const int64_t row = first + blockIdx.x;
    float v[8], one[8], sum = 0.0f, sq = 0.0f, delta = 0.0f, m = 0.0f;
    load8<XF>(one, d.x, row * d.ld_x, 1);
    if (d.res) {
        load8<SF>(v, d.res, row * d.ld_res, 1);
        one[0] += v[0];
        if constexpr (!SF) one[0] = bf_f(bf_one(one[0]));
    }
    __syncthreads();                    // sum may be written over x or the residual
    const auto again = [&](int64_t j, int n) {
        if (d.res) load8<SF>(v, d.sum, row * d.ld_sum + j, n);
        else load8<XF>(v, d.x, row * d.ld_x + j, n);
    };
    for (int64_t j = 8 * threadIdx.x; j < d.N; j += 8 * kNormBlock) {
        const int n = valid8(d.N, j);
        sum8<XF, SF>(v, d, row, j, n);
#pragma unroll
        for (int k = 0; k < 8; ++k) sum += k < n ? v[k] - one[0] : 0.0f;
    }
    if (!d.rms) m = one[0] + row_sum<4>(sum, part) / (float)d.N;
    for (int64_t j = 8 * threadIdx.x; j < d.N; j += 8 * kNormBlock) {
        const int n = valid8(d.N, j);
        again(j, n);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float e = k < n ? v[k] - m : 0.0f;
            sq = fmaf(e, e, sq);
            delta += e;
        }
    }
    row_sums<4>(sq, delta, parts);
    delta = d.rms ? 0.0f : delta / (float)d.N;
    const float rstd = row_rstd(sq / (float)d.N, delta, d.eps), shift = d.rms ? 0.0f : -delta * rstd;
    if (d.stats && threadIdx.x == 0) {
        d.stats[2 * row] = m + delta;
        d.stats[2 * row + 1] = rstd;
    }
    for (int64_t j = 8 * threadIdx.x; j < d.N; j += 8 * kNormBlock) {
        const int n = valid8(d.N, j);
        again(j, n);
        norm8<YF>(v, d, m, rstd, shift, row, j, n);
    }
}

template <bool XF, bool SF, bool YF>
static hipError_t norm_typed(const NormDesc& d, hipStream_t st) {
    if (d.N > 16384) {
        // a launch's threads are counted in 32 bits
        constexpr int64_t kLaunch = (int64_t(1) << 31) / kNormBlock;
        for (int64_t done = 0; done < d.M; done += kLaunch) {
            const unsigned blocks = (unsigned)(d.M - done < kLaunch ? d.M - done : kLaunch);
            hipLaunchKernelGGL((k_norm_long<XF, SF, YF>), dim3(blocks), dim3(kNormBlock), 0, st, d, done);
            const hipError_t e = hipGetLastError();
            if (e != hipSuccess) return e;
        }
        return hipSuccess;
    }
    const int W = d.N <= 1024 ? 1 : d.N <= 4096 ? 4 : 8;
    const auto k = d.N <= 512     ? k_norm<XF, SF, YF, 1, 1>
                   : d.N <= 1024  ? k_norm<XF, SF, YF, 1, 2>
                   : d.N <= 2048  ? k_norm<XF, SF, YF, 4, 1>
                   : d.N <= 4096  ? k_norm<XF, SF, YF, 4, 2>
                   : d.N <= 8192  ? k_norm<XF, SF, YF, 8, 2>
                   : d.N <= 12288 ? k_norm<XF, SF, YF, 8, 3>
                                  : k_norm<XF, SF, YF, 8, 4>;
    // sixteen waves to a compute unit, which then take rows in turn
    const int64_t groups = W == 1 ? (d.M + 3) / 4 : d.M, most = W == 8 ? 512 : 1024;
    const int64_t blocks = groups < most ? groups : most;
    hipLaunchKernelGGL(k, dim3((unsigned)blocks), dim3(W == 8 ? 512 : kNormBlock), 0, st, d, blocks);
    return hipGetLastError();
}

hipError_t launch_norm(const NormDesc& d, hipStream_t st) {
    if (d.x_f32) {
        if (d.sum_f32) return d.y_f32 ? norm_typed<true, true, true>(d, st) : norm_typed<true, true, false>(d, st);
        return d.y_f32 ? norm_typed<true, false, true>(d, st) : norm_typed<true, false, false>(d, st);
    }
    if (d.sum_f32) return d.y_f32 ? norm_typed<false, true, true>(d, st) : norm_typed<false, true, false>(d, st);
    return d.y_f32 ? norm_typed<false, false, true>(d, st) : norm_typed<false, false, false>(d, st);
}

// ---------------------------------------------------------------------------
// the gradient
// ---------------------------------------------------------------------------

constexpr int kGradBlock = 512, kGradWaves = kGradBlock / 64;

// k_norm_grad's waves: as many as its registers leave room for.
template <int C>
constexpr int kRowWaves = C == 1 ? 16 : 8;
static int grad_waves(int64_t N) {          // to a row
    return N <= 512 ? 1 : N <= 1024 ? 2 : N <= 2048 ? 4 : N <= 4096 || N > 8192 ? 8 : 16;
}
static int64_t grad_rows(int64_t N) { return N <= 8192 ? 16 / grad_waves(N) : 1; }      // at a time
// Workgroups of a gradient by M rows of N columns, each of which leaves a row of partial
// sums for the weight and one for the bias.
static int64_t grad_blocks(int64_t M, int64_t N) {
    const int64_t need = (M + grad_rows(N) - 1) / grad_rows(N);
    return need < 256 ? need : 256;
}
static int64_t up8(int64_t n) { return (n + 7) / 8 * 8; }

struct NormGradArgs {
    NormGradDesc d;
    int64_t ld_part;                // row length of partial sums
    int64_t parts;
    float* part;                    // [parts, 2, ld_part], or nullptr
};

// What a lane needs of eight columns of a row: h, g, and what they add to the row's sums
// and to the columns'.
template <bool DF, bool XF>
__device__ __forceinline__ void grad8(float dy[8], float h[8], const NormGradDesc& d, float mean, float rstd,
                                      int64_t row, int64_t j, int n) {
    load8<DF>(dy, d.dy, row * d.ld_dy + j, n);
    load8<XF>(h, d.x, row * d.ld_x + j, n);
#pragma unroll
    for (int k = 0; k < 8; ++k) h[k] = k < n ? (h[k] - mean) * rstd : 0.0f;
}
template <bool OF>
__device__ __forceinline__ void put_dx8(const float g[8], const float h[8], const NormGradDesc& d, float mg, float mgh,
                                        float rstd, int64_t row, int64_t j, int n) {
    float r[8], o[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) r[k] = 0.0f;
    if (d.res) load8<OF>(r, d.res, row * d.ld_res + j, n);
#pragma unroll
    for (int k = 0; k < 8; ++k) o[k] = fmaf(rstd, fmaf(-h[k], mgh, g[k] - mg), r[k]);
    store8<OF>(d.dx, row * d.ld_dx + j, o, n);
}

// W waves to a row of at most 512 W C columns; a workgroup takes every parts-th group of G
// rows and keeps the columns' sums in registers. The next rows' loads are under way while
// the sums of one are made, if C = 1 and at most one matrix is f32. Of C = 3 a row stays as
// it was loaded between its sums and dx, half the registers where it is bf16.
template <bool DF, bool XF, bool OF, int W, int C>
__global__ void __launch_bounds__(64 * kRowWaves<C>) k_norm_grad(const NormGradArgs a) {
    constexpr int G = kRowWaves<C> / W, kCols = 512 * W * C;
    constexpr bool kAhead = C == 1 && DF + XF + OF < 2;
    __shared__ float part[2][G][W][2];
    __shared__ float cols[G > 1 ? G * kCols : 1];
    const NormGradDesc& d = a.d;
    const int t = threadIdx.x % (64 * W), group = threadIdx.x / (64 * W);
    float aw[C][8], ab[C][8];
    int j[C], n[C];
    RawWeights w[C];
    Raw<DF> dy[C];
    Raw<XF> x[C];
    Raw<OF> res[C];
    float mean = 0.0f, rstd = 0.0f;
    const int64_t stride = a.parts * G;
    int64_t base = (int64_t)blockIdx.x * G;
    // where the next row's loads and this one's stores go, advanced instead of multiplied anew
    const int64_t row0 = base + group;
    int64_t at_dy = row0 * d.ld_dy, at_x = row0 * d.ld_x, at_res = row0 * d.ld_res, at_dx = row0 * d.ld_dx, at_stats = 2 * row0;
    const auto ask = [&](bool on) {
#pragma unroll
        for (int i = 0; i < C; ++i) {
            dy[i].load(d.dy, at_dy + j[i], on ? n[i] : 0);
            x[i].load(d.x, at_x + j[i], on ? n[i] : 0);
            if (d.res) res[i].load(d.res, at_res + j[i], on ? n[i] : 0);
        }
        mean = on ? d.stats[at_stats] : 0.0f;
        rstd = on ? d.stats[at_stats + 1] : 0.0f;
        at_dy += stride * d.ld_dy;
        at_x += stride * d.ld_x;
        at_res += stride * d.ld_res;
        at_stats += 2 * stride;
    };
#pragma unroll
    for (int i = 0; i < C; ++i) {
        j[i] = 8 * (t + 64 * W * i);
        n[i] = valid8(d.N, j[i]);
#pragma unroll
        for (int k = 0; k < 8; ++k) aw[i][k] = ab[i][k] = 0.0f;
    }
    if (kAhead) ask(row0 < d.M);
#pragma unroll
    for (int i = 0; i < C; ++i) w[i].load(d.w, j[i], n[i], kOnes);
    const float per_n = 1.0f / (float)d.N;
    int turn = 0;
    // The same turns for all waves: the last rows may be there for some groups only. Columns
    // that do not exist have dy and h 0, and so add nothing to the sums.
#pragma unroll 1
    for (; base < d.M; base += stride, turn ^= 1) {
        const int64_t row = base + group;
        if (!kAhead) ask(row < d.M);
        float sg = 0.0f, sgh = 0.0f;
        const float r = rstd, m = mean;
        Raw<DF> dy0[C];
        Raw<XF> x0[C];
        Raw<OF> add0[C];
        float g[8], h[8];
        const auto row8 = [&](int i) {          // dy w and h of a chunk
            dy0[i].get(g);
            x0[i].get(h);
#pragma unroll
            for (int k = 0; k < 8; ++k) h[k] = (h[k] - (n[i] > 0 ? m : 0.0f)) * r;
            if (n[i] > 0 && n[i] < 8)
#pragma unroll
                for (int k = 1; k < 8; ++k)
                    if (k >= n[i]) h[k] = 0.0f;
        };
#pragma unroll
        for (int i = 0; i < C; ++i) {
            dy0[i] = dy[i];
            x0[i] = x[i];
            if (d.res) add0[i] = res[i];
            row8(i);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                aw[i][k] = fmaf(g[k], h[k], aw[i][k]);
                ab[i][k] += g[k];
                g[k] *= w[i].get(k);
                sg += g[k];
                sgh = fmaf(g[k], h[k], sgh);
            }
            if (C > 1) {
                dy0[i].keep();
                x0[i].keep();
            }
        }
        if (kAhead) ask(row + stride < d.M);
        sg = wave_sum(sg);
        sgh = wave_sum(sgh);
        if constexpr (W > 1) {
            float(*const at)[2] = part[turn][group];
            if ((t & 63) == 0) {
                at[t >> 6][0] = sg;
                at[t >> 6][1] = sgh;
            }
            __syncthreads();
            sg = at[0][0];
            sgh = at[0][1];
#pragma unroll
            for (int q = 1; q < W; ++q) {
                sg += at[q][0];
                sgh += at[q][1];
            }
        }
        sg = d.rms ? 0.0f : sg * per_n;
        sgh *= per_n;
#pragma unroll
        for (int i = 0; i < C; ++i) {
            if (C > 1) {
                row8(i);
#pragma unroll
                for (int k = 0; k < 8; ++k) g[k] *= w[i].get(k);
            }
            float add[8];
            if (d.res) add0[i].get(add);
#pragma unroll
            for (int k = 0; k < 8; ++k) g[k] = fmaf(r, fmaf(-h[k], sgh, g[k] - sg), d.res ? add[k] : 0.0f);
            Raw<OF> out;
            out.set(g);
            out.store(d.dx, at_dx + j[i], row < d.M ? n[i] : 0);
        }
        at_dx += stride * d.ld_dx;
    }
    if (!a.part) return;
    float* const out = a.part + (int64_t)blockIdx.x * 2 * a.ld_part;
    if constexpr (G == 1) {
#pragma unroll
        for (int i = 0; i < C; ++i)
            if (j[i] < d.N) {
                store8_f(out + j[i], aw[i], 8);
                store8_f(out + a.ld_part + j[i], ab[i], 8);
            }
    } else {
        // the groups' sums in LDS, joined in order
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            __syncthreads();
#pragma unroll
            for (int i = 0; i < C; ++i)
                store8_f(cols + group * kCols + 8 * (t + 64 * W * i), s ? ab[i] : aw[i], 8);
            __syncthreads();
            for (int at = threadIdx.x; at < kCols && at < d.N; at += 64 * kRowWaves<C>) {
                float v = cols[at];
#pragma unroll
                for (int q = 1; q < G; ++q) v += cols[q * kCols + at];
                out[s * a.ld_part + at] = v;
            }
        }
    }
}

// Rows of any length: dx with the row read twice, and the columns' sums in a kernel of
// their own, which reads dy and x once more.
template <bool DF, bool XF, bool OF>
__global__ void __launch_bounds__(kGradBlock) k_norm_dx_long(const NormGradArgs a, int64_t first) {
    __shared__ float part[2][kGradWaves];
    const NormGradDesc& d = a.d;
    const int64_t row = first + blockIdx.x;
    const float mean = d.stats[2 * row], rstd = d.stats[2 * row + 1];
    float g[8], h[8], w[8], sg = 0.0f, sgh = 0.0f;
    const auto load = [&](int64_t j, int n) {
        weights8(w, d.w, j, n);
        grad8<DF, XF>(g, h, d, mean, rstd, row, j, n);
#pragma unroll
        for (int k = 0; k < 8; ++k) g[k] *= w[k];
    };
    for (int64_t j = 8 * threadIdx.x; j < d.N; j += 8 * kGradBlock) {
        load(j, valid8(d.N, j));
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            sg += g[k];
            sgh = fmaf(g[k], h[k], sgh);
        }
    }
    sg = d.rms ? 0.0f : row_sum<kGradWaves>(sg, part[0]) / (float)d.N;
    sgh = row_sum<kGradWaves>(sgh, part[1]) / (float)d.N;
    for (int64_t j = 8 * threadIdx.x; j < d.N; j += 8 * kGradBlock) {
        const int n = valid8(d.N, j);
        load(j, n);
        put_dx8<OF>(g, h, d, sg, sgh, rstd, row, j, n);
    }
}
template <bool DF, bool XF>
__global__ void __launch_bounds__(kGradBlock) k_norm_columns(const NormGradArgs a) {
    __shared__ float cols[kGradWaves * 512];
    const NormGradDesc& d = a.d;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t j0 = (int64_t)blockIdx.x * 512, j = j0 + 8 * lane;
    const int n = valid8(d.N, j);
    float aw[8], ab[8], g[8], h[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) aw[k] = ab[k] = 0.0f;
    for (int64_t row = (int64_t)blockIdx.y * kGradWaves + wave; row < d.M; row += a.parts * kGradWaves) {
        grad8<DF, XF>(g, h, d, d.stats[2 * row], d.stats[2 * row + 1], row, j, n);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            aw[k] = fmaf(g[k], h[k], aw[k]);
            ab[k] += g[k];
        }
    }
    float* const out = a.part + (int64_t)blockIdx.y * 2 * a.ld_part;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        __syncthreads();
        store8_f(cols + wave * 512 + 8 * lane, s ? ab : aw, 8);
        __syncthreads();
        if (j0 + threadIdx.x < d.N) {
            float v = cols[threadIdx.x];
#pragma unroll
            for (int q = 1; q < kGradWaves; ++q) v += cols[q * 512 + threadIdx.x];
            out[s * a.ld_part + j0 + threadIdx.x] = v;
        }
    }
}

// Joins the partial sums, in order: 64 columns of the weight's or the bias's (blockIdx.y)
// to a workgroup, each of its 16 waves every 16th row, then the waves'.
__global__ void __launch_bounds__(1024) k_norm_join(const NormGradArgs a) {
    __shared__ float s[16][64];
    const NormGradDesc& d = a.d;
    void* const to = blockIdx.y ? d.db : d.dw;
    if (!to) return;
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int64_t j = (int64_t)blockIdx.x * 64 + lane;
    float v = 0.0f;
    if (j < d.N) {
        const float* from = a.part + blockIdx.y * a.ld_part + j;
#pragma unroll 8
        for (int64_t r = wave; r < a.parts; r += 16) v += from[r * 2 * a.ld_part];
    }
    s[wave][lane] = v;
    __syncthreads();
    if (wave || j >= d.N) return;
#pragma unroll
    for (int q = 1; q < 16; ++q) v += s[q][lane];
    if (d.grad_f32) {
        float* o = static_cast<float*>(to) + j;
        *o = d.accumulate ? *o + v : v;
    } else {
        uint16_t* o = static_cast<uint16_t*>(to) + j;
        *o = bf_one(d.accumulate ? bf_f(*o) + v : v);
    }
}

size_t norm_ws_bytes(int64_t M, int64_t N) {
    return (size_t)grad_blocks(M, N) * 2 * (size_t)up8(N) * sizeof(float);
}

template <bool DF, bool XF, bool OF>
static hipError_t grad_typed(const NormGradArgs& a, hipStream_t st) {
    const NormGradDesc& d = a.d;
    // more chunks to a lane than three, or three of f32, spill
    if (d.N > (DF + XF + OF < 2 ? 12288 : 8192)) {
        constexpr int64_t kLaunch = (int64_t(1) << 31) / kGradBlock;
        // before dx, which may be written over dy or x
        if (a.part) {
            hipLaunchKernelGGL((k_norm_columns<DF, XF>), dim3((unsigned)((d.N + 511) / 512), (unsigned)a.parts),
                               dim3(kGradBlock), 0, st, a);
            const hipError_t e = hipGetLastError();
            if (e != hipSuccess) return e;
        }
        for (int64_t done = 0; done < d.M; done += kLaunch) {
            const unsigned blocks = (unsigned)(d.M - done < kLaunch ? d.M - done : kLaunch);
            hipLaunchKernelGGL((k_norm_dx_long<DF, XF, OF>), dim3(blocks), dim3(kGradBlock), 0, st, a, done);
            const hipError_t e = hipGetLastError();
            if (e != hipSuccess) return e;
        }
        return hipSuccess;
    }
    const auto k = d.N <= 512    ? k_norm_grad<DF, XF, OF, 1, 1>
                   : d.N <= 1024 ? k_norm_grad<DF, XF, OF, 2, 1>
                   : d.N <= 2048 ? k_norm_grad<DF, XF, OF, 4, 1>
                   : d.N <= 4096 ? k_norm_grad<DF, XF, OF, 8, 1>
                   : d.N <= 8192 ? k_norm_grad<DF, XF, OF, 16, 1>
                                 : k_norm_grad<DF, XF, OF, 8, DF + XF + OF < 2 ? 3 : 1>;      // or not reached
    hipLaunchKernelGGL(k, dim3((unsigned)a.parts), dim3(d.N <= 8192 ? 1024 : 512), 0, st, a);
    return hipGetLastError();
}

hipError_t launch_norm_grad(const NormGradDesc& d, hipStream_t st) {
    NormGradArgs a{};
    a.d = d;
    a.parts = grad_blocks(d.M, d.N);
    a.ld_part = up8(d.N);
    a.part = d.dw || d.db ? d.ws : nullptr;
    if (d.M > 0) {
        const int type = (d.dy_f32 ? 4 : 0) | (d.x_f32 ? 2 : 0) | (d.dx_f32 ? 1 : 0);
        static hipError_t (*const run[8])(const NormGradArgs&, hipStream_t) = {
            grad_typed<false, false, false>, grad_typed<false, false, true>, grad_typed<false, true, false>,
            grad_typed<false, true, true>,   grad_typed<true, false, false>, grad_typed<true, false, true>,
            grad_typed<true, true, false>,   grad_typed<true, true, true>};
        const hipError_t e = run[type](a, st);
        if (e != hipSuccess) return e;
    }
    if (!d.dw && !d.db) return hipSuccess;
    hipLaunchKernelGGL(k_norm_join, dim3((unsigned)((d.N + 63) / 64), 2), dim3(1024), 0, st, a);
    return hipGetLastError();
}

}  // namespace zk
