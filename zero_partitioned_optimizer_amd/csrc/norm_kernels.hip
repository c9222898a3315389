// norm_kernels.hip -- the norm of a block's rows and its gradient:
//   forward   s = residual + x; y = (s - mean) rstd w + b
//   gradient  h = (x - mean) rstd, g = dy w: dx = residual_grad + rstd (g - mean(g) - h mean(g h)),
//             dw = [dw +] sum of dy h over the rows, db = [db +] sum of dy
// Bound by HBM: each matrix is read or written once. A row stays in registers between its
// sums and its outputs, eight columns to a lane and 16 bytes to a load.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "layer_device.h"

namespace zk {

template <bool F>
__device__ __forceinline__ void load8(float v[8], const void* p, int64_t at, int n) {
    if constexpr (F) load8_f(v, static_cast<const float*>(p) + at, n);
    else load8_bf(v, static_cast<const uint16_t*>(p) + at, n);
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

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int m = 32; m > 0; m >>= 1) v += __shfl_xor(v, m);
    return v;
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
__device__ __forceinline__ void norm8(const float v[8], const NormDesc& d, float mean, float rstd, int64_t row,
                                      int64_t j, int n) {
    float w[8], b[8], y[8];
    weights8(w, d.w, j, n);
#pragma unroll
    for (int k = 0; k < 8; ++k) b[k] = 0.0f;
    if (d.b) load8_bf(b, d.b + j, n);
#pragma unroll
    for (int k = 0; k < 8; ++k) y[k] = (v[k] - mean) * rstd * w[k] + b[k];
    store8<YF>(d.y, row * d.ld_y + j, y, n);
}

// W waves to a row of at most 512 W C columns, held in registers.
template <bool XF, bool SF, bool YF, int W, int C>
__global__ void __launch_bounds__(kNormBlock) k_norm(const NormDesc d, int64_t first) {
    __shared__ float part[2][4];
    const int t = W == 1 ? threadIdx.x & 63 : threadIdx.x;
    const int64_t row = first + (W == 1 ? (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6) : blockIdx.x);
    if (row >= d.M) return;
    float v[C][8], sum = 0.0f, sq = 0.0f, mean = 0.0f;
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const int64_t j = 8 * (t + 64 * W * i);
        const int n = valid8(d.N, j);
        sum8<XF, SF>(v[i], d, row, j, n);
    }
    if (!d.rms) {
#pragma unroll
        for (int i = 0; i < C; ++i)
#pragma unroll
            for (int k = 0; k < 8; ++k) sum += v[i][k];
        mean = row_sum<W>(sum, part[0]) / (float)d.N;
    }
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const int n = valid8(d.N, 8 * (t + 64 * W * i));
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float e = k < n ? v[i][k] - mean : 0.0f;
            sq = fmaf(e, e, sq);
        }
    }
    const float rstd = 1.0f / sqrtf(row_sum<W>(sq, part[1]) / (float)d.N + d.eps);
    if (d.stats && t == 0) {
        d.stats[2 * row] = mean;
        d.stats[2 * row + 1] = rstd;
    }
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const int64_t j = 8 * (t + 64 * W * i);
        const int n = valid8(d.N, j);
        if (n > 0) norm8<YF>(v[i], d, mean, rstd, row, j, n);
    }
}

// Rows of any length, read again for each sum (from the caches, up to some length).
template <bool XF, bool SF, bool YF>
__global__ void __launch_bounds__(kNormBlock) k_norm_long(const NormDesc d, int64_t first) {
    __shared__ float part[2][4];
    const int64_t row = first + blockIdx.x;
    float v[8], sum = 0.0f, sq = 0.0f, mean = 0.0f;
    const auto again = [&](int64_t j, int n) {
        if (d.res) load8<SF>(v, d.sum, row * d.ld_sum + j, n);
        else load8<XF>(v, d.x, row * d.ld_x + j, n);
    };
    for (int64_t j = 8 * threadIdx.x; j < d.N; j += 8 * kNormBlock) {
        sum8<XF, SF>(v, d, row, j, valid8(d.N, j));
#pragma unroll
        for (int k = 0; k < 8; ++k) sum += v[k];
    }
    if (!d.rms) mean = row_sum<4>(sum, part[0]) / (float)d.N;
    for (int64_t j = 8 * threadIdx.x; j < d.N; j += 8 * kNormBlock) {
        const int n = valid8(d.N, j);
        again(j, n);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float e = k < n ? v[k] - mean : 0.0f;
            sq = fmaf(e, e, sq);
        }
    }
    const float rstd = 1.0f / sqrtf(row_sum<4>(sq, part[1]) / (float)d.N + d.eps);
    if (d.stats && threadIdx.x == 0) {
        d.stats[2 * row] = mean;
        d.stats[2 * row + 1] = rstd;
    }
    for (int64_t j = 8 * threadIdx.x; j < d.N; j += 8 * kNormBlock) {
        const int n = valid8(d.N, j);
        again(j, n);
        norm8<YF>(v, d, mean, rstd, row, j, n);
    }
}

template <bool XF, bool SF, bool YF>
static hipError_t norm_typed(const NormDesc& d, hipStream_t st) {
    const bool one = d.N <= 1024;                       // a wave to a row, four rows to a workgroup
    const auto k = d.N <= 512     ? k_norm<XF, SF, YF, 1, 1>
                   : d.N <= 1024  ? k_norm<XF, SF, YF, 1, 2>
                   : d.N <= 2048  ? k_norm<XF, SF, YF, 4, 1>
                   : d.N <= 4096  ? k_norm<XF, SF, YF, 4, 2>
                   : d.N <= 8192  ? k_norm<XF, SF, YF, 4, 4>
                   : d.N <= 16384 ? k_norm<XF, SF, YF, 4, 8>
                                  : k_norm_long<XF, SF, YF>;
    const int64_t rows = one ? 4 : 1, all = (d.M + rows - 1) / rows;
    // a launch's threads are counted in 32 bits
    constexpr int64_t kLaunch = (int64_t(1) << 31) / kNormBlock;
    for (int64_t done = 0; done < all; done += kLaunch) {
        const unsigned blocks = (unsigned)(all - done < kLaunch ? all - done : kLaunch);
        hipLaunchKernelGGL(k, dim3(blocks), dim3(kNormBlock), 0, st, d, done * rows);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
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

// Workgroups of a gradient by M rows of N columns, each of which leaves a row of partial
// sums for the weight and one for the bias.
static int64_t grad_rows(int64_t N) { return N <= 1024 ? kGradWaves : 1; }       // at a time
static int64_t grad_blocks(int64_t M, int64_t N) {
    const int64_t need = (M + grad_rows(N) - 1) / grad_rows(N);
    return need < 512 ? need : 512;
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

// W waves to a row of at most 512 W C columns; a workgroup takes every parts-th group of
// 8 / W rows and keeps the columns' sums in registers.
template <bool DF, bool XF, bool OF, int W, int C>
__global__ void __launch_bounds__(kGradBlock) k_norm_grad(const NormGradArgs a) {
    constexpr int G = kGradWaves / W, kCols = 512 * W * C;
    __shared__ float part[2][2][kGradWaves];
    __shared__ float cols[G > 1 ? G * kCols : 1];
    const NormGradDesc& d = a.d;
    const int t = W == 1 ? threadIdx.x & 63 : threadIdx.x, group = W == 1 ? threadIdx.x >> 6 : 0;
    float w[C][8], aw[C][8], ab[C][8];
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const int64_t j = 8 * (t + 64 * W * i);
        weights8(w[i], d.w, j, valid8(d.N, j));
#pragma unroll
        for (int k = 0; k < 8; ++k) aw[i][k] = ab[i][k] = 0.0f;
    }
    int turn = 0;
    for (int64_t row = (int64_t)blockIdx.x * G + group; row < d.M; row += a.parts * G, turn ^= 1) {
        const float mean = d.stats[2 * row], rstd = d.stats[2 * row + 1];
        float g[C][8], h[C][8], sg = 0.0f, sgh = 0.0f;
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const int64_t j = 8 * (t + 64 * W * i);
            grad8<DF, XF>(g[i], h[i], d, mean, rstd, row, j, valid8(d.N, j));
        }
#pragma unroll
        for (int i = 0; i < C; ++i)
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                aw[i][k] = fmaf(g[i][k], h[i][k], aw[i][k]);
                ab[i][k] += g[i][k];
                g[i][k] *= w[i][k];
                sg += g[i][k];
                sgh = fmaf(g[i][k], h[i][k], sgh);
            }
        sg = d.rms ? 0.0f : row_sum<W>(sg, part[turn][0]) / (float)d.N;
        sgh = row_sum<W>(sgh, part[turn][1]) / (float)d.N;
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const int64_t j = 8 * (t + 64 * W * i);
            const int n = valid8(d.N, j);
            if (n > 0) put_dx8<OF>(g[i], h[i], d, sg, sgh, rstd, row, j, n);
        }
    }
    if (!a.part) return;
    float* const out = a.part + (int64_t)blockIdx.x * 2 * a.ld_part;
    if constexpr (G == 1) {
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const int64_t j = 8 * (t + 64 * W * i);
            if (j < d.N) {
                store8_f(out + j, aw[i], 8);
                store8_f(out + a.ld_part + j, ab[i], 8);
            }
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
            for (int j = threadIdx.x; j < kCols && j < d.N; j += kGradBlock) {
                float v = cols[j];
#pragma unroll
                for (int q = 1; q < G; ++q) v += cols[q * kCols + j];
                out[s * a.ld_part + j] = v;
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
    if (d.N > 16384) {
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
                   : d.N <= 1024 ? k_norm_grad<DF, XF, OF, 1, 2>
                   : d.N <= 4096 ? k_norm_grad<DF, XF, OF, 8, 1>
                   : d.N <= 8192 ? k_norm_grad<DF, XF, OF, 8, 2>
                                 : k_norm_grad<DF, XF, OF, 8, 4>;
    hipLaunchKernelGGL(k, dim3((unsigned)a.parts), dim3(kGradBlock), 0, st, a);
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
