// dropout_kernels.hip -- dropout alone: y = residual + D(x), and the gradient of
// dropout behind an activation, dz = D'(dy) * act'(z). The mask is a function of
// (seed, offset, row, column) and is never stored.
//
// Bound by HBM: each input is read once and the output written once. A thread
// takes eight consecutive columns of one row, 16 bytes of bf16 and one draw of the
// generator: 16384 x 11008 f32 in and out 246 us, 5.9 TB/s; GELU's gradient over
// 8192 x 11008 (three bf16 matrices) 105 us, 5.2 TB/s. Two or four groups to a
// thread were no faster.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "layer_device.h"

namespace zk {

constexpr int kDropBlock = 256;

struct DropoutArgs {
    DropoutDesc d;
    int64_t first;                  // the launch's first thread among all
    int64_t groups;                 // groups of eight columns per row
    double inv_groups;
};

template <bool XF, bool YF, bool GRAD>
__global__ void __launch_bounds__(kDropBlock) k_dropout(const DropoutArgs g) {
    const DropoutDesc& d = g.d;
    const int64_t id = g.first + (int64_t)blockIdx.x * kDropBlock + threadIdx.x;
    // row = id / groups from the reciprocal, corrected by one (ids stay below 2^51)
    int64_t row = (int64_t)((double)id * g.inv_groups);
    if (row * g.groups > id) --row;
    else if ((row + 1) * g.groups <= id) ++row;
    if (row >= d.M) return;
    const int64_t c = id - row * g.groups, j = 8 * c;
    const int n = d.N - j < 8 ? (int)(d.N - j) : 8;
    float v[8], t[8];
    if constexpr (XF) load8_f(v, static_cast<const float*>(d.x) + row * d.ld_x + j, n);
    else load8_bf(v, static_cast<const uint16_t*>(d.x) + row * d.ld_x + j, n);
    if constexpr (GRAD) {
        if (d.z) {
            load8_bf(t, d.z + row * d.ld_z + j, n);
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] *= act_slope(d.act, t[k]);
        }
    } else if (d.res) {
        if constexpr (YF) load8_f(t, static_cast<const float*>(d.res) + row * d.ld_res + j, n);
        else load8_bf(t, static_cast<const uint16_t*>(d.res) + row * d.ld_res + j, n);
    }
    if (d.drop.thr) drop8(v, d.drop, drop_offset(d.drop), (uint32_t)row, (uint32_t)c);
    if constexpr (!GRAD) {
        if (d.res)
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] += t[k];
    }
    if constexpr (YF) store8_f(static_cast<float*>(d.y) + row * d.ld_y + j, v, n);
    else store8_bf(static_cast<uint16_t*>(d.y) + row * d.ld_y + j, v, n);
}

template <bool XF, bool YF>
static void launch_typed(const DropoutArgs& g, bool grad, unsigned blocks, hipStream_t st) {
    if (grad) hipLaunchKernelGGL((k_dropout<XF, YF, true>), dim3(blocks), dim3(kDropBlock), 0, st, g);
    else hipLaunchKernelGGL((k_dropout<XF, YF, false>), dim3(blocks), dim3(kDropBlock), 0, st, g);
}

hipError_t launch_dropout(const DropoutDesc& d, bool grad, hipStream_t st) {
    DropoutArgs g{};
    g.d = d;
    g.groups = (d.N + 7) / 8;
    g.inv_groups = 1.0 / (double)g.groups;
    const int64_t all = (d.M * g.groups + kDropBlock - 1) / kDropBlock;
    // a launch's threads are counted in 32 bits
    constexpr int64_t kLaunch = (int64_t(1) << 31) / kDropBlock;
    for (int64_t done = 0; done < all; done += kLaunch) {
        const unsigned blocks = (unsigned)(all - done < kLaunch ? all - done : kLaunch);
        g.first = done * kDropBlock;
        if (d.x_f32 && d.y_f32) launch_typed<true, true>(g, grad, blocks, st);
        else if (d.x_f32) launch_typed<true, false>(g, grad, blocks, st);
        else if (d.y_f32) launch_typed<false, true>(g, grad, blocks, st);
        else launch_typed<false, false>(g, grad, blocks, st);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace zk
