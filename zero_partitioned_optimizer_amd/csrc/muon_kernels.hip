// muon_kernels.hip -- the elementwise ends of the matrix step:
//   momentum  m' = mu m + g;  u = g + mu m' or m'
//   update    p' = p decay - lr o;  slot = bf16(p')
// Bound by HBM: each array is read or written once. A thread takes eight elements.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "layer_device.h"
#include "muon_internal.h"

namespace zk {

constexpr int kFlatBlock = 256;

template <bool GF, bool UF>
__global__ void __launch_bounds__(kFlatBlock) k_momentum(const MomentumDesc d, int64_t first) {
    const int64_t i = first + 8 * ((int64_t)blockIdx.x * kFlatBlock + threadIdx.x);
    if (i >= d.n || (d.stats && d.stats->overflow)) return;
    const int n = d.n - i < 8 ? (int)(d.n - i) : 8;
    float g[8], m[8];
    if constexpr (GF) load8_f(g, static_cast<const float*>(d.grad) + i, n);
    else load8_bf(g, static_cast<const uint16_t*>(d.grad) + i, n);
    load8_f(m, d.momentum + i, n);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        m[k] = d.mu * m[k] + g[k];
        g[k] = d.nesterov ? g[k] + d.mu * m[k] : m[k];
    }
    store8_f(d.momentum + i, m, n);
    if constexpr (UF) store8_f(static_cast<float*>(d.u) + i, g, n);
    else store8_bf(static_cast<uint16_t*>(d.u) + i, g, n);
}

__global__ void __launch_bounds__(kFlatBlock) k_update(const UpdateDesc d, int64_t first) {
    const int64_t i = first + 8 * ((int64_t)blockIdx.x * kFlatBlock + threadIdx.x);
    if (i >= d.n || (d.stats && d.stats->overflow)) return;
    const int n = d.n - i < 8 ? (int)(d.n - i) : 8;
    float p[8], o[8];
    load8_f(p, d.p + i, n);
    load8_bf(o, d.o + i, n);
#pragma unroll
    for (int k = 0; k < 8; ++k) p[k] = p[k] * d.decay - d.lr * o[k];
    store8_f(d.p + i, p, n);
    if (d.slot) store8_bf(d.slot + i, p, n);
}

// A launch's threads are counted in 32 bits.
template <typename Desc>
static hipError_t by_element(void (*k)(const Desc, int64_t), const Desc& d, hipStream_t st) {
    constexpr int64_t kLaunch = int64_t(1) << 33;
    for (int64_t done = 0; done < d.n; done += kLaunch) {
        const int64_t left = d.n - done < kLaunch ? d.n - done : kLaunch;
        hipLaunchKernelGGL(k, dim3((unsigned)((left + 8 * kFlatBlock - 1) / (8 * kFlatBlock))), dim3(kFlatBlock), 0, st,
                           d, done);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

hipError_t launch_momentum(const MomentumDesc& d, hipStream_t st) {
    return by_element(d.grad_f32 ? (d.u_f32 ? k_momentum<true, true> : k_momentum<true, false>)
                                 : (d.u_f32 ? k_momentum<false, true> : k_momentum<false, false>),
                      d, st);
}
hipError_t launch_update(const UpdateDesc& d, hipStream_t st) { return by_element(k_update, d, st); }

}  // namespace zk
