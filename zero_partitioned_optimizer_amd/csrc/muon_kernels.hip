// muon_kernels.hip -- the elementwise ends of the matrix step:
//   momentum  m' = mu m + g;  u = g + mu m' or m'
//   update    p' = p decay - lr o;  slot = bf16(p')
// Bound by HBM: each array is read or written once, f32 16 bytes to a lane, four elements to
// a thread (eight, or two or four groups of four, were 3 to 15% slower). Loads do not stay in
// the caches; stores do where all outputs fit the Infinity Cache, for whoever reads them next
// (GPT-2 small's shard of 15.6M: momentum from f32 to bf16 34.5 us, update 31.3 us), and
// not beyond (a Llama-7B shaped layer's 202M elements 451 us, 6.3 TB/s, and 375 us, 6.5 TB/s;
// 511 and 431 with cached stores, 492 and 417 with cached loads too).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "layer_device.h"
#include "muon_internal.h"

namespace zk {

constexpr int kFlatBlock = 256;
typedef uint32_t v2u __attribute__((ext_vector_type(2)));
typedef v2u v2u_any __attribute__((aligned(2)));

// Up to four elements (n of them) at any element's address.
__device__ __forceinline__ v4f load4(const float* p, int n) {
    if (n >= 4) return __builtin_nontemporal_load(reinterpret_cast<const v4f_any*>(p));
    v4f v = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int k = 0; k < 3; ++k)
        if (k < n) v[k] = p[k];
    return v;
}
__device__ __forceinline__ v4f load4(const uint16_t* p, int n) {
    if (n >= 4) {
        const v2u w = __builtin_nontemporal_load(reinterpret_cast<const v2u_any*>(p));
        return v4f{bf_lo(w[0]), bf_hi(w[0]), bf_lo(w[1]), bf_hi(w[1])};
    }
    v4f v = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int k = 0; k < 3; ++k)
        if (k < n) v[k] = bf_f(p[k]);
    return v;
}
template <bool CACHED>
__device__ __forceinline__ void store4(float* p, v4f v, int n) {
    if (n >= 4) {
        if constexpr (CACHED) *reinterpret_cast<v4f_any*>(p) = v;
        else __builtin_nontemporal_store(v, reinterpret_cast<v4f_any*>(p));
    } else {
#pragma unroll
        for (int k = 0; k < 3; ++k)
            if (k < n) p[k] = v[k];
    }
}
template <bool CACHED>
__device__ __forceinline__ void store4(uint16_t* p, v4f v, int n) {
    if (n >= 4) {
        const v2u w = {bf_pack(v[0], v[1]), bf_pack(v[2], v[3])};
        if constexpr (CACHED) *reinterpret_cast<v2u_any*>(p) = w;
        else __builtin_nontemporal_store(w, reinterpret_cast<v2u_any*>(p));
    } else {
#pragma unroll
        for (int k = 0; k < 3; ++k)
            if (k < n) p[k] = bf_one(v[k]);
    }
}

template <typename G, typename U, bool CACHED>
__global__ void __launch_bounds__(kFlatBlock) k_momentum(const MomentumDesc d, int64_t first) {
    const int64_t i = first + 4 * ((int64_t)blockIdx.x * kFlatBlock + threadIdx.x);
    if (i >= d.n || (d.stats && d.stats->overflow)) return;
    const int n = d.n - i < 4 ? (int)(d.n - i) : 4;
    const v4f g = load4(static_cast<const G*>(d.grad) + i, n), old = load4(d.momentum + i, n);
    v4f m, u;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        m[k] = d.mu * old[k] + g[k];
        u[k] = d.nesterov ? g[k] + d.mu * m[k] : m[k];
    }
    store4<CACHED>(d.momentum + i, m, n);
    store4<CACHED>(static_cast<U*>(d.u) + i, u, n);
}

template <bool CACHED>
__global__ void __launch_bounds__(kFlatBlock) k_update(const UpdateDesc d, int64_t first) {
    const int64_t i = first + 4 * ((int64_t)blockIdx.x * kFlatBlock + threadIdx.x);
    if (i >= d.n || (d.stats && d.stats->overflow)) return;
    const int n = d.n - i < 4 ? (int)(d.n - i) : 4;
    const v4f o = load4(d.o + i, n);
    v4f p = load4(d.p + i, n);
#pragma unroll
    for (int k = 0; k < 4; ++k) p[k] = p[k] * d.decay - d.lr * o[k];
    store4<CACHED>(d.p + i, p, n);
    if (d.slot) store4<CACHED>(d.slot + i, p, n);
}

// Whether n elements of so many bytes fit the Infinity Cache of 256 MB.
static bool cached(int64_t n, int bytes) { return n <= (int64_t(256) << 20) / bytes; }

// A launch's threads are counted in 32 bits.
template <typename Desc>
static hipError_t by_element(void (*k)(const Desc, int64_t), const Desc& d, hipStream_t st) {
    constexpr int64_t kLaunch = int64_t(1) << 32;
    for (int64_t done = 0; done < d.n; done += kLaunch) {
        const int64_t left = d.n - done < kLaunch ? d.n - done : kLaunch;
        hipLaunchKernelGGL(k, dim3((unsigned)((left + 4 * kFlatBlock - 1) / (4 * kFlatBlock))), dim3(kFlatBlock), 0, st,
                           d, done);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

template <bool CACHED>
static hipError_t momentum(const MomentumDesc& d, hipStream_t st) {
    return by_element(d.grad_f32 ? (d.u_f32 ? k_momentum<float, float, CACHED> : k_momentum<float, uint16_t, CACHED>)
                                 : (d.u_f32 ? k_momentum<uint16_t, float, CACHED> : k_momentum<uint16_t, uint16_t, CACHED>),
                      d, st);
}
hipError_t launch_momentum(const MomentumDesc& d, hipStream_t st) {
    return cached(d.n, d.u_f32 ? 8 : 6) ? momentum<true>(d, st) : momentum<false>(d, st);
}
hipError_t launch_update(const UpdateDesc& d, hipStream_t st) {
    return by_element(cached(d.n, d.slot ? 6 : 4) ? k_update<true> : k_update<false>, d, st);
}

}  // namespace zk
