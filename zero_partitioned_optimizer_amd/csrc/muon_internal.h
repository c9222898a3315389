// muon_internal.h -- internal interface between the C entry points of the matrix step
// (muon_abi.cpp) and its gfx950 kernels (muon_kernels.hip, orth_kernels.hip). Not
// installed, not part of the ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "zero_muon.h"

namespace zk {

struct MomentumDesc {
    int64_t n;
    const void* grad;
    float* momentum;
    void* u;
    bool grad_f32, u_f32, nesterov;
    float mu;
    const zero_stats* stats;        // device, may be nullptr: its overflow flag stops the writes
};
hipError_t launch_momentum(const MomentumDesc& d, hipStream_t st);

struct UpdateDesc {
    int64_t n;
    float* p;
    const uint16_t* o;
    uint16_t* slot;                 // or nullptr
    float lr, decay;
    const zero_stats* stats;
};
hipError_t launch_update(const UpdateDesc& d, hipStream_t st);

struct OrthDesc {
    int64_t batch, rows, cols;
    const void* x;
    int64_t ld_x, stride_x;
    bool x_f32;
    uint16_t* o;
    int64_t ld_o, stride_o;
    int32_t steps;
    const double* coefficients;     // steps triples
    double eps;
    float scale;
    void* ws;                       // orth_ws_bytes
};
size_t orth_ws_bytes(int64_t batch, int64_t rows, int64_t cols);
hipError_t launch_orthogonalize(const OrthDesc& d, hipStream_t st);

}  // namespace zk
