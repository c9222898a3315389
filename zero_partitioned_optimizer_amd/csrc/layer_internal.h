// layer_internal.h -- internal interface between the C entry points of the layer
// operators (layer_abi.cpp) and their gfx950 kernels (linear_kernels.hip,
// dropout_kernels.hip, norm_kernels.hip). Not installed, not part of the ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "zero_layer.h"

namespace zk {

// Dropout as the kernels take it: element (i, j) is dropped when its 16-bit draw
// is below thr, and kept elements are multiplied by scale; thr = 0 is no dropout.
struct Drop {
    uint32_t thr;
    float scale;                    // 65536 / (65536 - thr), rounded once
    uint32_t k0, k1;                // the seed's two halves: the generator's key
    uint64_t offset;
    const int64_t* counter;         // device, added to offset; may be nullptr
};

// One product C[p, q] = sum_r A(p, r) B(q, r) with an epilogue. An operand either
// holds its outer index in rows (element (o, r) at o * ld + r) or, "reduced rows",
// the reduction index in rows (element (o, r) at r * ld + o).
enum Epilogue { kEpiForward = 0, kEpiGradInput = 1, kEpiGradWeight = 2 };

struct ProductDesc {
    const uint16_t* a;
    const uint16_t* b;
    int64_t lda, ldb;
    bool ta, tb;                    // reduced rows
    int64_t P, Q, R;
    Epilogue epi;
    void* out;                      // [P, Q], bf16 or f32
    int64_t ld_out;
    bool out_f32;
    const uint16_t* bias;           // forward: [Q] or nullptr
    const void* res;                // forward: the residual; weight gradient: the old values
    int64_t ld_res;                 // (both of out's type), or nullptr
    const uint16_t* z_in;           // gradient by input: pre-activation [P, Q] or nullptr
    uint16_t* z_out;                // forward: pre-activation to store, or nullptr
    int64_t ld_z;
    int32_t act;
    Drop drop;
    void* bias_out;                 // weight gradient: the bias's, of out's type, or nullptr
    bool bias_of_a;                 // ... the sums over r of a, or of b
    bool bias_add;                  // ... added to what it holds
    float* ws;                      // product_ws_bytes
    float* ws_sums;                 // sums_ws_bytes
};

// Workspace bytes that launch_product needs for a product of these sizes, and
// for the bias gradient beside it.
size_t product_ws_bytes(int64_t P, int64_t Q, int64_t R, bool ta, bool tb);
// The same for one call, operand a with outer rows: 0 where the operands' alignment lets
// it do without, as one token's usually does.
size_t product_ws_needed(const uint16_t* a, int64_t lda, const uint16_t* b, int64_t ldb, int64_t P, int64_t Q,
                         int64_t R, bool tb);
size_t sums_ws_bytes(int64_t P, int64_t Q, int64_t R, bool of_a);
// Whether the output's tiles fit one launch, whose threads a 32-bit count holds.
inline bool product_fits(int64_t P, int64_t Q) {
    constexpr int64_t kSide = int64_t(1) << 29, kTiles = int64_t(1) << 23;
    return P <= kSide && Q <= kSide && ((P + 127) / 128) * ((Q + 127) / 128) <= kTiles;
}
hipError_t launch_product(const ProductDesc& d, hipStream_t st);

// Elementwise over [M, N]: y = res + D(x), or (grad) y = D'(x) * act'(z).
struct DropoutDesc {
    int64_t M, N;
    const void* x;
    int64_t ld_x;
    bool x_f32;
    const void* res;                // of y's type, or nullptr
    int64_t ld_res;
    const uint16_t* z;              // or nullptr
    int64_t ld_z;
    int32_t act;
    void* y;
    int64_t ld_y;
    bool y_f32;
    Drop drop;
};
hipError_t launch_dropout(const DropoutDesc& d, bool grad, hipStream_t st);

// A norm of each row of [M, N], and its gradient. `_f32` flags: f32 in place of bf16.
struct NormDesc {
    int64_t M, N;
    const void* x;
    const void* res;                // of sum's type, or nullptr (then sum is too)
    void* sum;
    void* y;
    int64_t ld_x, ld_res, ld_sum, ld_y;
    bool x_f32, sum_f32, y_f32, rms;
    float eps;
    const uint16_t* w;              // or nullptr: ones
    const uint16_t* b;              // or nullptr: zeros
    float* stats;                   // [M, 2], or nullptr
};
hipError_t launch_norm(const NormDesc& d, hipStream_t st);

struct NormGradDesc {
    int64_t M, N;
    const void* dy;
    const void* x;
    const void* res;                // of dx's type, or nullptr
    void* dx;
    int64_t ld_dy, ld_x, ld_res, ld_dx;
    bool dy_f32, x_f32, dx_f32, rms;
    const uint16_t* w;              // or nullptr: ones
    const float* stats;
    void* dw;                       // or nullptr, both
    void* db;
    bool grad_f32, accumulate;
    float* ws;                      // norm_ws_bytes, where dw or db is wanted
};
size_t norm_ws_bytes(int64_t M, int64_t N);
hipError_t launch_norm_grad(const NormGradDesc& d, hipStream_t st);

}  // namespace zk
