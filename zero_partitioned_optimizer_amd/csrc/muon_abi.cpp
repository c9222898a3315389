// muon_abi.cpp -- the C entry points of the matrix step (momentum, orthogonalisation,
// update): argument validation and the descriptors of their kernels, which live in
// muon_kernels.hip and orth_kernels.hip.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "abi_checks.h"
#include "muon_internal.h"
#include "zero_internal.h"
#include "zero_muon.h"

namespace {

using namespace zl;

static_assert(sizeof(zero_muon_momentum_args) == 64 && sizeof(zero_muon_update_args) == 56 &&
                  sizeof(zero_orthogonalize_args) == 120,
              "the argument blocks of the ABI");

constexpr int64_t kMaxFlat = int64_t(1) << 40;
constexpr int64_t kMaxSmall = int64_t(1) << 15, kMaxLarge = int64_t(1) << 20, kMaxStride = int64_t(1) << 50;
constexpr int32_t kMaxSteps = 64;
// 2^13 times what a step rounds, 2^-22 of the norm or so, is 2e-3 of it. Seven steps of the default
// coefficients are 5,752; eight leave 6e-3 on a matrix of rank 1, and ten 7e-2 (fp32 operations 2e-3
// and 3e-2).
constexpr double kMaxGain = 8192.0;

int check_n(const char* fn, int64_t n) {
    if (n >= 0 && n <= kMaxFlat) return ZERO_OK;
    set_error("%s: n=%lld outside [0, 2^40]", fn, (long long)n);
    return ZERO_E_RANGE;
}

int check_value(const char* fn, const char* name, double v, double least, double most, bool open = false) {
    if (v >= least && (open ? v < most : v <= most)) return ZERO_OK;        // not for a NaN
    set_error("%s: %s=%g outside [%g, %g%c", fn, name, v, least, most, open ? ')' : ']');
    return ZERO_E_INVAL;
}

Mat flat(const char* name, const void* p, int64_t n, int64_t esize, bool written, bool optional = false) {
    return Mat{name, p, 1, n, n, esize, written, false, optional};
}

bool sides_fit(int64_t batch, int64_t rows, int64_t cols) {
    const int64_t small = rows < cols ? rows : cols, large = rows < cols ? cols : rows;
    return batch >= 0 && batch <= kMaxDim && small >= 0 && small <= kMaxSmall && large <= kMaxLarge;
}

// From a stack's first element to behind its last.
int64_t extent(int64_t batch, int64_t rows, int64_t cols, int64_t ld, int64_t stride) {
    return (batch - 1) * (batch > 1 ? stride : 0) + (rows - 1) * ld + cols;
}

int check_stack(const char* fn, const char* name, int64_t batch, int64_t rows, int64_t cols, int64_t ld, int64_t stride) {
    if (ld < cols || ld > kMaxLd) {
        set_error("%s: ld of %s is %lld, outside [%lld, 2^40]", fn, name, (long long)ld, (long long)cols);
        return ZERO_E_RANGE;
    }
    const int64_t least = (rows - 1) * ld + cols;       // below 2^61
    if (batch > 1 && (stride < least || stride > kMaxStride)) {
        set_error("%s: batch stride of %s is %lld, outside [%lld, 2^50]", fn, name, (long long)stride, (long long)least);
        return ZERO_E_RANGE;
    }
    if (batch > 1 && (batch - 1) > (int64_t(1) << 60) / stride) {
        set_error("%s: %lld matrices of %s, %lld apart, leave the address space", fn, (long long)batch, name,
                  (long long)stride);
        return ZERO_E_RANGE;
    }
    return ZERO_OK;
}

}  // namespace

extern "C" {

int zero_muon_momentum(const zero_muon_momentum_args* args, void* stream) {
    static const char* fn = "zero_muon_momentum";
    if (!args) {
        set_error("%s: args is NULL", fn);
        return ZERO_E_INVAL;
    }
    const zero_muon_momentum_args& a = *args;
    int rc;
    if ((rc = check_n(fn, a.n)) || (rc = check_type(fn, "grad_dtype", a.grad_dtype)) ||
        (rc = check_type(fn, "u_dtype", a.u_dtype)) || (rc = check_value(fn, "mu", a.mu, 0.0, 1.0, true)))
        return rc;
    if (a.n == 0) return ZERO_OK;
    Mat m[] = {flat("grad", a.grad, a.n, size_of(a.grad_dtype), false),
               flat("momentum", a.momentum, a.n, 4, true), flat("u", a.u, a.n, size_of(a.u_dtype), true),
               flat("stats_dev", a.stats_dev, sizeof(zero_stats) / 8, 8, false, true)};
    m[0].elementwise = m[2].elementwise = true;
    if ((rc = check_mats(fn, m, 4))) return rc;
    zk::MomentumDesc d{};
    d.n = a.n;
    d.grad = a.grad;
    d.momentum = a.momentum;
    d.u = a.u;
    d.grad_f32 = a.grad_dtype == ZERO_F32;
    d.u_f32 = a.u_dtype == ZERO_F32;
    d.nesterov = a.nesterov != 0;
    d.mu = (float)a.mu;
    d.stats = a.stats_dev;
    return hip_error(zk::launch_momentum(d, static_cast<hipStream_t>(stream)), fn);
}

int zero_muon_update(const zero_muon_update_args* args, void* stream) {
    static const char* fn = "zero_muon_update";
    if (!args) {
        set_error("%s: args is NULL", fn);
        return ZERO_E_INVAL;
    }
    const zero_muon_update_args& a = *args;
    int rc;
    if ((rc = check_n(fn, a.n)) || (rc = check_value(fn, "lr", a.lr, 0.0, 1e30)) ||
        (rc = check_value(fn, "weight_decay", a.weight_decay, 0.0, 1e30)))
        return rc;
    if (a.n == 0) return ZERO_OK;
    const Mat m[] = {flat("p", a.p, a.n, 4, true), flat("o", a.o, a.n, 2, false),
                     flat("slot_bf16", a.slot_bf16, a.n, 2, true, true),
                     flat("stats_dev", a.stats_dev, sizeof(zero_stats) / 8, 8, false, true)};
    if ((rc = check_mats(fn, m, 4))) return rc;
    zk::UpdateDesc d{};
    d.n = a.n;
    d.p = a.p;
    d.o = a.o;
    d.slot = a.slot_bf16;
    d.lr = (float)a.lr;
    d.decay = (float)(1.0 - a.lr * a.weight_decay);
    d.stats = a.stats_dev;
    return hip_error(zk::launch_update(d, static_cast<hipStream_t>(stream)), fn);
}

size_t zero_orthogonalize_workspace_bytes(int64_t batch, int64_t rows, int64_t cols) {
    return sides_fit(batch, rows, cols) ? zk::orth_ws_bytes(batch, rows, cols) : 0;
}

int zero_orthogonalize(const zero_orthogonalize_args* args, void* stream) {
    static const char* fn = "zero_orthogonalize";
    static const double kDefault[3] = {3.4445, -4.7750, 2.0315};
    if (!args) {
        set_error("%s: args is NULL", fn);
        return ZERO_E_INVAL;
    }
    const zero_orthogonalize_args& a = *args;
    int rc;
    if (!sides_fit(a.batch, a.rows, a.cols)) {
        set_error("%s: %lld matrices of %lld x %lld: batch outside [0, 2^31 - 1], the smaller side [0, 2^15] or "
                  "the larger [0, 2^20]", fn, (long long)a.batch, (long long)a.rows, (long long)a.cols);
        return ZERO_E_RANGE;
    }
    if (a.steps < 1 || a.steps > kMaxSteps) {
        set_error("%s: steps=%d outside [1, %d]", fn, (int)a.steps, (int)kMaxSteps);
        return ZERO_E_INVAL;
    }
    if ((rc = check_type(fn, "x_dtype", a.x_dtype)) || (rc = check_value(fn, "eps", a.eps, 1e-30, 1e30)) ||
        (rc = check_value(fn, "scale", a.scale, -1e4, 1e4)))
        return rc;
    double coefficients[3 * kMaxSteps];
    for (int k = 0; k < 3 * a.steps; ++k) {
        coefficients[k] = a.coefficients ? a.coefficients[k] : kDefault[k % 3];
        if ((rc = check_value(fn, "a coefficient", coefficients[k], -1e4, 1e4))) return rc;
    }
    double gain = 1.0;
    for (int k = 0; k < a.steps; ++k) gain *= fmax(1.0, fabs(coefficients[3 * k]));
    if (gain > kMaxGain) {
        set_error("%s: the first coefficients of %d steps multiply to %g, above %g: roundings would grow by that", fn,
                  (int)a.steps, gain, kMaxGain);
        return ZERO_E_INVAL;
    }
    if (a.batch == 0 || a.rows == 0 || a.cols == 0) return ZERO_OK;
    if ((rc = check_stack(fn, "x", a.batch, a.rows, a.cols, a.ld_x, a.stride_x)) ||
        (rc = check_stack(fn, "o", a.batch, a.rows, a.cols, a.ld_o, a.stride_o)))
        return rc;
    const size_t need = zk::orth_ws_bytes(a.batch, a.rows, a.cols);
    const Mat m[] = {flat("x", a.x, extent(a.batch, a.rows, a.cols, a.ld_x, a.stride_x), size_of(a.x_dtype), false),
                     flat("o", a.o, extent(a.batch, a.rows, a.cols, a.ld_o, a.stride_o), 2, true),
                     ws_mat(a.workspace_dev, need)};
    if ((rc = check_ws(fn, a.workspace_dev, a.ws_bytes, need))) return rc;
    for (int i = 0; i < 2; ++i) {
        if (!m[i].p) {
            set_error("%s: %s is NULL", fn, m[i].name);
            return ZERO_E_INVAL;
        }
        if (reinterpret_cast<uintptr_t>(m[i].p) % (uintptr_t)m[i].esize != 0) {
            set_error("%s: %s=%p is not aligned to its %d-byte elements", fn, m[i].name, m[i].p, (int)m[i].esize);
            return ZERO_E_ALIGN;
        }
        for (int k = i + 1; k < 3; ++k)
            if (meet(m[i], m[k])) {
                set_error("%s: %s and %s overlap", fn, m[i].name, m[k].name);
                return ZERO_E_INVAL;
            }
    }
    zk::OrthDesc d{};
    d.batch = a.batch;
    d.rows = a.rows;
    d.cols = a.cols;
    d.x = a.x;
    d.ld_x = a.ld_x;
    d.stride_x = a.batch > 1 ? a.stride_x : 0;
    d.x_f32 = a.x_dtype == ZERO_F32;
    d.o = a.o;
    d.ld_o = a.ld_o;
    d.stride_o = a.batch > 1 ? a.stride_o : 0;
    d.steps = a.steps;
    d.coefficients = coefficients;
    d.eps = a.eps;
    d.scale = (float)a.scale;
    d.ws = a.workspace_dev;
    return hip_error(zk::launch_orthogonalize(d, static_cast<hipStream_t>(stream)), fn);
}

}  // extern "C"
