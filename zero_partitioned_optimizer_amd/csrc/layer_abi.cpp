// layer_abi.cpp -- the C entry points of the layer operators (linear products and
// their gradients, dropout): argument validation and the descriptors of their
// kernels, which live in linear_kernels.hip and dropout_kernels.hip.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "layer_internal.h"
#include "zero_internal.h"
#include "zero_layer.h"

namespace {

using zl::set_error;

static_assert(sizeof(zero_dropout) == 32 && sizeof(zero_linear_args) == 176 &&
                  sizeof(zero_linear_grad_input_args) == 152 && sizeof(zero_linear_grad_weight_args) == 112 &&
                  sizeof(zero_dropout_args) == 128,
              "the argument blocks of the ABI");

constexpr int64_t kMaxDim = INT32_MAX;
constexpr int64_t kMaxLd = int64_t(1) << 40;

// One matrix argument. `written` outputs may not overlap any other matrix, unless
// both are elementwise (`elem` > 0) and exactly the same.
struct Mat {
    const char* name;
    const void* p;
    int64_t rows, cols, ld;
    int64_t esize;
    bool written;
    bool elementwise;
    bool optional;
};

bool empty(const Mat& m) { return !m.p || m.rows == 0 || m.cols == 0; }

// Whether any element belongs to both: their address ranges meet, and, where both
// have the same row length, so do their columns within it.
bool meet(const Mat& a, const Mat& b) {
    if (empty(a) || empty(b)) return false;
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
    const uintptr_t la = (uintptr_t)(a.ld * a.esize), lb = (uintptr_t)(b.ld * b.esize);
    const uintptr_t wa = (uintptr_t)(a.cols * a.esize), wb = (uintptr_t)(b.cols * b.esize);
    const uintptr_t a1 = a0 + la * (uintptr_t)(a.rows - 1) + wa, b1 = b0 + lb * (uintptr_t)(b.rows - 1) + wb;
    if (a1 <= b0 || b1 <= a0) return false;
    if (la != lb || a.rows == 1 || b.rows == 1) return true;
    const uintptr_t shift = b0 >= a0 ? (b0 - a0) % la : (la - (a0 - b0) % la) % la;
    return shift < wa || shift + wb > la;
}

int check_mats(const char* fn, const Mat* m, int n) {
    for (int i = 0; i < n; ++i) {
        if (m[i].optional && !m[i].p) continue;
        if (m[i].rows == 0 || m[i].cols == 0) continue;
        if (!m[i].p) {
            set_error("%s: %s is NULL", fn, m[i].name);
            return ZERO_E_INVAL;
        }
        if (reinterpret_cast<uintptr_t>(m[i].p) % (uintptr_t)m[i].esize != 0) {
            set_error("%s: %s=%p is not aligned to its %d-byte elements", fn, m[i].name, m[i].p,
                      (int)m[i].esize);
            return ZERO_E_ALIGN;
        }
        if (m[i].ld < m[i].cols || m[i].ld > kMaxLd) {
            set_error("%s: ld of %s is %lld, outside [%lld, 2^40]", fn, m[i].name, (long long)m[i].ld,
                      (long long)m[i].cols);
            return ZERO_E_RANGE;
        }
    }
    for (int i = 0; i < n; ++i)
        for (int k = i + 1; k < n; ++k) {
            if (!m[i].written && !m[k].written) continue;
            if (!meet(m[i], m[k])) continue;
            const bool same = m[i].elementwise && m[k].elementwise && !(m[i].written && m[k].written) &&
                              m[i].p == m[k].p && m[i].ld == m[k].ld && m[i].esize == m[k].esize;
            if (same) continue;
            set_error("%s: %s and %s overlap", fn, m[i].name, m[k].name);
            return ZERO_E_INVAL;
        }
    return ZERO_OK;
}

int check_dims(const char* fn, int64_t M, int64_t K, int64_t N) {
    if (M < 0 || K < 0 || N < 0 || M > kMaxDim || K > kMaxDim || N > kMaxDim) {
        set_error("%s: sizes M=%lld K=%lld N=%lld outside [0, 2^31 - 1]", fn, (long long)M, (long long)K,
                  (long long)N);
        return ZERO_E_RANGE;
    }
    return ZERO_OK;
}

int check_output(const char* fn, int64_t rows, int64_t cols) {
    if (zk::product_fits(rows, cols)) return ZERO_OK;
    set_error("%s: an output of %lld x %lld is more than 2^23 tiles of 128 x 128 or 2^29 a side", fn,
              (long long)rows, (long long)cols);
    return ZERO_E_RANGE;
}

int check_type(const char* fn, const char* name, int32_t ty) {
    if (ty == ZERO_F32 || ty == ZERO_BF16) return ZERO_OK;
    set_error("%s: %s=%d is neither ZERO_F32 nor ZERO_BF16", fn, name, (int)ty);
    return ZERO_E_INVAL;
}

int check_act(const char* fn, int32_t act) {
    if (act >= ZERO_ACT_NONE && act <= ZERO_ACT_SILU) return ZERO_OK;
    set_error("%s: unknown act %d", fn, (int)act);
    return ZERO_E_INVAL;
}

int check_w_layout(const char* fn, int32_t lay) {
    if (lay == ZERO_W_OUT_IN || lay == ZERO_W_IN_OUT) return ZERO_OK;
    set_error("%s: unknown w_layout %d", fn, (int)lay);
    return ZERO_E_INVAL;
}

int make_drop(const char* fn, const zero_dropout& in, zk::Drop* out) {
    *out = zk::Drop{};
    if (!(in.p >= 0.0 && in.p <= 1.0 - 1.0 / 65536.0)) {
        set_error("%s: dropout p=%g outside [0, 1 - 2^-16]", fn, in.p);
        return ZERO_E_INVAL;
    }
    if (reinterpret_cast<uintptr_t>(in.counter_dev) % 8 != 0) {
        set_error("%s: dropout counter_dev=%p is not 8-byte aligned", fn, (const void*)in.counter_dev);
        return ZERO_E_ALIGN;
    }
    out->thr = (uint32_t)nearbyint(in.p * 65536.0);
    out->scale = (float)(65536.0 / (65536.0 - (double)out->thr));
    out->k0 = (uint32_t)in.seed;
    out->k1 = (uint32_t)(in.seed >> 32);
    out->offset = in.offset;
    out->counter = in.counter_dev;
    return ZERO_OK;
}

int check_ws(const char* fn, const void* ws, size_t have, size_t need) {
    if (need == 0) return ZERO_OK;
    if (!ws) {
        set_error("%s: workspace_dev is NULL, %zu bytes are needed", fn, need);
        return ZERO_E_INVAL;
    }
    if (reinterpret_cast<uintptr_t>(ws) % 16 != 0) {
        set_error("%s: workspace_dev=%p is not 16-byte aligned", fn, ws);
        return ZERO_E_ALIGN;
    }
    if (have < need) {
        set_error("%s: ws_bytes=%zu, %zu are needed", fn, have, need);
        return ZERO_E_RANGE;
    }
    return ZERO_OK;
}

int64_t size_of(int32_t ty) { return ty == ZERO_F32 ? 4 : 2; }

Mat ws_mat(void* ws, size_t need) {
    return Mat{"workspace_dev", need ? ws : nullptr, 1, (int64_t)need, (int64_t)need, 1, true, false, true};
}

// Bytes of the weight gradient's product and, behind it, of the bias gradient.
size_t weight_ws(bool oi, int64_t M, int64_t K, int64_t N, size_t* product) {
    const int64_t P = oi ? N : K, Q = oi ? K : N;
    *product = (zk::product_ws_bytes(P, Q, M, true, true) + 15) & ~(size_t)15;
    return *product + zk::sums_ws_bytes(P, Q, M, oi);
}

}  // namespace

extern "C" {

size_t zero_linear_workspace_bytes(int32_t kind, int32_t w_layout, int64_t M, int64_t K, int64_t N) {
    if (M < 0 || K < 0 || N < 0 || M > kMaxDim || K > kMaxDim || N > kMaxDim) return 0;
    if (w_layout != ZERO_W_OUT_IN && w_layout != ZERO_W_IN_OUT) return 0;
    const bool oi = w_layout == ZERO_W_OUT_IN;
    size_t product;
    const int64_t rows = kind == ZERO_LINEAR_GRAD_WEIGHT ? N : M, cols = kind == ZERO_LINEAR_FORWARD ? N : K;
    if (!zk::product_fits(rows, cols)) return 0;
    if (kind == ZERO_LINEAR_FORWARD) return zk::product_ws_bytes(M, N, K, false, !oi);
    if (kind == ZERO_LINEAR_GRAD_INPUT) return zk::product_ws_bytes(M, K, N, false, oi);
    if (kind == ZERO_LINEAR_GRAD_WEIGHT) return weight_ws(oi, M, K, N, &product);
    return 0;
}

int zero_linear_forward(const zero_linear_args* args, void* stream) {
    static const char* fn = "zero_linear_forward";
    if (!args) {
        set_error("%s: args is NULL", fn);
        return ZERO_E_INVAL;
    }
    const zero_linear_args& a = *args;
    int rc;
    zk::Drop drop;
    if ((rc = check_dims(fn, a.M, a.K, a.N)) || (rc = check_output(fn, a.M, a.N)) ||
        (rc = check_type(fn, "y_dtype", a.y_dtype)) ||
        (rc = check_act(fn, a.act)) || (rc = check_w_layout(fn, a.w_layout)) ||
        (rc = make_drop(fn, a.dropout, &drop)))
        return rc;
    const bool oi = a.w_layout == ZERO_W_OUT_IN;
    const int64_t ob = size_of(a.y_dtype);
    if (a.M == 0 || a.N == 0) return ZERO_OK;
    const size_t need = zk::product_ws_needed(a.x, a.ld_x, a.w, a.ld_w, a.M, a.N, a.K, !oi);
    const Mat m[] = {{"x", a.x, a.M, a.K, a.ld_x, 2, false, false, false},
                     {"w", a.w, oi ? a.N : a.K, oi ? a.K : a.N, a.ld_w, 2, false, false, false},
                     {"bias", a.bias, 1, a.N, a.N, 2, false, false, true},
                     {"residual", a.residual, a.M, a.N, a.ld_residual, ob, false, true, true},
                     {"y", a.y, a.M, a.N, a.ld_y, ob, true, true, false},
                     {"preact", a.preact, a.M, a.N, a.ld_preact, 2, true, false, true},
                     ws_mat(a.workspace_dev, need)};
    if ((rc = check_mats(fn, m, 7))) return rc;
    if ((rc = check_ws(fn, a.workspace_dev, a.ws_bytes, need))) return rc;
    zk::ProductDesc d{};
    d.a = a.x;
    d.lda = a.ld_x;
    d.b = a.w;
    d.ldb = a.ld_w;
    d.tb = !oi;
    d.P = a.M;
    d.Q = a.N;
    d.R = a.K;
    d.epi = zk::kEpiForward;
    d.out = a.y;
    d.ld_out = a.ld_y;
    d.out_f32 = a.y_dtype == ZERO_F32;
    d.bias = a.bias;
    d.res = a.residual;
    d.ld_res = a.ld_residual;
    d.z_out = a.preact;
    d.ld_z = a.ld_preact;
    d.act = a.act;
    d.drop = drop;
    d.ws = static_cast<float*>(a.workspace_dev);
    return zl::hip_error(zk::launch_product(d, static_cast<hipStream_t>(stream)), fn);
}

int zero_linear_grad_input(const zero_linear_grad_input_args* args, void* stream) {
    static const char* fn = "zero_linear_grad_input";
    if (!args) {
        set_error("%s: args is NULL", fn);
        return ZERO_E_INVAL;
    }
    const zero_linear_grad_input_args& a = *args;
    int rc;
    zk::Drop drop;
    if ((rc = check_dims(fn, a.M, a.K, a.N)) || (rc = check_output(fn, a.M, a.K)) ||
        (rc = check_type(fn, "dx_dtype", a.dx_dtype)) ||
        (rc = check_act(fn, a.act)) || (rc = check_w_layout(fn, a.w_layout)) ||
        (rc = make_drop(fn, a.dropout, &drop)))
        return rc;
    const bool oi = a.w_layout == ZERO_W_OUT_IN;
    const bool act = a.act != ZERO_ACT_NONE;
    if (a.M == 0 || a.K == 0) return ZERO_OK;
    const size_t need = zk::product_ws_needed(a.dz, a.ld_dz, a.w, a.ld_w, a.M, a.K, a.N, oi);
    const Mat m[] = {{"dz", a.dz, a.M, a.N, a.ld_dz, 2, false, false, false},
                     {"w", a.w, oi ? a.N : a.K, oi ? a.K : a.N, a.ld_w, 2, false, false, false},
                     {"preact", act ? a.preact : nullptr, a.M, a.K, a.ld_preact, 2, false, true, !act},
                     {"dx", a.dx, a.M, a.K, a.ld_dx, size_of(a.dx_dtype), true, true, false},
                     ws_mat(a.workspace_dev, need)};
    if ((rc = check_mats(fn, m, 5))) return rc;
    if ((rc = check_ws(fn, a.workspace_dev, a.ws_bytes, need))) return rc;
    zk::ProductDesc d{};
    d.a = a.dz;
    d.lda = a.ld_dz;
    d.b = a.w;
    d.ldb = a.ld_w;
    d.tb = oi;
    d.P = a.M;
    d.Q = a.K;
    d.R = a.N;
    d.epi = zk::kEpiGradInput;
    d.out = a.dx;
    d.ld_out = a.ld_dx;
    d.out_f32 = a.dx_dtype == ZERO_F32;
    d.z_in = act ? a.preact : nullptr;
    d.ld_z = a.ld_preact;
    d.act = a.act;
    d.drop = drop;
    d.ws = static_cast<float*>(a.workspace_dev);
    return zl::hip_error(zk::launch_product(d, static_cast<hipStream_t>(stream)), fn);
}

int zero_linear_grad_weight(const zero_linear_grad_weight_args* args, void* stream) {
    static const char* fn = "zero_linear_grad_weight";
    if (!args) {
        set_error("%s: args is NULL", fn);
        return ZERO_E_INVAL;
    }
    const zero_linear_grad_weight_args& a = *args;
    int rc;
    if ((rc = check_dims(fn, a.M, a.K, a.N)) || (rc = check_output(fn, a.N, a.K)) ||
        (rc = check_type(fn, "grad_dtype", a.grad_dtype)) ||
        (rc = check_w_layout(fn, a.w_layout)))
        return rc;
    const bool oi = a.w_layout == ZERO_W_OUT_IN;
    const int64_t gb = size_of(a.grad_dtype);
    size_t product;
    size_t need = weight_ws(oi, a.M, a.K, a.N, &product);
    if (!a.dbias) need = product;
    if (a.N == 0) return ZERO_OK;
    const Mat m[] = {{"dz", a.dz, a.M, a.N, a.ld_dz, 2, false, false, false},
                     {"x", a.x, a.M, a.K, a.ld_x, 2, false, false, false},
                     {"dw", a.dw, oi ? a.N : a.K, oi ? a.K : a.N, a.ld_dw, gb, true, false, false},
                     {"dbias", a.dbias, 1, a.N, a.N, gb, true, false, true},
                     ws_mat(a.workspace_dev, need)};
    if ((rc = check_mats(fn, m, 5))) return rc;
    if ((rc = check_ws(fn, a.workspace_dev, a.ws_bytes, need))) return rc;
    zk::ProductDesc d{};
    d.a = oi ? a.dz : a.x;
    d.lda = oi ? a.ld_dz : a.ld_x;
    d.b = oi ? a.x : a.dz;
    d.ldb = oi ? a.ld_x : a.ld_dz;
    d.ta = d.tb = true;
    d.P = oi ? a.N : a.K;
    d.Q = oi ? a.K : a.N;
    d.R = a.M;
    d.epi = zk::kEpiGradWeight;
    d.out = a.dw;
    d.ld_out = a.ld_dw;
    d.out_f32 = a.grad_dtype == ZERO_F32;
    d.res = a.accumulate ? a.dw : nullptr;
    d.ld_res = a.ld_dw;
    d.ws = static_cast<float*>(a.workspace_dev);
    d.bias_out = a.dbias;
    d.bias_of_a = oi;
    d.bias_add = a.accumulate != 0;
    d.ws_sums = reinterpret_cast<float*>(static_cast<char*>(a.workspace_dev) + product);
    return zl::hip_error(zk::launch_product(d, static_cast<hipStream_t>(stream)), fn);
}

static int dropout(const char* fn, const zero_dropout_args* args, bool grad, void* stream) {
    if (!args) {
        set_error("%s: args is NULL", fn);
        return ZERO_E_INVAL;
    }
    const zero_dropout_args& a = *args;
    int rc;
    zk::Drop drop;
    if ((rc = check_dims(fn, a.M, 0, a.N)) || (rc = check_type(fn, "x_dtype", a.x_dtype)) ||
        (rc = check_type(fn, "y_dtype", a.y_dtype)) || (rc = check_act(fn, a.act)) ||
        (rc = make_drop(fn, a.dropout, &drop)))
        return rc;
    const bool act = a.act != ZERO_ACT_NONE;
    if (grad ? a.residual != nullptr : act || a.preact != nullptr) {
        set_error("%s: %s", fn, grad ? "a gradient takes no residual" : "dropout alone takes no act or preact");
        return ZERO_E_INVAL;
    }
    const int64_t xb = size_of(a.x_dtype), yb = size_of(a.y_dtype);
    if (a.M == 0 || a.N == 0) return ZERO_OK;
    const Mat m[] = {{grad ? "dy" : "x", a.x, a.M, a.N, a.ld_x, xb, false, true, false},
                     {"residual", a.residual, a.M, a.N, a.ld_residual, yb, false, true, true},
                     {"preact", act ? a.preact : nullptr, a.M, a.N, a.ld_preact, 2, false, true, !act},
                     {grad ? "dz" : "y", a.y, a.M, a.N, a.ld_y, yb, true, true, false}};
    if ((rc = check_mats(fn, m, 4))) return rc;
    zk::DropoutDesc d{};
    d.M = a.M;
    d.N = a.N;
    d.x = a.x;
    d.ld_x = a.ld_x;
    d.x_f32 = a.x_dtype == ZERO_F32;
    d.res = a.residual;
    d.ld_res = a.ld_residual;
    d.z = act ? a.preact : nullptr;
    d.ld_z = a.ld_preact;
    d.act = a.act;
    d.y = a.y;
    d.ld_y = a.ld_y;
    d.y_f32 = a.y_dtype == ZERO_F32;
    d.drop = drop;
    return zl::hip_error(zk::launch_dropout(d, grad, static_cast<hipStream_t>(stream)), fn);
}

int zero_dropout_add(const zero_dropout_args* args, void* stream) {
    return dropout("zero_dropout_add", args, false, stream);
}

int zero_dropout_grad(const zero_dropout_args* args, void* stream) {
    return dropout("zero_dropout_grad", args, true, stream);
}

}  // extern "C"
