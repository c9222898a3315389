// layer_abi.cpp -- the C entry points of the layer operators (linear products and
// their gradients, dropout, norms): argument validation and the descriptors of their
// kernels, which live in linear_kernels.hip, dropout_kernels.hip and norm_kernels.hip.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "abi_checks.h"
#include "layer_internal.h"
#include "zero_internal.h"
#include "zero_layer.h"

namespace {

using namespace zl;

static_assert(sizeof(zero_dropout) == 32 && sizeof(zero_linear_args) == 176 &&
                  sizeof(zero_linear_grad_input_args) == 152 && sizeof(zero_linear_grad_weight_args) == 112 &&
                  sizeof(zero_dropout_args) == 128 && sizeof(zero_norm_args) == 128 &&
                  sizeof(zero_norm_grad_args) == 152,
              "the argument blocks of the ABI");

int check_output(const char* fn, int64_t rows, int64_t cols) {
    if (zk::product_fits(rows, cols)) return ZERO_OK;
    set_error("%s: an output of %lld x %lld is more than 2^23 tiles of 128 x 128 or 2^29 a side", fn,
              (long long)rows, (long long)cols);
    return ZERO_E_RANGE;
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

// Norms of rows up to this length: what joins the columns' sums fits one launch.
constexpr int64_t kMaxNorm = int64_t(1) << 24;

int check_norm(const char* fn, int64_t M, int64_t N, int32_t kind) {
    int rc;
    if ((rc = check_dims(fn, M, 0, N))) return rc;
    if (N > kMaxNorm) {
        set_error("%s: rows of N=%lld, above 2^24", fn, (long long)N);
        return ZERO_E_RANGE;
    }
    if (kind == ZERO_NORM_LAYER || kind == ZERO_NORM_RMS) return ZERO_OK;
    set_error("%s: unknown kind %d", fn, (int)kind);
    return ZERO_E_INVAL;
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

int zero_norm_forward(const zero_norm_args* args, void* stream) {
    static const char* fn = "zero_norm_forward";
    if (!args) {
        set_error("%s: args is NULL", fn);
        return ZERO_E_INVAL;
    }
    const zero_norm_args& a = *args;
    int rc;
    if ((rc = check_norm(fn, a.M, a.N, a.kind)) || (rc = check_type(fn, "x_dtype", a.x_dtype)) ||
        (rc = check_type(fn, "sum_dtype", a.sum_dtype)) || (rc = check_type(fn, "y_dtype", a.y_dtype)))
        return rc;
    if (!(a.eps >= 0.0 && a.eps <= 1e30)) {
        set_error("%s: eps=%g outside [0, 1e30]", fn, a.eps);
        return ZERO_E_INVAL;
    }
    if (a.M == 0 || a.N == 0) return ZERO_OK;
    if (!a.residual != !a.sum) {
        set_error("%s: %s", fn, a.sum ? "a sum without a residual" : "a residual without a sum to store");
        return ZERO_E_INVAL;
    }
    const int64_t xb = size_of(a.x_dtype), sb = size_of(a.sum_dtype), yb = size_of(a.y_dtype);
    const Mat m[] = {{"x", a.x, a.M, a.N, a.ld_x, xb, false, true, false},
                     {"residual", a.residual, a.M, a.N, a.ld_residual, sb, false, true, true},
                     {"weight", a.weight, 1, a.N, a.N, 2, false, false, true},
                     {"bias", a.bias, 1, a.N, a.N, 2, false, false, true},
                     {"y", a.y, a.M, a.N, a.ld_y, yb, true, true, false},
                     {"sum", a.sum, a.M, a.N, a.ld_sum, sb, true, true, true},
                     {"stats", a.stats, a.M, 2, 2, 4, true, false, true}};
    if ((rc = check_mats(fn, m, 7))) return rc;
    zk::NormDesc d{};
    d.M = a.M;
    d.N = a.N;
    d.x = a.x;
    d.res = a.residual;
    d.sum = a.sum;
    d.y = a.y;
    d.ld_x = a.ld_x;
    d.ld_res = a.ld_residual;
    d.ld_sum = a.ld_sum;
    d.ld_y = a.ld_y;
    d.x_f32 = a.x_dtype == ZERO_F32;
    d.sum_f32 = a.sum_dtype == ZERO_F32;
    d.y_f32 = a.y_dtype == ZERO_F32;
    d.rms = a.kind == ZERO_NORM_RMS;
    d.eps = (float)a.eps;
    d.w = a.weight;
    d.b = a.bias;
    d.stats = a.stats;
    return zl::hip_error(zk::launch_norm(d, static_cast<hipStream_t>(stream)), fn);
}

size_t zero_norm_workspace_bytes(int64_t M, int64_t N) {
    return M < 0 || N < 1 || M > kMaxDim || N > kMaxNorm ? 0 : zk::norm_ws_bytes(M, N);
}

int zero_norm_grad(const zero_norm_grad_args* args, void* stream) {
    static const char* fn = "zero_norm_grad";
    if (!args) {
        set_error("%s: args is NULL", fn);
        return ZERO_E_INVAL;
    }
    const zero_norm_grad_args& a = *args;
    int rc;
    if ((rc = check_norm(fn, a.M, a.N, a.kind)) || (rc = check_type(fn, "dy_dtype", a.dy_dtype)) ||
        (rc = check_type(fn, "x_dtype", a.x_dtype)) || (rc = check_type(fn, "dx_dtype", a.dx_dtype)) ||
        (rc = check_type(fn, "grad_dtype", a.grad_dtype)))
        return rc;
    const bool sums = a.dweight || a.dbias;
    if (a.N == 0 || (a.M == 0 && !sums)) return ZERO_OK;
    const int64_t db = size_of(a.dy_dtype), xb = size_of(a.x_dtype), ob = size_of(a.dx_dtype), gb = size_of(a.grad_dtype);
    const size_t need = sums ? zk::norm_ws_bytes(a.M, a.N) : 0;
    const Mat m[] = {{"dy", a.dy, a.M, a.N, a.ld_dy, db, false, true, false},
                     {"x", a.x, a.M, a.N, a.ld_x, xb, false, true, false},
                     {"weight", a.weight, 1, a.N, a.N, 2, false, false, true},
                     {"stats", a.stats, a.M, 2, 2, 4, false, false, false},
                     {"residual_grad", a.residual_grad, a.M, a.N, a.ld_residual_grad, ob, false, true, true},
                     {"dx", a.dx, a.M, a.N, a.ld_dx, ob, true, true, false},
                     {"dweight", a.dweight, 1, a.N, a.N, gb, true, false, true},
                     {"dbias", a.dbias, 1, a.N, a.N, gb, true, false, true},
                     ws_mat(a.workspace_dev, need)};
    if ((rc = check_ws(fn, a.workspace_dev, a.ws_bytes, need)) || (rc = check_mats(fn, m, 9))) return rc;
    zk::NormGradDesc d{};
    d.M = a.M;
    d.N = a.N;
    d.dy = a.dy;
    d.x = a.x;
    d.res = a.residual_grad;
    d.dx = a.dx;
    d.ld_dy = a.ld_dy;
    d.ld_x = a.ld_x;
    d.ld_res = a.ld_residual_grad;
    d.ld_dx = a.ld_dx;
    d.dy_f32 = a.dy_dtype == ZERO_F32;
    d.x_f32 = a.x_dtype == ZERO_F32;
    d.dx_f32 = a.dx_dtype == ZERO_F32;
    d.rms = a.kind == ZERO_NORM_RMS;
    d.w = a.weight;
    d.stats = a.stats;
    d.dw = a.dweight;
    d.db = a.dbias;
    d.grad_f32 = a.grad_dtype == ZERO_F32;
    d.accumulate = a.accumulate != 0;
    d.ws = static_cast<float*>(a.workspace_dev);
    return zl::hip_error(zk::launch_norm_grad(d, static_cast<hipStream_t>(stream)), fn);
}

}  // extern "C"
