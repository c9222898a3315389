// abi_checks.h -- argument checks shared by the C entry points of the layer operators
// and of the matrix step (layer_abi.cpp, muon_abi.cpp): matrices with their row
// lengths and overlaps, sizes, types and workspaces.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "zero_internal.h"

namespace zl {

constexpr int64_t kMaxDim = INT32_MAX;
constexpr int64_t kMaxLd = int64_t(1) << 40;

// One matrix argument. `written` outputs may not overlap any other matrix, unless
// both are elementwise and exactly the same.
struct Mat {
    const char* name;
    const void* p;
    int64_t rows, cols, ld;
    int64_t esize;
    bool written;
    bool elementwise;
    bool optional;
};

inline bool empty(const Mat& m) { return !m.p || m.rows == 0 || m.cols == 0; }

// Whether any element belongs to both: their address ranges meet, and, where both
// have the same row length, so do their columns within it.
inline bool meet(const Mat& a, const Mat& b) {
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

inline int check_mats(const char* fn, const Mat* m, int n) {
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

inline int check_dims(const char* fn, int64_t M, int64_t K, int64_t N) {
    if (M < 0 || K < 0 || N < 0 || M > kMaxDim || K > kMaxDim || N > kMaxDim) {
        set_error("%s: sizes M=%lld K=%lld N=%lld outside [0, 2^31 - 1]", fn, (long long)M, (long long)K,
                  (long long)N);
        return ZERO_E_RANGE;
    }
    return ZERO_OK;
}

inline int check_type(const char* fn, const char* name, int32_t ty) {
    if (ty == ZERO_F32 || ty == ZERO_BF16) return ZERO_OK;
    set_error("%s: %s=%d is neither ZERO_F32 nor ZERO_BF16", fn, name, (int)ty);
    return ZERO_E_INVAL;
}

inline int check_ws(const char* fn, const void* ws, size_t have, size_t need) {
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

inline int64_t size_of(int32_t ty) { return ty == ZERO_F32 ? 4 : 2; }

inline Mat ws_mat(void* ws, size_t need) {
    return Mat{"workspace_dev", need ? ws : nullptr, 1, (int64_t)need, (int64_t)need, 1, true, false, true};
}

}  // namespace zl
