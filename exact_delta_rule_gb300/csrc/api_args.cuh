// Argument checks that the C entry points share.
#pragma once

#include <string.h>

#include <initializer_list>

#include "internal.cuh"

namespace efla {

inline size_t es(efla_dtype t) { return t == EFLA_BF16 ? 2 : 4; }
inline bool dtype_ok(efla_dtype t) { return t == EFLA_BF16 || t == EFLA_F32; }

enum Role { IN, IN_OPT, OUT, OUT_OPT };
struct Arg {
    const char *name;
    const void *p;
    size_t bytes;
    Role role;
    const char *may_be[2] = {nullptr, nullptr};  // an output may be exactly the inputs of these names
};

// Whether output o may lie where x does: x is an input that o's contract names, at the same address.
inline bool may_share(const Arg &o, const Arg &x) {
    if (x.p != o.p || x.bytes != o.bytes || (x.role != IN && x.role != IN_OPT)) return false;
    for (const char *name : o.may_be)
        if (name && strcmp(name, x.name) == 0) return true;
    return false;
}

// Every non-optional argument with bytes > 0 present, every pointer 16-byte aligned, no output
// overlapping any other argument than an input it may be.
inline efla_status check_args(std::initializer_list<Arg> args) {
    for (const Arg &a : args) {
        if (!a.p && a.bytes > 0 && (a.role == IN || a.role == OUT))
            return api_fail(EFLA_ERR_INVALID_ARG, "%s must be non-NULL", a.name);
        if (reinterpret_cast<uintptr_t>(a.p) & 15u)
            return api_fail(EFLA_ERR_INVALID_ARG, "%s=%p is not 16-byte aligned", a.name, a.p);
    }
    for (const Arg &o : args) {
        if ((o.role != OUT && o.role != OUT_OPT) || !o.p || o.bytes == 0) continue;
        const uintptr_t o0 = reinterpret_cast<uintptr_t>(o.p), o1 = o0 + o.bytes;
        for (const Arg &x : args) {
            if (&x == &o || !x.p || x.bytes == 0 || may_share(o, x)) continue;
            const uintptr_t x0 = reinterpret_cast<uintptr_t>(x.p), x1 = x0 + x.bytes;
            if (o0 < x1 && x0 < o1) return api_fail(EFLA_ERR_INVALID_ARG, "output %s overlaps %s", o.name, x.name);
        }
    }
    return EFLA_OK;
}

inline efla_status launched(cudaError_t e, const char *what) {
    if (e != cudaSuccess) return api_fail(EFLA_ERR_CUDA, "%s: %s (%s)", what, cudaGetErrorName(e), cudaGetErrorString(e));
    return api_ok();
}

inline efla_status need_workspace(const void *ws, size_t have, size_t need) {
    if (need > 0 && (!ws || have < need))
        return api_fail(EFLA_ERR_INVALID_ARG, "workspace of %zu bytes needed (got %zu at %p)", need, ws ? have : (size_t)0, ws);
    return EFLA_OK;
}

}  // namespace efla
