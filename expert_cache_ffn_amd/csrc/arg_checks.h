// Argument checks that the dense and the token operators' entry points share.
#pragma once

#include <cstdint>
#include <initializer_list>

#include "ecf_internal.h"

namespace ecf {

inline size_t al256(size_t v) { return (v + 255) & ~(size_t)255; }
inline int64_t ld_or(int64_t ld, int64_t width) { return ld ? ld : width; }

inline bool dense_dtype(int32_t t) { return t == ECF_F32 || t == ECF_BF16 || t == ECF_F16; }
inline size_t dense_esize(int dtype) { return dtype == ECF_F32 ? 4 : 2; }

inline int check_vector(const char *what, const char *name, const void *p, int dtype)
{
    if ((uintptr_t)p % dense_esize(dtype))
        return set_error(ECF_EINVAL, "%s: %s is not aligned to its elements", what, name);
    return ECF_OK;
}

inline int check_ws(const char *what, const void *ws, size_t have, size_t need)
{
    if (!need)
        return ECF_OK;
    if (!ws || have < need)
        return set_error(ECF_ENOSPC, "%s: needs %zu bytes of workspace, got %zu", what, need, ws ? have : (size_t)0);
    if ((uintptr_t)ws % 256)
        return set_error(ECF_EINVAL, "%s: the workspace is not at a 256-byte boundary", what);
    return ECF_OK;
}

inline int check_grad_dtype(const char *what, int32_t t, int32_t dtype)
{
    if (t != dtype && t != ECF_F32)
        return set_error(ECF_EINVAL, "%s: wgrad_dtype must be dtype or ECF_F32 (got %d)", what, t);
    return ECF_OK;
}

// A matrix operand at its elements' alignment, whose rows may lie apart.
constexpr int64_t kMaxStride = (int64_t)1 << 31;
inline int check_rows(const char *what, const char *name, const void *p, int64_t ld, int64_t width, size_t esize)
{
    if (!p)
        return set_error(ECF_EINVAL, "%s: %s is NULL", what, name);
    if ((uintptr_t)p % esize)
        return set_error(ECF_EINVAL, "%s: %s is not aligned to its %zu-byte elements", what, name, esize);
    if (ld < width)
        return set_error(ECF_EINVAL, "%s: the row stride of %s (%lld) is below its width %lld", what, name,
                         (long long)ld, (long long)width);
    if (ld >= kMaxStride)
        return set_error(ECF_EUNSUPPORTED, "%s: the row stride of %s (%lld) is 2^31 or more", what, name, (long long)ld);
    return ECF_OK;
}
inline int check_rows(const char *what, const char *name, const void *p, int64_t ld, int64_t width, int dtype)
{
    return check_rows(what, name, p, ld, width, dense_esize(dtype));
}

inline int check_aligned(const char *what, const char *name, const void *p, size_t esize)
{
    if ((uintptr_t)p % esize)
        return set_error(ECF_EINVAL, "%s: %s is not aligned to its %zu-byte elements", what, name, esize);
    return ECF_OK;
}

inline int check_present(const char *what, const char *name, const void *p, size_t esize)
{
    if (!p)
        return set_error(ECF_EINVAL, "%s: %s is NULL", what, name);
    return check_aligned(what, name, p, esize);
}

inline int check_same_stride(const char *what, const char *a, const void *p, int64_t lda, const char *b, const void *q, int64_t ldb)
{
    if (p && p == q && lda != ldb)
        return set_error(ECF_EINVAL, "%s: %s is %s with another row stride (%lld and %lld)", what, a, b, (long long)lda,
                         (long long)ldb);
    return ECF_OK;
}

// An output that starts where another one or an input does: blocks would read what
// others have written.  (Other overlaps are the caller's to avoid.)
struct Named {
    const char *name;
    const void *p;
};
inline int check_apart(const char *what, std::initializer_list<Named> outs, std::initializer_list<Named> ins)
{
    for (const Named *o = outs.begin(); o != outs.end(); ++o) {
        if (!o->p)
            continue;
        for (const Named &i : ins)
            if (i.p == o->p)
                return set_error(ECF_EINVAL, "%s: %s and %s are the same memory", what, o->name, i.name);
        for (const Named *q = outs.begin(); q != o; ++q)
            if (q->p == o->p)
                return set_error(ECF_EINVAL, "%s: %s and %s are the same memory", what, o->name, q->name);
    }
    return ECF_OK;
}

#define ECF_TRY(expr)                  \
    do {                               \
        const int _rc = (expr);        \
        if (_rc != ECF_OK)             \
            return _rc;                \
    } while (0)

}  // namespace ecf
