// api_tokens.hpp -- argument checks that the token operators' C ABI layers
// (api_tokens.hip, api_cache.hip) share.
#pragma once

#include "../../include/mp3d.h"
#include "api_common.hpp"
#include "dtype.hpp"
#include "tokens.hpp"

namespace mp3d {

constexpr int64_t kMaxLen = (int64_t)1 << 30;      // tokens of a sequence
constexpr int64_t kMaxElems = (int64_t)1 << 40;    // elements of a tensor

inline int elem_bytes(int dtype) { return dtype == MP3D_F32 ? 4 : 2; }

inline int check_dtype(int dtype)
{
    if (dtype != MP3D_F32 && dtype != MP3D_F16 && dtype != MP3D_BF16)
        return fail(MP3D_EDTYPE, "dtype %d is not MP3D_F32, MP3D_F16 or MP3D_BF16", dtype);
    return MP3D_OK;
}

// a * b * c * d within kMaxElems (all >= 0)
inline bool too_many(int64_t a, int64_t b, int64_t c, int64_t d)
{
    const int64_t v[4] = {a, b, c, d};
    int64_t n = 1;
    for (int i = 0; i < 4; ++i) {
        if (v[i] == 0) return false;
        if (n > kMaxElems / v[i]) return true;
        n *= v[i];
    }
    return false;
}

inline bool aligned(const void *p, int64_t bytes) { return (uintptr_t)p % (uintptr_t)bytes == 0; }

inline int check_strides(const int64_t *s, const char *name)
{
    if (!s) return fail(MP3D_EINVAL, "%s strides are NULL", name);
    for (int i = 0; i < 3; ++i)
        if (s[i] < 0 || s[i] > kMaxElems)
            return fail(MP3D_EINVAL, "%s stride %lld is out of range", name, (long long)s[i]);
    return MP3D_OK;
}

template <typename F>
inline int by_dtype(int dtype, F f)
{
    if (dtype == MP3D_F32) return f(F32{});
    if (dtype == MP3D_F16) return f(F16{});
    return f(BF16{});
}

// 16-byte rows: every base and stride a multiple of 16 bytes
inline bool wide_rows(const void *p, const int64_t *s, int es)
{
    return aligned(p, 16) && s[0] * es % 16 == 0 && s[1] * es % 16 == 0 && s[2] * es % 16 == 0;
}

inline int check_launch(int64_t blocks)
{
    if (blocks > kInt32Max / 256)
        return fail(MP3D_EOVERFLOW, "the call needs more workgroups than one launch takes");
    return MP3D_OK;
}

inline int check_workspace(const void *ws, size_t have, size_t need)
{
    if (need == 0) return MP3D_OK;
    if (!ws || have < need || !aligned(ws, 16))
        return fail(MP3D_EWORKSPACE, "the call needs a 16-byte aligned workspace of %zu bytes, "
                    "got %zu", need, ws ? have : (size_t)0);
    return MP3D_OK;
}

}  // namespace mp3d
