// api_cache.hip -- the C ABI of caches and of attention over them
// (include/mp3d.h): argument checks and plans.  Every check runs before the
// first launch.
#include <stdio.h>

#include <algorithm>

#include "api_tokens.hpp"
#include "cache.hpp"

namespace mp3d {

static_assert(kPlain == MP3D_CACHE_PLAIN && kE4M3 == MP3D_CACHE_E4M3 && kE2M1 == MP3D_CACHE_E2M1,
              "the formats of the C ABI");

namespace {

int row_bytes(int format, int D) { return format == kE4M3 ? code_bytes<kE4M3>(D) : code_bytes<kE2M1>(D); }

// Bases, strides (in units of es bytes) and a row's bytes are multiples of n.
bool divides(int n, const mp3d_cache &c, int es, int bytes)
{
    if (!aligned(c.k, n) || !aligned(c.v, n) || bytes % n) return false;
    for (int i = 0; i < 3; ++i)
        if (c.k_stride[i] * es % n || c.v_stride[i] * es % n) return false;
    return true;
}

int check_cache(const mp3d_cache &c, int format, int32_t H, int32_t D, const char *name)
{
    if (c.B < 0 || c.T < 0) return fail(MP3D_EINVAL, "%s cache: B and T must be >= 0", name);
    if (c.B > kMaxLen || c.T > kMaxLen || too_many(c.B, c.T, H, D))
        return fail(MP3D_EOVERFLOW, "%s cache: B*T*H*D is out of range", name);
    if (c.B == 0 || c.T == 0) return MP3D_OK;
    int rc;
    if ((rc = check_strides(c.k_stride, "key")) || (rc = check_strides(c.v_stride, "value")))
        return rc;
    if (format != kPlain && ((rc = check_strides(c.k_scale_stride, "key scale")) ||
                             (rc = check_strides(c.v_scale_stride, "value scale"))))
        return rc;
    return MP3D_OK;
}

// (apart from the sizes alone: a workspace's size needs no pointers)
int check_pointers(const mp3d_cache &c, int format, const char *name)
{
    if (c.B == 0 || c.T == 0) return MP3D_OK;
    if (!c.k || !c.v || (format != kPlain && (!c.k_scale || !c.v_scale)))
        return fail(MP3D_EINVAL, "%s cache: a part is NULL", name);
    return MP3D_OK;
}

int cache_call(const mp3d_cache *c, int format, void *k, void *v, int dtype, int64_t T, int32_t H,
               int32_t D, const int64_t *k_stride, const int64_t *v_stride, const int32_t *start,
               const int32_t *count, bool read, void *stream)
{
    TimingScope timing_scope;
    if (!c) return fail(MP3D_EINVAL, "the cache is NULL");
    int rc = check_dtype(dtype);
    if (rc) return rc;
    if (format != kE4M3 && format != kE2M1)
        return fail(MP3D_EINVAL, "format %d is not MP3D_CACHE_E4M3 or MP3D_CACHE_E2M1", format);
    if (H < 1 || H > 65536 || D < 1 || D > kCacheMaxD)
        return fail(MP3D_EINVAL, "H=%d must be in 1 .. 65536 and D=%d in 1 .. %d", H, D, kCacheMaxD);
    if (T < 0) return fail(MP3D_EINVAL, "T must be >= 0");
    if ((rc = check_cache(*c, format, H, D, "the"))) return rc;
    if (T > kMaxLen || too_many(c->B, T, H, D))
        return fail(MP3D_EOVERFLOW, "B*T*H*D is out of range");
    if (c->B == 0 || T == 0 || (!read && c->T == 0)) return MP3D_OK;
    if (!k || !v) return fail(MP3D_EINVAL, "k or v is NULL");
    if ((rc = check_pointers(*c, format, "the"))) return rc;
    const int es = elem_bytes(dtype);
    if (read ? !aligned(k, 16) || !aligned(v, 16) : !aligned(k, es) || !aligned(v, es))
        return fail(MP3D_EINVAL, "k or v is not aligned (%d bytes)", read ? 16 : es);
    if (!read) {
        if ((rc = check_strides(k_stride, "k")) || (rc = check_strides(v_stride, "v"))) return rc;
        // rows that are one another's would be written by several at once
        const int64_t n[3] = {c->B, c->T, H};
        for (int i = 0; i < 3; ++i)
            if (n[i] > 1 && (c->k_stride[i] == 0 || c->v_stride[i] == 0 ||
                             c->k_scale_stride[i] == 0 || c->v_scale_stride[i] == 0))
                return fail(MP3D_EINVAL, "the rows of a cache that is written must be apart");
    }
    CachePlan p = {};
    p.x[0] = k;
    p.x[1] = v;
    p.codes[0] = (uint8_t *)c->k;
    p.codes[1] = (uint8_t *)c->v;
    p.scales[0] = (uint8_t *)c->k_scale;
    p.scales[1] = (uint8_t *)c->v_scale;
    for (int i = 0; i < 3; ++i) {
        p.xs[0][i] = read ? 0 : k_stride[i];
        p.xs[1][i] = read ? 0 : v_stride[i];
        p.cs[0][i] = c->k_stride[i];
        p.cs[1][i] = c->v_stride[i];
        p.ss[0][i] = c->k_scale_stride[i];
        p.ss[1][i] = c->v_scale_stride[i];
    }
    p.start = start;
    p.count = count;
    p.rows = c->T;
    p.B = (int32_t)c->B;
    p.T = (int32_t)T;
    p.H = H;
    p.D = D;
    p.format = format;
    // 8 channels a thread (4 of float32 to read): whole, and at a multiple of their bytes
    const int per = read && es == 4 ? 4 : 8;
    const bool elements = read || (wide_rows(k, k_stride, es) && wide_rows(v, v_stride, es));
    p.vec = D % per == 0 && elements &&
            (c->T == 0 || divides(per * (format == kE4M3 ? 2 : 1) / 2, *c, 1, row_bytes(format, D)));
    plan_cache(&p, es, read);
    if ((rc = check_launch((int64_t)p.tiles * p.B * 2))) return rc;
    if (log_enabled())
        fprintf(stderr, "[mp3d] cache %s dtype=%d format=%d vec=%d\n", read ? "read" : "write",
                dtype, format, p.vec);
    return by_dtype(dtype, [&](auto t) {
        return hip_status(launch_cache<decltype(t)>(p, read, (hipStream_t)stream),
                          read ? "cache read launch" : "cache write launch");
    });
}

int cached_args(const mp3d_attention_cache *d, CachedArgs *c)
{
    if (!d) return fail(MP3D_EINVAL, "the attention descriptor is NULL");
    int rc = check_dtype(d->dtype);
    if (rc) return rc;
    if (d->format != kPlain && d->format != kE4M3 && d->format != kE2M1)
        return fail(MP3D_EINVAL, "format %d is not one of enum mp3d_cache_format", d->format);
    if (d->B < 0 || d->Tq < 0) return fail(MP3D_EINVAL, "B and Tq must be >= 0");
    if (d->Hq < 1 || d->Hk < 1 || d->Hq % d->Hk)
        return fail(MP3D_EINVAL, "Hq=%d must be a positive multiple of Hk=%d", d->Hq, d->Hk);
    if (d->D < 1 || d->D > kAttnMaxD)
        return fail(MP3D_EINVAL, "D=%d must be in 1 .. %d", d->D, kAttnMaxD);
    if ((rc = check_cache(d->own, d->format, d->Hk, d->D, "own")) ||
        (rc = check_cache(d->prefix, d->format, d->Hk, d->D, "prefix")))
        return rc;
    if (d->own.B != d->B)
        return fail(MP3D_EINVAL, "the own cache is of %lld sequences, q of %lld",
                    (long long)d->own.B, (long long)d->B);
    const int64_t N = d->prefix.B;
    if (N > 0 && d->B % N)
        return fail(MP3D_EINVAL, "%lld sequences do not divide among %lld prefixes",
                    (long long)d->B, (long long)N);
    const int64_t S = N > 0 ? d->B / N : 1;
    if (d->Tq > kMaxLen || d->B > kMaxLen || too_many(d->B, d->Tq, d->Hq, d->D) ||
        d->Tq * d->Hq > kInt32Max / 2 || S * d->Tq * (d->Hq / d->Hk) > kInt32Max / 2)
        return fail(MP3D_EOVERFLOW, "B*Tq*Hq*D is out of range");
    if (d->causal != 0 && d->causal != 1) return fail(MP3D_EINVAL, "causal must be 0 or 1");
    if (!(d->softcap == 0.f || (d->softcap >= 1e-30f && d->softcap <= 1e30f)))
        return fail(MP3D_EINVAL, "softcap must be 0 (none) or in 1e-30 .. 1e30");
    if (!(d->scale == d->scale) || d->scale > 1e30f || d->scale < -1e30f)
        return fail(MP3D_EINVAL, "scale must be finite");
    if (d->axes < 0 || d->axes > 3) return fail(MP3D_EINVAL, "axes must be in 0 .. 3");
    // (a tensor without elements may be NULL)
    if (d->axes > 0 && (!d->slopes || (d->B * d->Tq > 0 && !d->pos_q) ||
                        (d->B * d->own.T > 0 && !d->pos_k) || (N * d->prefix.T > 0 && !d->pos_prefix)))
        return fail(MP3D_EINVAL, "a distance bias needs slopes and all positions");
    if ((rc = check_strides(d->q_stride, "q"))) return rc;
    *c = CachedArgs{};
    AttnArgs &a = c->a;
    for (int i = 0; i < 3; ++i) a.qs[i] = d->q_stride[i];
    a.B = (int32_t)d->B;
    a.Tq = (int32_t)d->Tq;
    a.Hq = d->Hq;
    a.Hk = d->Hk;
    a.G = d->Hq / d->Hk;
    a.D = d->D;
    a.scale = d->scale;
    a.cap = d->softcap;
    a.slopes = d->slopes;
    a.pos_q = d->pos_q;
    a.axes = d->axes;
    a.causal = d->causal;
    c->format = d->format;
    c->f32 = d->dtype == MP3D_F32;
    const int es = elem_bytes(d->dtype);
    const int unit = d->format == kE4M3 ? 16 : 8;          // bytes of 16 channels
    const mp3d_cache *src[2] = {&d->prefix, &d->own};
    for (int i = 0; i < 2; ++i) {
        CachedPart &p = c->part[i];
        const mp3d_cache &x = *src[i];
        p.k = x.k;
        p.v = x.v;
        p.k_scale = (const uint8_t *)x.k_scale;
        p.v_scale = (const uint8_t *)x.v_scale;
        for (int j = 0; j < 3; ++j) {
            p.ks[j] = x.k_stride[j];
            p.vs[j] = x.v_stride[j];
            p.kss[j] = x.k_scale_stride[j];
            p.vss[j] = x.v_scale_stride[j];
        }
        p.len = i ? d->kv_len : d->prefix_len;
        p.pos = i ? d->pos_k : d->pos_prefix;
        p.caches = (int32_t)x.B;
        p.T = p.caches ? (int32_t)x.T : 0;                 // (no prefix has no rows)
        p.seqs = i ? 1 : (int32_t)S;
        // whole units, or what there is: of the strides, and with the addresses
        const bool plain = d->format == kPlain;
        const int size = plain ? es : 1, most = plain ? 16 : unit;
        uint64_t bits = plain ? d->D * es : row_bytes(d->format, d->D);
        for (int j = 0; j < 3; ++j) bits |= (uint64_t)(p.ks[j] * size) | (uint64_t)(p.vs[j] * size);
        auto width = [&](uint64_t x) {
            const int w = (int)std::min<uint64_t>(most, x & -x);
            return w >= 4 ? w : size;
        };
        p.width = width(bits | (uintptr_t)x.k | (uintptr_t)x.v);
        if (p.caches == 0 || p.T == 0) continue;
        // (a row's offset in a tile has to be within 31 bits)
        const int64_t far = (int64_t)1 << 24;
        if (width(bits) != most || (plain && d->D % 8) || (d->format == kE2M1 && d->D % 2) ||
            p.ks[1] >= far || p.vs[1] >= far ||
            (!plain && (p.kss[1] >= far || p.vss[1] >= far)))
            c->any_strides = 1;
        if (c->any_strides || p.width != most) c->any = 1;
    }
    return MP3D_OK;
}

// The workspace of a call.  Its plan depends on whether kv_len is given and on
// the caches' addresses, which a caller may not have yet: the most that the call
// takes with any of them.
size_t cached_workspace(const CachedArgs &c, int cus)
{
    size_t most = 0;
    const int32_t lengths = 0;             // (its address is looked at, no more)
    for (int any = c.any_strides; any <= 1; ++any)
        for (const int32_t *len : {(const int32_t *)nullptr, &lengths}) {
            CachedArgs x = c;
            x.any = any;
            x.part[1].len = len;
            most = std::max(most, plan_attn_cached(&x, cus));
        }
    return most;
}

}  // namespace

}  // namespace mp3d

using namespace mp3d;

extern "C" {

int mp3d_cache_write(const mp3d_cache *cache, int format, const void *k, const void *v, int dtype,
                     int64_t T, int32_t H, int32_t D, const int64_t *k_stride,
                     const int64_t *v_stride, const int32_t *start, const int32_t *count,
                     void *stream)
{
    return cache_call(cache, format, const_cast<void *>(k), const_cast<void *>(v), dtype, T, H, D,
                      k_stride, v_stride, start, count, false, stream);
}

int mp3d_cache_read(const mp3d_cache *cache, int format, void *k, void *v, int dtype, int64_t T,
                    int32_t H, int32_t D, const int32_t *start, const int32_t *count, void *stream)
{
    return cache_call(cache, format, k, v, dtype, T, H, D, nullptr, nullptr, start, count, true,
                      stream);
}

int mp3d_attention_cached_workspace_bytes(const mp3d_attention_cache *d, size_t *bytes)
{
    if (!bytes) return fail(MP3D_EINVAL, "bytes is NULL");
    CachedArgs c;
    const int rc = cached_args(d, &c);
    if (rc) return rc;
    *bytes = c.a.B == 0 || c.a.Tq == 0 ? 0 : cached_workspace(c, device_cus());
    return MP3D_OK;
}

int mp3d_attention_cached(const mp3d_attention_cache *d, const void *q, void *out, float *lse,
                          void *workspace, size_t workspace_bytes, void *stream)
{
    TimingScope timing_scope;
    CachedArgs c;
    int rc = cached_args(d, &c);
    if (rc) return rc;
    AttnArgs &a = c.a;
    if (a.B == 0 || a.Tq == 0) return MP3D_OK;
    if (!q || !out || !lse) return fail(MP3D_EINVAL, "a tensor is NULL");
    if ((rc = check_pointers(d->own, d->format, "own")) ||
        (rc = check_pointers(d->prefix, d->format, "prefix")))
        return rc;
    const int es = elem_bytes(d->dtype);
    if (!aligned(q, es) || !aligned(out, 16) || !aligned(lse, 4))
        return fail(MP3D_EINVAL, "a tensor is not aligned (out: 16 bytes, others: an element)");
    if (d->format == kPlain && !(aligned(d->own.k, es) && aligned(d->own.v, es) &&
                                 aligned(d->prefix.k, es) && aligned(d->prefix.v, es)))
        return fail(MP3D_EINVAL, "a cache is not aligned to its elements");
    a.q = q;
    a.out = out;
    a.lse = lse;
    a.vec = wide_rows(q, a.qs, es) && a.D % 8 == 0;
    const int cus = device_cus();
    if ((rc = check_workspace(workspace, workspace_bytes, cached_workspace(c, cus)))) return rc;
    plan_attn_cached(&c, cus);
    if ((rc = check_launch(c.part[0].blocks + c.part[1].blocks))) return rc;
    place_attn_cached(&c, workspace);
    if (log_enabled())
        fprintf(stderr, "[mp3d] attention over caches dtype=%d format=%d prefix: %d chunks of %d, "
                "wr=%d; own: %d of %d, wr=%d\n", d->dtype, d->format, c.part[0].nsplit,
                c.part[0].chunk, c.part[0].wr, c.part[1].nsplit, c.part[1].chunk, c.part[1].wr);
    return by_dtype(d->dtype, [&](auto t) {
        return hip_status(launch_attn_cached<decltype(t)>(c, (hipStream_t)stream),
                          "attention over caches launch");
    });
}

}  // extern "C"
