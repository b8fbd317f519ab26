// api_tokens.hip -- the C ABI of the token operators (include/mp3d.h, the
// section on operators over a pooled volume's tokens): argument checks, the
// choice of kernel, workspaces.  Every check runs before the first launch.
#include <stdio.h>

#include <initializer_list>

#include "api_tokens.hpp"

namespace mp3d {

namespace {

// --- rotary positions

int rope(const void *q, const void *k, void *qo, void *ko, int dtype, int64_t B, int64_t T,
         int32_t Hq, int32_t Hk, int32_t D, const int64_t *q_stride, const int64_t *k_stride,
         const int64_t *qo_stride, const int64_t *ko_stride, const float *inv_freq,
         const int32_t *pairs, const int32_t *positions, const int32_t *grid, int interleaved,
         float sign, void *stream)
{
    TimingScope timing_scope;
    int rc = check_dtype(dtype);
    if (rc) return rc;
    if (B < 0 || T < 0 || Hq < 0 || Hk < 0 || Hq > 65536 || Hk > 65536)
        return fail(MP3D_EINVAL, "B and T must be >= 0, the head counts in 0 .. 65536");
    if (D < 1 || D > 65536) return fail(MP3D_EINVAL, "D=%d must be in 1 .. 65536", D);
    if (T > kMaxLen || B > kMaxLen || too_many(B, T, (int64_t)Hq + Hk, D))
        return fail(MP3D_EOVERFLOW, "B*T*H*D is out of range");
    if (!pairs) return fail(MP3D_EINVAL, "pairs is NULL");
    int64_t P = 0;
    for (int a = 0; a < 3; ++a) {
        if (pairs[a] < 0 || pairs[a] > D)
            return fail(MP3D_EINVAL, "pairs[%d]=%d is out of range", a, pairs[a]);
        P += pairs[a];
    }
    if (2 * P > D)
        return fail(MP3D_EINVAL, "%lld pairs do not fit %d channels", (long long)P, D);
    if (interleaved != 0 && interleaved != 1)
        return fail(MP3D_EINVAL, "interleaved must be 0 or 1");
    if (positions && grid) return fail(MP3D_EINVAL, "give either positions or grid");
    if (grid) {
        for (int a = 0; a < 3; ++a)
            if (grid[a] < 1) return fail(MP3D_EINVAL, "grid extents must be >= 1");
        if ((int64_t)grid[0] * grid[1] > kInt32Max ||
            (int64_t)grid[0] * grid[1] * grid[2] != T)
            return fail(MP3D_EINVAL, "T=%lld tokens do not fill a grid of %d x %d x %d",
                        (long long)T, grid[0], grid[1], grid[2]);
    }
    if (B == 0 || T == 0 || Hq + Hk == 0) return MP3D_OK;
    if (!positions && !grid) return fail(MP3D_EINVAL, "give either positions or grid");
    if (P > 0 && !inv_freq) return fail(MP3D_EINVAL, "inv_freq is NULL");
    if (Hq > 0 && (!q || !qo)) return fail(MP3D_EINVAL, "q or its output is NULL");
    if (Hk > 0 && (!k || !ko)) return fail(MP3D_EINVAL, "k or its output is NULL");

    RopePlan p = {};
    const int es = elem_bytes(dtype);
    const void *src[2] = {q, k};
    void *dst[2] = {qo, ko};
    const int64_t *ss[2] = {q_stride, k_stride}, *ds[2] = {qo_stride, ko_stride};
    const char *names[2] = {"q", "k"};
    const int32_t heads[2] = {Hq, Hk};
    int vec = 16 / es;
    // the widest access that divides every row's start, the halves and the rest
    auto fits = [&](int64_t elems) {
        while (vec > 1 && elems % vec) vec /= 2;
    };
    fits(D);
    fits(interleaved ? 2 * P : P);
    for (int i = 0; i < 2; ++i) {
        p.heads[i] = heads[i];
        if (!heads[i]) continue;
        if ((rc = check_strides(ss[i], names[i])) || (rc = check_strides(ds[i], "output")))
            return rc;
        p.src[i] = src[i];
        p.dst[i] = dst[i];
        for (int j = 0; j < 3; ++j) {
            p.ss[i][j] = ss[i][j];
            p.ds[i][j] = ds[i][j];
            fits(ss[i][j]);
            fits(ds[i][j]);
        }
        if (!aligned(src[i], es) || !aligned(dst[i], es))
            return fail(MP3D_EINVAL, "%s is not aligned to its elements", names[i]);
        while (vec > 1 && !(aligned(src[i], (int64_t)vec * es) &&
                            aligned(dst[i], (int64_t)vec * es)))
            vec /= 2;
    }
    if (vec == 4 && es == 2) vec = 2;      // the kernels' widths: 16 bytes, 2 elements, 1
    p.pos = positions;
    p.freq = inv_freq;
    p.B = B;
    p.T = T;
    p.D = D;
    p.P = (int32_t)P;
    p.e0 = pairs[0];
    p.e1 = pairs[0] + pairs[1];
    p.gh = grid ? grid[1] : 1;
    p.gw = grid ? grid[2] : 1;
    p.interleaved = interleaved;
    p.sign = sign;
    p.vec = vec;
    const int np = interleaved ? (vec > 1 ? vec / 2 : 1) : vec;
    p.rot_units = (int32_t)(P / np);
    p.units = p.rot_units + (int32_t)((D - 2 * P) / vec);
    p.tpb = p.units < kBlock ? kBlock / p.units : 1;
    plan_rope_heads(&p);
    if (log_enabled())
        fprintf(stderr, "[mp3d] rope dtype=%d vec=%d units=%d heads/thread=%d\n", dtype, vec,
                p.units, p.hpt);
    return by_dtype(dtype, [&](auto t) {
        return hip_status(launch_rope<decltype(t)>(p, (hipStream_t)stream), "rope launch");
    });
}

// --- gated norm

int norm_plan(NormPlan *p, const void *x, const void *h, const void *gate,
              const void *post_weight, const void *pre_weight, int dtype, int64_t rows, int32_t C,
              int64_t gate_rows, float residual_scale, int kind, int parts, float eps)
{
    int rc = check_dtype(dtype);
    if (rc) return rc;
    if (rows < 0) return fail(MP3D_EINVAL, "rows must be >= 0");
    if (C < 1 || C > kNormMaxC)
        return fail(MP3D_EINVAL, "C=%d must be in 1 .. %d", C, kNormMaxC);
    if (rows > kInt32Max || too_many(rows, C, 1, 1))
        return fail(MP3D_EOVERFLOW, "rows*C is out of range");
    if (kind != MP3D_NORM_RMS && kind != MP3D_NORM_LAYER)
        return fail(MP3D_EINVAL, "kind %d is not MP3D_NORM_RMS or MP3D_NORM_LAYER", kind);
    if (parts & ~(MP3D_NORM_POST | MP3D_NORM_PRE))
        return fail(MP3D_EINVAL, "parts %d has unknown bits", parts);
    if (!(eps >= 0.f)) return fail(MP3D_EINVAL, "eps must be >= 0");
    const bool work = rows > 0;
    if (work && !x) return fail(MP3D_EINVAL, "x is NULL");
    if (work && !h && (gate || post_weight || (parts & MP3D_NORM_POST)))
        return fail(MP3D_EINVAL, "a gate, a post weight or a post norm needs h");
    if (work && !h && !(parts & MP3D_NORM_PRE))
        return fail(MP3D_EINVAL, "nothing to do: no h and no norm before the next block");
    if (pre_weight && !(parts & MP3D_NORM_PRE))
        return fail(MP3D_EINVAL, "a pre weight needs MP3D_NORM_PRE");
    if (gate && (gate_rows < 1 || rows % gate_rows))
        return fail(MP3D_EINVAL, "%lld rows do not divide among %lld gate rows", (long long)rows,
                    (long long)gate_rows);
    *p = NormPlan{};
    p->x = x;
    p->h = h;
    p->gate = gate;
    p->post = post_weight;
    p->pre = pre_weight;
    p->rows = rows;
    p->C = C;
    p->gate_rows = gate ? gate_rows : 0;
    p->rpg = gate ? rows / gate_rows : rows;
    p->rs = residual_scale;
    p->eps = eps;
    p->layer = kind == MP3D_NORM_LAYER;
    p->has_post = (parts & MP3D_NORM_POST) != 0;
    p->has_pre = (parts & MP3D_NORM_PRE) != 0;
    const int es = elem_bytes(dtype);
    for (const void *t : {x, h, gate, post_weight, pre_weight})
        if (!aligned(t, es)) return fail(MP3D_EINVAL, "a tensor is not aligned to its elements");
    return MP3D_OK;
}

bool all_aligned16(std::initializer_list<const void *> v)
{
    for (const void *p : v)
        if (!aligned(p, 16)) return false;
    return true;
}

// --- attention

int attn_args(const mp3d_attention *d, AttnArgs *a)
{
    if (!d) return fail(MP3D_EINVAL, "the attention descriptor is NULL");
    int rc = check_dtype(d->dtype);
    if (rc) return rc;
    if (d->B < 0 || d->Tq < 0 || d->Tk < 0)
        return fail(MP3D_EINVAL, "B, Tq and Tk must be >= 0");
    if (d->Hq < 1 || d->Hk < 1 || d->Hq % d->Hk)
        return fail(MP3D_EINVAL, "Hq=%d must be a positive multiple of Hk=%d", d->Hq, d->Hk);
    if (d->D < 1 || d->D > kAttnMaxD)
        return fail(MP3D_EINVAL, "D=%d must be in 1 .. %d", d->D, kAttnMaxD);
    if (d->Tq > kMaxLen || d->Tk > kMaxLen || d->B > kMaxLen || d->Tq * d->Hq > kInt32Max ||
        too_many(d->B, d->Tq, d->Hq, d->D) || too_many(d->B, d->Tk, d->Hk, d->D))
        return fail(MP3D_EOVERFLOW, "B*T*H*D is out of range");
    if (d->causal != 0 && d->causal != 1) return fail(MP3D_EINVAL, "causal must be 0 or 1");
    if (!(d->softcap == 0.f || (d->softcap >= 1e-30f && d->softcap <= 1e30f)))
        return fail(MP3D_EINVAL, "softcap must be 0 (none) or in 1e-30 .. 1e30");
    if (!(d->scale == d->scale) || d->scale > 1e30f || d->scale < -1e30f)
        return fail(MP3D_EINVAL, "scale must be finite");
    if (d->prefix && !d->causal) return fail(MP3D_EINVAL, "a prefix needs causal");
    if (d->doc_offsets && (d->n_docs < 1 || d->n_docs > kInt32Max - 1))
        return fail(MP3D_EINVAL, "n_docs must be >= 1");
    if (d->axes < 0 || d->axes > 3) return fail(MP3D_EINVAL, "axes must be in 0 .. 3");
    // (a tensor without elements may be NULL)
    if (d->axes > 0 && (!d->slopes || (d->B * d->Tq > 0 && !d->pos_q) ||
                        (d->B * d->Tk > 0 && !d->pos_k)))
        return fail(MP3D_EINVAL, "a distance bias needs slopes, pos_q and pos_k");
    if ((rc = check_strides(d->q_stride, "q")) || (rc = check_strides(d->k_stride, "k")) ||
        (rc = check_strides(d->v_stride, "v")))
        return rc;
    *a = AttnArgs{};
    for (int i = 0; i < 3; ++i) {
        a->qs[i] = d->q_stride[i];
        a->ks[i] = d->k_stride[i];
        a->vs[i] = d->v_stride[i];
    }
    a->B = (int32_t)d->B;
    a->Tq = (int32_t)d->Tq;
    a->Tk = (int32_t)d->Tk;
    a->Hq = d->Hq;
    a->Hk = d->Hk;
    a->G = d->Hq / d->Hk;
    a->D = d->D;
    a->scale = d->scale;
    a->cap = d->softcap;
    a->slopes = d->slopes;
    a->pos_q = d->pos_q;
    a->pos_k = d->pos_k;
    a->axes = d->axes;
    a->causal = d->causal;
    a->ndocs = d->doc_offsets ? d->n_docs : 0;
    a->docs = d->doc_offsets;
    a->prefix = d->prefix;
    a->kv_len = d->kv_len;
    a->f16 = d->dtype == MP3D_F16;
    return MP3D_OK;
}

}  // namespace

}  // namespace mp3d

using namespace mp3d;

extern "C" {

int mp3d_rope_forward(const void *q, const void *k, void *q_out, void *k_out, int dtype, int64_t B,
                      int64_t T, int32_t Hq, int32_t Hk, int32_t D, const int64_t *q_stride,
                      const int64_t *k_stride, const int64_t *q_out_stride,
                      const int64_t *k_out_stride, const float *inv_freq, const int32_t *pairs,
                      const int32_t *positions, const int32_t *grid, int interleaved, void *stream)
{
    return rope(q, k, q_out, k_out, dtype, B, T, Hq, Hk, D, q_stride, k_stride, q_out_stride,
                k_out_stride, inv_freq, pairs, positions, grid, interleaved, 1.f, stream);
}

int mp3d_rope_backward(const void *gq, const void *gk, void *gq_out, void *gk_out, int dtype,
                       int64_t B, int64_t T, int32_t Hq, int32_t Hk, int32_t D,
                       const int64_t *q_stride, const int64_t *k_stride,
                       const int64_t *q_out_stride, const int64_t *k_out_stride,
                       const float *inv_freq, const int32_t *pairs, const int32_t *positions,
                       const int32_t *grid, int interleaved, void *stream)
{
    return rope(gq, gk, gq_out, gk_out, dtype, B, T, Hq, Hk, D, q_stride, k_stride, q_out_stride,
                k_out_stride, inv_freq, pairs, positions, grid, interleaved, -1.f, stream);
}

int mp3d_gated_norm_forward(const void *x, const void *h, const void *gate,
                            const void *post_weight, const void *pre_weight, void *y, void *z,
                            float *stats, int dtype, int64_t rows, int32_t C, int64_t gate_rows,
                            float residual_scale, int kind, int parts, float eps, void *stream)
{
    TimingScope timing_scope;
    NormPlan p;
    int rc = norm_plan(&p, x, h, gate, post_weight, pre_weight, dtype, rows, C, gate_rows,
                       residual_scale, kind, parts, eps);
    if (rc) return rc;
    if (rows == 0) return MP3D_OK;
    if ((h && !y) || (p.has_pre && !z)) return fail(MP3D_EINVAL, "an output is NULL");
    const int es = elem_bytes(dtype);
    if (!aligned(y, es) || !aligned(z, es) || !aligned(stats, 16))
        return fail(MP3D_EINVAL, "an output is not aligned");
    p.y = y;
    p.z = z;
    p.stats = stats;
    plan_norm(&p, es, all_aligned16({x, h, gate, post_weight, pre_weight, y, z}));
    if (log_enabled())
        fprintf(stderr, "[mp3d] gated norm forward dtype=%d threads=%d ept=%d vec=%d\n", dtype,
                p.threads, p.ept, p.vec);
    return by_dtype(dtype, [&](auto t) {
        return hip_status(launch_norm_forward<decltype(t)>(p, (hipStream_t)stream),
                          "gated norm forward launch");
    });
}

int mp3d_gated_norm_workspace_bytes(int dtype, int64_t rows, int32_t C, int64_t gate_rows,
                                    size_t *bytes)
{
    if (!bytes) return fail(MP3D_EINVAL, "bytes is NULL");
    int rc = check_dtype(dtype);
    if (rc) return rc;
    if (rows < 0 || rows > kInt32Max || C < 1 || C > kNormMaxC || gate_rows < 0 ||
        (gate_rows > 0 && rows % gate_rows))
        return fail(MP3D_EINVAL, "rows, C or gate_rows is out of range");
    NormPlan p = {};
    p.rows = rows;
    p.C = C;
    p.gate_rows = gate_rows;
    plan_norm(&p, elem_bytes(dtype), false);
    *bytes = rows ? plan_norm_backward(&p) : 0;
    return MP3D_OK;
}

int mp3d_gated_norm_backward(const void *dy, const void *dz, const void *x, const void *h,
                             const void *gate, const void *post_weight, const void *pre_weight,
                             const float *stats, void *dx, void *dh, float *dgate,
                             float *dpost_weight, float *dpre_weight, int dtype, int64_t rows,
                             int32_t C, int64_t gate_rows, float residual_scale, int kind,
                             int parts, float eps, void *workspace, size_t workspace_bytes,
                             void *stream)
{
    TimingScope timing_scope;
    NormPlan p;
    int rc = norm_plan(&p, x, h, gate, post_weight, pre_weight, dtype, rows, C, gate_rows,
                       residual_scale, kind, parts, eps);
    if (rc) return rc;
    if (rows == 0) {
        // sums over no rows
        if (gate && dgate && too_many(gate_rows, C, 1, 1))
            return fail(MP3D_EOVERFLOW, "gate_rows*C is out of range");
        p.dgate = gate ? dgate : nullptr;
        p.dpost = dpost_weight;
        p.dpre = dpre_weight;
        return hip_status(launch_norm_no_rows(p, (hipStream_t)stream), "gated norm launch");
    }
    if (!stats || !dx || (h && !dh) || (p.has_pre && !dz))
        return fail(MP3D_EINVAL, "stats, dz or an output is NULL");
    if ((dgate == nullptr) != (gate == nullptr))
        return fail(MP3D_EINVAL, "dgate goes with gate");
    if ((dpost_weight && !post_weight) || (dpre_weight && !pre_weight))
        return fail(MP3D_EINVAL, "a weight's gradient needs the weight");
    const int es = elem_bytes(dtype);
    for (const void *t : {dy, dz, (const void *)dx, (const void *)dh})
        if (!aligned(t, es)) return fail(MP3D_EINVAL, "a tensor is not aligned to its elements");
    if (!aligned(stats, 16)) return fail(MP3D_EINVAL, "stats is not 16-byte aligned");
    p.dy = dy;
    p.dz = dz;
    p.stats = const_cast<float *>(stats);
    p.dx = dx;
    p.dh = dh;
    p.dgate = dgate;
    p.dpost = dpost_weight;
    p.dpre = dpre_weight;
    plan_norm(&p, es, all_aligned16({x, h, gate, post_weight, pre_weight, dy, dz, dx, dh}));
    const size_t need = plan_norm_backward(&p);
    if ((rc = check_workspace(workspace, workspace_bytes, need))) return rc;
    p.part = (float *)workspace;
    if (log_enabled())
        fprintf(stderr, "[mp3d] gated norm backward dtype=%d threads=%d ept=%d vec=%d nwg=%d\n",
                dtype, p.threads, p.ept, p.vec, p.nwg);
    return by_dtype(dtype, [&](auto t) {
        return hip_status(launch_norm_backward<decltype(t)>(p, (hipStream_t)stream),
                          "gated norm backward launch");
    });
}

int mp3d_attention_workspace_bytes(const mp3d_attention *d, int backward, size_t *bytes)
{
    if (!bytes) return fail(MP3D_EINVAL, "bytes is NULL");
    AttnArgs a;
    int rc = attn_args(d, &a);
    if (rc) return rc;
    *bytes = 0;
    // (the backward without queries still writes dk and dv)
    if (a.B == 0 || (a.Tq == 0 && (!backward || a.Tk == 0))) return MP3D_OK;
    if (backward) *bytes = plan_attn_backward(&a);
    else if (attn_split_wanted(a, d->dtype == MP3D_F32)) *bytes = plan_attn_split(&a);
    else *bytes = (size_t)attn_order_bytes(a, false);
    return MP3D_OK;
}

int mp3d_attention_forward(const mp3d_attention *d, const void *q, const void *k, const void *v,
                           void *out, float *lse, void *workspace, size_t workspace_bytes,
                           void *stream)
{
    TimingScope timing_scope;
    AttnArgs a;
    int rc = attn_args(d, &a);
    if (rc) return rc;
    if (a.B == 0 || a.Tq == 0) return MP3D_OK;
    if (!q || !out || !lse || (a.Tk > 0 && (!k || !v)))
        return fail(MP3D_EINVAL, "a tensor is NULL");
    const int es = elem_bytes(d->dtype);
    if (!aligned(q, es) || !aligned(k, es) || !aligned(v, es) || !aligned(out, 16) ||
        !aligned(lse, 4))
        return fail(MP3D_EINVAL, "a tensor is not aligned (out: 16 bytes, others: an element)");
    a.q = q;
    a.k = k;
    a.v = v;
    a.out = out;
    a.lse = lse;
    a.vec = wide_rows(q, a.qs, es) && wide_rows(k, a.ks, es) && wide_rows(v, a.vs, es);
    const bool split = attn_split_wanted(a, d->dtype == MP3D_F32);
    if (split) {
        if ((rc = check_workspace(workspace, workspace_bytes, plan_attn_split(&a)))) return rc;
        if ((rc = check_launch((int64_t)a.nrb * a.Hk * a.B * a.nsplit))) return rc;
        place_attn_split(&a, workspace);
    } else {
        const size_t need = (size_t)attn_order_bytes(a, false);
        if ((rc = check_workspace(workspace, workspace_bytes, need))) return rc;
        if ((rc = check_launch((int64_t)((a.Tq + kAttnRows - 1) / kAttnRows) * a.B * a.Hq)))
            return rc;
        a.order_q = need ? (int32_t *)workspace : nullptr;
    }
    if (log_enabled())
        fprintf(stderr, "[mp3d] attention forward dtype=%d %s vec=%d nsplit=%d\n", d->dtype,
                split ? "split" : "tiled", a.vec, a.nsplit);
    return by_dtype(d->dtype, [&](auto t) {
        using T = decltype(t);
        return hip_status(split ? launch_attn_split<T>(a, (hipStream_t)stream)
                                : launch_attn_forward<T>(a, (hipStream_t)stream),
                          "attention forward launch");
    });
}

int mp3d_attention_backward(const mp3d_attention *d, const void *dout, const int64_t *dout_stride,
                            const void *q, const void *k, const void *v, const void *out,
                            const float *lse, void *dq, void *dk, void *dv, void *workspace,
                            size_t workspace_bytes, void *stream)
{
    TimingScope timing_scope;
    AttnArgs a;
    int rc = attn_args(d, &a);
    if (rc) return rc;
    if (a.B == 0 || (a.Tq == 0 && a.Tk == 0)) return MP3D_OK;
    if ((rc = check_strides(dout_stride, "dout"))) return rc;
    if ((a.Tq > 0 && (!dout || !q || !out || !lse || !dq)) ||
        (a.Tk > 0 && (!k || !v || !dk || !dv)))
        return fail(MP3D_EINVAL, "a tensor is NULL");
    const int es = elem_bytes(d->dtype);
    if (!aligned(q, es) || !aligned(k, es) || !aligned(v, es) || !aligned(dout, es) ||
        !aligned(out, 16) || !aligned(dq, 16) || !aligned(dk, 16) || !aligned(dv, 16) ||
        !aligned(lse, 4))
        return fail(MP3D_EINVAL,
                    "a tensor is not aligned (out, dq, dk, dv: 16 bytes, others: an element)");
    a.q = q;
    a.k = k;
    a.v = v;
    a.dout = dout;
    a.out = const_cast<void *>(out);
    a.lse = const_cast<float *>(lse);
    a.dq = dq;
    a.dk = dk;
    a.dv = dv;
    for (int i = 0; i < 3; ++i) a.gs[i] = dout_stride[i];
    a.vec = wide_rows(q, a.qs, es) && wide_rows(k, a.ks, es) && wide_rows(v, a.vs, es) &&
            wide_rows(dout, a.gs, es);
    if ((rc = check_workspace(workspace, workspace_bytes, plan_attn_backward(&a)))) return rc;
    if ((rc = check_launch((int64_t)((a.Tq + kAttnRows - 1) / kAttnRows) * a.B * a.Hq)) ||
        (rc = check_launch((int64_t)((a.Tk + kAttnRows - 1) / kAttnRows) * a.B * a.Hk * a.gsplit)))
        return rc;
    place_attn_backward(&a, workspace);
    if (log_enabled())
        fprintf(stderr, "[mp3d] attention backward dtype=%d vec=%d gsplit=%d\n", d->dtype, a.vec,
                a.gsplit);
    return by_dtype(d->dtype, [&](auto t) {
        return hip_status(launch_attn_backward<decltype(t)>(a, (hipStream_t)stream),
                          "attention backward launch");
    });
}

}  // extern "C"
