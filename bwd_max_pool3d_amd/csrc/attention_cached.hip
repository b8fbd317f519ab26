// attention_cached.hip -- attention over caches: how the work is cut, and the
// join of its parts (the kernel that walks the caches: attention_cached.hpp).
#include "attention_cached.hpp"

namespace mp3d {

namespace {

constexpr int kJoinGroups = 8;
constexpr int64_t kJoinRow = 1 << 22;       // workgroups of the join in a row of its grid

// Joins the chunks of a row: a workgroup per row, 8 groups of 32 lanes with 4
// channels a lane.  The groups take the chunks that the row has keys in, in
// turn, each with a running maximum of its own, and are joined in LDS in a
// fixed order.
template <typename T>
__global__ __launch_bounds__(32 * kJoinGroups) void cached_join_kernel(CachedArgs c)
{
    using R = typename T::raw;
    constexpr int NG = kJoinGroups;
    __shared__ __align__(16) float jo[NG][kAttnMaxD];
    __shared__ float jm[NG], jl[NG];
    const AttnArgs &a = c.a;
    const int tid = threadIdx.x, g = tid >> 5, d0 = (tid & 31) * 4, per = a.Tq * a.G;
    const int64_t total = (int64_t)a.B * a.Hq * a.Tq, row = blockIdx.y * (int64_t)gridDim.x + blockIdx.x;
    if (row >= total) return;
    const int64_t bh = row / per;
    const int r = (int)(row - bh * per), t = r / a.G;
    const int b = (int)(bh / a.Hk), h = (int)(bh % a.Hk) * a.G + (r - t * a.G);
    const int ds = cached_stride(a.D);
    // its chunks of the prefix, then of the own cache
    const CachedPart &pre = c.part[0], &own = c.part[1];
    int n0 = 0, n1 = 0;
    if (pre.nsplit > 0) {
        const int end = cached_len(pre, b / pre.seqs);
        n0 = end / pre.chunk + (end % pre.chunk != 0);
    }
    if (own.nsplit > 0) {
        const int end = cached_end(c, true, cached_len(own, b), t);
        n1 = end / own.chunk + (end % own.chunk != 0);
    }
    float m = kNegInf, l = 0.f;
    f32x4 o = f32x4(0.f);
#pragma unroll 4
    for (int s = g; s < n0 + n1; s += NG) {
        const int64_t at = (s < n0 ? s : pre.nsplit + s - n0) * total + row;
        const float2 v = *(const float2 *)(a.part_ml + 2 * at);
        const f32x4 x = d0 < ds ? *(const f32x4 *)(a.part_o + at * ds + d0) : f32x4(0.f);
        const float mn = fmaxf(m, v.x), ms = mn == kNegInf ? 0.f : mn;
        const float fo = __builtin_amdgcn_exp2f(m - ms), fn = __builtin_amdgcn_exp2f(v.x - ms);
        l = l * fo + fn * v.y;
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = o[e] * fo + fn * x[e];
        m = mn;
    }
    *(f32x4 *)&jo[g][d0] = o;
    if (d0 == 0) {
        jm[g] = m;
        jl[g] = l;
    }
    __syncthreads();
    if (tid >= kAttnMaxD) return;
    float mt = kNegInf, lt = 0.f, ot = 0.f;
#pragma unroll
    for (int x = 0; x < NG; ++x) mt = fmaxf(mt, jm[x]);
    const float ms = mt == kNegInf ? 0.f : mt;
#pragma unroll
    for (int x = 0; x < NG; ++x) {
        const float f = __builtin_amdgcn_exp2f(jm[x] - ms);
        lt = fmaf(f, jl[x], lt);
        ot = fmaf(f, jo[x][tid], ot);
    }
    if (tid < a.D)
        ((R *)a.out)[(((int64_t)b * a.Tq + t) * a.Hq + h) * a.D + tid] =
            T::narrow(lt == 0.f ? 0.f : ot / lt);
    if (tid == 0)
        a.lse[((int64_t)b * a.Hq + h) * a.Tq + t] =
            lt == 0.f ? kNegInf : (mt + log2f(lt)) * kLn2;
}

}  // namespace

// Rows a workgroup, chunks and workgroups of both parts; returns the
// workspace's bytes.
size_t plan_attn_cached(CachedArgs *c)
{
    AttnArgs &a = c->a;
    for (CachedPart &p : c->part) {
        p.nsplit = 0;
        p.units = p.blocks = 0;
        p.chunk = 1;
        p.wr = 1;
        p.nrb = 1;
        if (p.caches == 0 || p.T == 0) continue;
        p.rows = (int32_t)((int64_t)p.seqs * a.Tq * a.G);
        if (c->format != kPlain) p.wr = p.rows <= 32 ? 1 : p.rows <= 64 ? 2 : 4;
        p.nrb = (p.rows + 32 * p.wr - 1) / (32 * p.wr);
        // tiles that a workgroup takes in one step
        const int64_t unit = (int64_t)kCachedKeys * (kCachedWaves / p.wr);
        const int64_t most = (p.T + unit - 1) / unit;
        const int64_t base = (int64_t)p.nrb * a.Hk * p.caches;
        const int64_t want = (p.wr > 1 ? 2 : 8) * device_cus();
        int64_t n = (want + base - 1) / base;
        n = n > most ? most : n;
        const int64_t chunk = (most + n - 1) / n * unit;
        p.chunk = (int32_t)chunk;
        p.nsplit = (int32_t)((p.T + chunk - 1) / chunk);
        p.units = (int64_t)a.Hk * p.caches * p.nsplit;
        p.blocks = p.nrb > 1 ? (p.units + 7) / 8 * 8 * p.nrb : p.units;
    }
    CachedPart &own = c->part[1];
    if (c->part[0].nsplit + own.nsplit == 0) {
        // no key anywhere: one workgroup a row block writes the zeros
        own.rows = a.Tq * a.G;
        own.nrb = (own.rows + 31) / 32;
        own.nsplit = 1;
        own.units = (int64_t)a.Hk * a.B;
        own.blocks = own.nrb > 1 ? (own.units + 7) / 8 * 8 * own.nrb : own.units;
    }
    const int64_t slots = c->part[0].nsplit + own.nsplit;
    if (slots == 1) return 0;
    const size_t all = (size_t)slots * a.B * a.Hq * a.Tq;
    return ((2 * all + 3) / 4 * 4 + all * cached_stride(a.D)) * sizeof(float);
}

void place_attn_cached(CachedArgs *c, void *workspace)
{
    const size_t all = (size_t)(c->part[0].nsplit + c->part[1].nsplit) * c->a.B * c->a.Hq * c->a.Tq;
    c->a.part_ml = (float *)workspace;
    c->a.part_o = c->a.part_ml + (2 * all + 3) / 4 * 4;
}

template <typename T>
hipError_t launch_attn_cached(const CachedArgs &c, hipStream_t s)
{
    const hipError_t e = c.format == kPlain  ? launch_cached_plain<T>(c, s)
                         : c.format == kE4M3 ? launch_cached_e4m3<T>(c, s)
                                             : launch_cached_e2m1<T>(c, s);
    if (e != hipSuccess) return e;         // the join would read what was not written
    if (c.part[0].nsplit + c.part[1].nsplit > 1) {
        // (a launch's first dimension takes 2^24 workgroups of 256)
        const int64_t rows = (int64_t)c.a.B * c.a.Hq * c.a.Tq, x = rows < kJoinRow ? rows : kJoinRow;
        launch_kernel((cached_join_kernel<T>), dim3((uint32_t)x, (uint32_t)((rows + x - 1) / x)),
                      dim3(32 * kJoinGroups), 0, s, c);
    }
    return hipGetLastError();
}

template hipError_t launch_attn_cached<F32>(const CachedArgs &, hipStream_t);
template hipError_t launch_attn_cached<F16>(const CachedArgs &, hipStream_t);
template hipError_t launch_attn_cached<BF16>(const CachedArgs &, hipStream_t);

}  // namespace mp3d
