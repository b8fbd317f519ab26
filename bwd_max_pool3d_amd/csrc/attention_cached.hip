// attention_cached.hip -- attention over caches: how the work is cut, and the
// join of its parts (the kernel that walks the caches: attention_cached.hpp).
#include "attention_cached.hpp"

#include <algorithm>

namespace mp3d {

namespace {

constexpr int kJoinGroups = 8;
constexpr int kAlone = 4 * kCachedKeys * kCachedWaves;    // keys that are not split
constexpr int64_t kJoinRow = 1 << 22;       // workgroups of the join in a row of its grid

// Joins the chunks of a row: NG groups of 32 lanes a row, with 4 channels a
// lane.  The groups take the chunks that the row has keys in, in turn, each
// with a running maximum of its own, and are joined in LDS in a fixed order.
// Few chunks: a group a row, and nothing to join.
template <typename T, int NG>
__global__ __launch_bounds__(32 * kJoinGroups) void cached_join_kernel(CachedArgs c)
{
    using R = typename T::raw;
    __shared__ __align__(16) float jo[kJoinGroups][kAttnMaxD];
    __shared__ float jm[kJoinGroups], jl[kJoinGroups];
    const AttnArgs &a = c.a;
    const int tid = threadIdx.x, group = tid >> 5, g = group % NG, d0 = (tid & 31) * 4,
              per = a.Tq * a.G;
    const int64_t total = (int64_t)a.B * a.Hq * a.Tq;
    const int64_t row = (blockIdx.y * (int64_t)gridDim.x + blockIdx.x) * (kJoinGroups / NG) + group / NG;
    if (row >= total) return;              // (with NG groups of kJoinGroups, all of them)
    const uint32_t in_b = (uint32_t)a.Hk * per;                    // rows of a sequence
    const int b = (int)(row / in_b);
    const uint32_t in = (uint32_t)(row - (int64_t)b * in_b), hk = in / (uint32_t)per, r = in - hk * per,
                   t = r / (uint32_t)a.G;
    const int h = hk * a.G + (r - t * a.G);
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
    R *const out = (R *)a.out + (((int64_t)b * a.Tq + t) * a.Hq + h) * a.D;
    float *const lse = a.lse + ((int64_t)b * a.Hq + h) * a.Tq + t;
    if constexpr (NG == 1) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (d0 + e < a.D) out[d0 + e] = T::narrow(l == 0.f ? 0.f : o[e] / l);
        if (d0 == 0) *lse = l == 0.f ? kNegInf : (m + log2f(l)) * kLn2;
    } else {
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
        if (tid < a.D) out[tid] = T::narrow(lt == 0.f ? 0.f : ot / lt);
        if (tid == 0) *lse = lt == 0.f ? kNegInf : (mt + log2f(lt)) * kLn2;
    }
}

}  // namespace

// Rows a workgroup, chunks and workgroups of both parts on a device of `cus`
// CUs; returns the workspace's bytes.  By the caches' rows, T: the lengths in use
// are on the device, and chunks behind them have nothing to do (one of 1000 keys,
// 32 heads on 8, e4m3: 11.4 us in a cache of 1024, 19.5 in one of 131072).
size_t plan_attn_cached(CachedArgs *c, int cus)
{
    AttnArgs &a = c->a;
    constexpr int64_t kStep = kCachedKeys * kCachedWaves;  // keys that a workgroup takes at a time
    // (a step of 128 rows takes three times one of 16; as twice it measured 4 %
    // more, as four times up to 30 %)
    auto kWeight = [](const CachedPart &p) -> int64_t { return p.mb == 16 ? 1 : 3; };
    auto blocks = [&](CachedPart &p) {
        p.units = (int64_t)a.Hk * p.caches * p.nsplit;
        p.blocks = p.nrb > 1 ? (p.units + 7) / 8 * 8 * p.nrb : p.units;
    };
    const bool plain = c->format == kPlain;
    const int few = plain || std::max(c->part[0].T, c->part[1].T) >= 16384 ? 32 : 64;
    int64_t cost = 0;                      // steps of 16 rows, over all workgroups
    bool wide = false;
    for (CachedPart &p : c->part) {
        p.nsplit = 0;
        p.units = p.blocks = 0;
        p.chunk = 1;
        p.rows = (int32_t)((int64_t)p.seqs * a.Tq * a.G);
        // Blocks of 16 rows or of 128.  Over a prefix, 16 heads on 4 of 128,
        // bfloat16, 48 / 64 / 96 / 256 rows: 10935 e4m3 keys 19.6 / 20.7 / 24.9 /
        // 39.1 us by 16, 20.5 / 22.8 / 24.9 / 31.3 by 128; 32768: 28.8 / 35.5 /
        // 41.7 / 74.8 and 28.8 / 30.2 / 32.1 / 43.9; plain, 10935: 21.6 / 20.4 /
        // 23.7 / 33.8 and 18.8 / 19.9 / 21.2 / 28.6.  (float32 is bound by its
        // matrix instructions either way, and 128 rows leave waves idle: 15
        // sequences of 7 tokens on three prefixes of 245 32 us by 128, 16 by 16.)
        // The same bound is taken with other widths and a cap, where 16 stay ahead
        // longer (48 / 64 / 96 / 256 rows: 64 channels, e4m3, 10935 12.7 / 13.1 /
        // 15.4 / 22.2 and 14.9 / 15.7 / 17.8 / 21.6; 128 and a cap, e4m3, 32768 26.9 /
        // 30.5 / 38.2 / 71.6 and 38.1 / 38.9 / 41.6 / 58.8; 32 channels, e4m3, 32768
        // 18.2 / 19.3 / 23.5 / 40.7 and 19.7 / 20.1 / 21.3 / 28.8).
        // One bound for both parts: a prefix, which has at least an own cache's
        // rows, then never has the smaller blocks (run_cached_rows).
        p.mb = p.rows <= few || c->f32 || (plain && c->any) ? 16 : 32;
        p.wr = p.mb == 16 ? 1 : 4;
        p.nrb = (p.rows + p.mb * p.wr - 1) / (p.mb * p.wr);
        if (p.caches == 0 || p.T == 0) continue;
        wide |= p.mb == 32;
        cost += (int64_t)p.nrb * a.Hk * p.caches * ((p.T + kStep - 1) / kStep) * kWeight(p);
    }
    // One round of workgroups: as many as run at once.  (e4m3 by three a CU where
    // the kernels leave room for two, and by two: 16 caches of 16384, 32 heads on 8
    // of 128 in float32 257 and 238 us, of 100 in bfloat16, which cannot go by 16
    // bytes, 316 and 240; plain float32 over 64 channels, which has room for one, by
    // two and by one 362 and 369, one cache of 32768 41 and 35, 8 of 1500 48 and
    // 54.)  Of 16 rows four where lengths are given, which leave some without keys
    // (16 caches of 9728 to 32768, e4m3: 145 us for three a CU, 134 for four, 150 to
    // 164 for six to twelve; plain 275 and 254).
    const int at_once = cached_occupancy(c->f32 ? 4 : 2, c->format, a.D <= 64 ? 64 : 128,
                                         c->any || attn_general(a), wide ? 32 : 16);
    const int64_t once = (int64_t)cus * std::max(2, at_once);
    const int64_t want = !wide && c->part[1].len ? 4 * (int64_t)cus : once;
    // Short calls: a workgroup's start takes as long as five steps and each
    // writes a chunk to join, so a workgroup takes up to three steps before a
    // CU gets a second one, of float32, whose steps are long, a third.  8
    // sequences of 200 on 4000, 32 heads on 8, at least one step and by this
    // rule: plain 18.5 and 12.5 us, e4m3 16.8 and 13.5, float32 29.0 and 26.8; 4 x
    // 2048 plain 10.6 and 9.6; one sequence of 2048, which keeps one step, 9.1,
    // with two 9.5.  (float32 as the others: that case 22.7, but 15 sequences of 7
    // tokens on three prefixes of 245 18.5 us for 16.1.)
    const int64_t spread = cus * (c->f32 ? 2 : 1);
    const int64_t per = std::max((cost + want - 1) / want,
                                 std::min<int64_t>(3, (cost + spread - 1) / spread));
    for (CachedPart &p : c->part) {
        if (p.caches == 0 || p.T == 0) continue;
        const int64_t steps = (p.T + kStep - 1) / kStep;
        int64_t n = (per + kWeight(p) - 1) / kWeight(p);
        n = n > steps ? steps : n;
        p.nsplit = (int32_t)((steps + n - 1) / n);
        p.chunk = (int32_t)((steps + p.nsplit - 1) / p.nsplit * kStep);
        blocks(p);
    }
    CachedPart &own = c->part[1];
    // Few keys and nothing to join with: not split, which saves the join (one
    // sequence, 16 heads on 4, plain, 256 / 512 / 768 / 1024 keys: 6.4 / 7.9 / 9.4
    // / 10.9 us, split 8.7 / 8.5 / 9.4 / 9.3; e4m3 7.3 / 9.6 / 11.8 / 14.3 and 9.3 /
    // 9.1 / 10.0 / 9.8; 32 sequences, e4m3, 9.1 / 11.4 / 13.7 / 16.2 and 10.8 / 13.1 /
    // 14.6 / 16.8), and a launch.  (float32 takes the same bound, though its steps
    // are longer: one sequence, e4m3, 256 / 512 / 1024 keys 14.8 / 22.6 / 38.2 whole
    // and 13.6 / 13.6 / 13.8 split; 32 sequences 15.4 / 24.2 / 41.7 and 14.5 / 20.4 /
    // 28.3, plain 15.8 / 23.5 / 36.5 and 14.9 / 29.2 / 39.1.)
    for (int i = 0; i < 2; ++i) {
        CachedPart &p = c->part[i];
        const bool many = (int64_t)p.nrb * a.Hk * p.caches >= 128;
        if (c->part[1 - i].nsplit == 0 && p.T <= (many ? 2 : 1) * kAlone) {
            p.nsplit = p.T > 0;
            p.chunk = 2 * kAlone;
            blocks(p);
        }
    }
    if (c->part[0].nsplit + own.nsplit == 0) {
        own.nsplit = 1;                    // no key anywhere: the zeros are written all the same
        blocks(own);
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
    const hipError_t e = c.format == kPlain  ? launch_cached<T, kPlain>(c, s)
                         : c.format == kE4M3 ? launch_cached<T, kE4M3>(c, s)
                                             : launch_cached<T, kE2M1>(c, s);
    if (e != hipSuccess) return e;         // the join would read what was not written
    const int slots = c.part[0].nsplit + c.part[1].nsplit;
    if (slots > 1) {
        // A group a row where rows are many and chunks few (8192 rows of 8: 9.8
        // us, 17 by eight groups; 512 rows of 8: 5.8 and 5.2).
        const int64_t rows = (int64_t)c.a.B * c.a.Hq * c.a.Tq;
        const bool one = rows >= 4096 && slots <= 16;
        const int64_t n = one ? (rows + kJoinGroups - 1) / kJoinGroups : rows;
        // (a launch's first dimension takes 2^24 workgroups of 256)
        const int64_t x = n < kJoinRow ? n : kJoinRow;
        const dim3 grid((uint32_t)x, (uint32_t)((n + x - 1) / x)), block(32 * kJoinGroups);
        if (one) launch_kernel((cached_join_kernel<T, 1>), grid, block, 0, s, c);
        else launch_kernel((cached_join_kernel<T, kJoinGroups>), grid, block, 0, s, c);
    }
    return hipGetLastError();
}

template hipError_t launch_attn_cached<F32>(const CachedArgs &, hipStream_t);
template hipError_t launch_attn_cached<F16>(const CachedArgs &, hipStream_t);
template hipError_t launch_attn_cached<BF16>(const CachedArgs &, hipStream_t);

}  // namespace mp3d
