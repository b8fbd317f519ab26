// attention_split.hip -- attention forward for few queries over many keys
// (single new tokens, short chunks), split over the keys and joined.
//
// Bound: HBM (the keys and values are read once; 4 G flop for each 2 bytes
// of them).  All query heads that share a key head, and all new tokens, are
// rows of one block of up to 32, so a key is read once for all of them.  A
// workgroup takes one block of rows and one chunk of keys; its four waves
// take tiles of 32 keys in turn, each through a part of LDS of its own, so
// no wave waits for another until the end.  The next tile's loads are in
// flight while a tile is worked on.  Every wave keeps its own running
// maximum and sum; the four are joined in LDS, the chunks by a second
// kernel.  Chunks have a fixed length whatever the sequence's: those past a
// short sequence's end return at once, so long and short caches balance.
#include "attention.hpp"

namespace mp3d {

namespace {

constexpr int kSplitWaves = 4;
constexpr int kSplitKeys = 32;             // keys of a wave's tile
constexpr int kSplitPad = 4;               // floats between the rows of the join
constexpr float kRaise = 8.f;

template <typename T, int DP>
constexpr uint32_t split_lds()
{
    const uint32_t tiles = kSplitWaves * 2 * kSplitKeys * DP * sizeof(typename T::raw);
    const uint32_t join = kSplitWaves * 32 * (DP + kSplitPad) * sizeof(float);
    return (tiles > join ? tiles : join) + kSplitWaves * (3 * kSplitKeys + 64) * sizeof(float);
}

template <typename T, int DP>
__global__ __launch_bounds__(64 * kSplitWaves, (sizeof(typename T::raw) * DP > 256 ? 1 : 2))
void attn_split_kernel(AttnArgs a)
{
    using R = typename T::raw;
    constexpr int KB = kSplitKeys, NC = DP / 16, ND = DP / 32, NW = kSplitWaves;
    extern __shared__ __align__(16) unsigned char smem[];
    constexpr uint32_t rest =
        split_lds<T, DP>() - kSplitWaves * (3 * kSplitKeys + 64) * sizeof(float);
    const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, col = lane & 31,
              half = lane >> 5;
    R *const kt = (R *)smem + wave * 2 * KB * DP, *const vt = kt + KB * DP;
    float *const pk = (float *)(smem + rest) + wave * 3 * KB;        // [3][KB]
    float *const ml = (float *)(smem + rest) + NW * 3 * KB;          // [NW][32][2]

    // blocks of one (sequence, key head) and chunk follow each other
    int64_t id = blockIdx.x;
    const int rb = id % a.nrb;
    id /= a.nrb;
    const int hk = id % a.Hk;
    id /= a.Hk;
    const int b = id % a.B, sp_no = id / a.B;
    const int rows = a.Tq * a.G, r = rb * 32 + col, rc = min(r, rows - 1);
    const int t = rc / a.G, h = hk * a.G + (rc - t * a.G);
    const Span sp = row_span(a, b, t);

    int glo = sp.hi > sp.lo ? sp.lo : 0x7fffffff, ghi = sp.hi, alo = sp.lo, ahi = sp.hi;
#pragma unroll
    for (int m = 16; m; m >>= 1) {
        glo = min(glo, __shfl_xor(glo, m));
        ghi = max(ghi, __shfl_xor(ghi, m));
        alo = max(alo, __shfl_xor(alo, m));
        ahi = min(ahi, __shfl_xor(ahi, m));
    }
    glo = max(__builtin_amdgcn_readfirstlane(glo), sp_no * a.chunk);   // the same in every wave
    ghi = min((int64_t)__builtin_amdgcn_readfirstlane(ghi), ((int64_t)sp_no + 1) * a.chunk);
    alo = __builtin_amdgcn_readfirstlane(alo);
    ahi = __builtin_amdgcn_readfirstlane(ahi);

    const R *kp = (const R *)a.k + b * a.ks[0] + hk * a.ks[2];
    const R *vp = (const R *)a.v + b * a.vs[0] + hk * a.vs[2];
    f32x16 o[ND];
#pragma unroll
    for (int d = 0; d < ND; ++d) o[d] = f32x16(0.f);
    float m = kNegInf, l = 0.f;
    bool dropped = false;

    if (glo < ghi) {
        const R *qp = (const R *)a.q + b * a.qs[0] + h * a.qs[2] + (int64_t)t * a.qs[1];
        Frag<T> qf[NC];
#pragma unroll
        for (int c = 0; c < NC; ++c) qf[c] = load8<T>(qp, c * 16 + half * 8, a.D, a.vec);
        const Scores sc = scores(a);
        float pq[3], sl[3];
        int64_t base[3];
#pragma unroll
        for (int x = 0; x < 3; ++x) {
            if (x >= a.axes) break;
            const int32_t *p = a.pos_q + ((int64_t)x * a.B + b) * a.Tq;
            base[x] = p[0];
            pq[x] = (float)(p[t] - base[x]);
            sl[x] = a.slopes[h * a.axes + x] * sc.slope;
        }
        TileRegs<T, DP, KB, 64> kr, vr;
        int32_t pr[3];
        auto fetch = [&](int k0) {
            kr.load(kp, a.ks[1], k0, glo, ghi, a.D, a.vec, lane);
            vr.load(vp, a.vs[1], k0, glo, ghi, a.D, a.vec, lane);
#pragma unroll
            for (int x = 0; x < 3; ++x)
                if (x < a.axes && lane < KB)
                    pr[x] = a.pos_k[((int64_t)x * a.B + b) * a.Tk + min(k0 + lane, a.Tk - 1)];
        };
        const int kbeg = glo / KB * KB + wave * KB;
        if (kbeg < ghi) fetch(kbeg);
        for (int k0 = kbeg; k0 < ghi; k0 += NW * KB) {
            const bool part = !(alo <= k0 && k0 + KB <= ahi);
            // the wave's LDS operations keep their order: no barrier, only the
            // compiler must not move them across
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
            if (part) dropped |= vr.drop();
            kr.store(kt, lane);
            vr.store(vt, lane);
#pragma unroll
            for (int x = 0; x < 3; ++x)
                if (x < a.axes && lane < KB) pk[x * KB + lane] = (float)(pr[x] - base[x]);
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
            if (k0 + NW * KB < ghi) fetch(k0 + NW * KB);

            f32x16 s = f32x16(0.f);
#pragma unroll
            for (int c = 0; c < NC; ++c)
                s = mma<T>(row_frag<T, DP>(kt, col, c * 16 + half * 8), qf[c], s);
            if (sc.multiply) s *= sc.scale;
            if (a.cap > 0.f) cap_scores<T>(s, sc);
#pragma unroll
            for (int x = 0; x < 3; ++x) {
                if (x >= a.axes) break;
                const f32x16 p = acc_rows(pk + x * KB, half);
#pragma unroll
                for (int e = 0; e < 16; ++e) s[e] = fmaf(-sl[x], fabsf(p[e] - pq[x]), s[e]);
            }
            // (a chunk's ends are multiples of the tile, or the ends of every span)
            if (part) {
                const uint32_t at = k0 + 4 * half - sp.lo, len = sp.hi - sp.lo;
#pragma unroll
                for (int e = 0; e < 16; ++e) s[e] = at + acc_row(e, 0) < len ? s[e] : kNegInf;
            }
            float mx = s[0];
#pragma unroll
            for (int e = 1; e < 16; ++e) mx = fmaxf(mx, s[e]);
            mx = halves_max(mx) * sc.mul;
            if (__any(mx > m + kRaise)) {
                // (each query by itself: its result does not depend on its neighbours)
                const float mn = mx > m + kRaise ? mx : m;
                const float al = __builtin_amdgcn_exp2f(m - (mn == kNegInf ? 0.f : mn));
                l *= al;
#pragma unroll
                for (int d = 0; d < ND; ++d)
#pragma unroll
                    for (int e = 0; e < 16; ++e) o[d][e] *= al;
                m = mn;
            }
            const float ms = m == kNegInf ? 0.f : m;
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                s[e] = __builtin_amdgcn_exp2f(fmaf(s[e], sc.mul, -ms));
                l += s[e];
            }
            const Frag<T> p0 = pack8<T>(s, 0), p1 = pack8<T>(s, 1);
#pragma unroll
            for (int d = 0; d < ND; ++d) {
                o[d] = mma<T>(col_frag<T, DP>(vt, 0, d * 32, lane), p0, o[d]);
                o[d] = mma<T>(col_frag<T, DP>(vt, 1, d * 32, lane), p1, o[d]);
            }
        }
        if (__any(dropped)) {
            for (int k0 = kbeg; k0 < ghi; k0 += NW * KB) {
                if (alo <= k0 && k0 + KB <= ahi) continue;
                for (int key = max(k0, glo); key < min(k0 + KB, ghi); ++key) {
                    if (key < sp.lo || key >= sp.hi) continue;
                    const R *p = vp + (int64_t)key * a.vs[1];
#pragma unroll
                    for (int d = 0; d < ND; ++d)
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const int x = d * 32 + acc_row(e, half);
                            const float v = x < a.D ? T::widen(p[x]) : 0.f;
                            if (!(fabsf(v) < __builtin_huge_valf())) o[d][e] += v;
                        }
                }
            }
        }
    }
    l = halves_sum(l);

    // join the four waves
    __syncthreads();
    float *const jo = (float *)smem;                       // [NW][32][DP + pad]
    constexpr int JW = DP + kSplitPad;
    if (half == 0) {
        ml[(wave * 32 + col) * 2] = m;
        ml[(wave * 32 + col) * 2 + 1] = l;
    }
#pragma unroll
    for (int d = 0; d < ND; ++d)
#pragma unroll
        for (int e = 0; e < 16; e += 4)
            *(f32x4 *)(jo + (wave * 32 + col) * JW + d * 32 + acc_row(e, half)) =
                f32x4{o[d][e], o[d][e + 1], o[d][e + 2], o[d][e + 3]};
    __syncthreads();
    const int64_t row0 = ((int64_t)b * a.Hk + hk) * rows + rb * 32;
    const int64_t all = (int64_t)a.B * a.Hk * rows;
    for (int x = tid; x < 32 * DP; x += 64 * NW) {
        const int rr = x / DP, d = x - rr * DP;
        if (rb * 32 + rr >= rows) break;
        float mt = kNegInf;
#pragma unroll
        for (int w = 0; w < NW; ++w) mt = fmaxf(mt, ml[(w * 32 + rr) * 2]);
        const float ms = mt == kNegInf ? 0.f : mt;
        float lt = 0.f, ot = 0.f;
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            const float f = __builtin_amdgcn_exp2f(ml[(w * 32 + rr) * 2] - ms);
            lt = fmaf(f, ml[(w * 32 + rr) * 2 + 1], lt);
            ot = fmaf(f, jo[(w * 32 + rr) * JW + d], ot);
        }
        if (a.nsplit > 1) {
            const int64_t at = sp_no * all + row0 + rr;
            if (d < a.D) a.part_o[at * a.D + d] = ot;
            if (d == 0) *(float2 *)(a.part_ml + 2 * at) = make_float2(mt, lt);
        } else {
            const int tt = (rb * 32 + rr) / a.G, hh = hk * a.G + (rb * 32 + rr) % a.G;
            if (d < a.D)
                ((R *)a.out)[(((int64_t)b * a.Tq + tt) * a.Hq + hh) * a.D + d] =
                    T::narrow(lt == 0.f ? 0.f : ot / lt);
            if (d == 0)
                a.lse[((int64_t)b * a.Hq + hh) * a.Tq + tt] =
                    lt == 0.f ? kNegInf : (mt + log2f(lt)) * kLn2;
        }
    }
}

// Joins the chunks: one wave per row, its lanes over the channels.
template <typename T>
__global__ __launch_bounds__(256) void attn_join_kernel(AttnArgs a)
{
    using R = typename T::raw;
    const int lane = threadIdx.x & 63, rows = a.Tq * a.G;
    const int64_t all = (int64_t)a.B * a.Hk * rows;
    const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (row >= all) return;
    float mt = kNegInf;
    for (int s = lane; s < a.nsplit; s += 64) mt = fmaxf(mt, a.part_ml[2 * (s * all + row)]);
#pragma unroll
    for (int x = 32; x; x >>= 1) mt = fmaxf(mt, __shfl_xor(mt, x));
    const float ms = mt == kNegInf ? 0.f : mt;
    float lt = 0.f, o[kAttnMaxD / 64] = {0.f, 0.f};
#pragma unroll 4
    for (int s = 0; s < a.nsplit; ++s) {
        const float2 v = *(const float2 *)(a.part_ml + 2 * (s * all + row));
        const float f = __builtin_amdgcn_exp2f(v.x - ms);
        lt = fmaf(f, v.y, lt);
#pragma unroll
        for (int x = 0; x < kAttnMaxD / 64; ++x)
            if (lane + 64 * x < a.D)
                o[x] = fmaf(f, a.part_o[(s * all + row) * a.D + lane + 64 * x], o[x]);
    }
    const int64_t bh = row / rows;
    const int r = (int)(row - bh * rows), t = r / a.G;
    const int64_t b = bh / a.Hk;
    const int h = (int)(bh - b * a.Hk) * a.G + (r - t * a.G);
    const float inv = lt == 0.f ? 0.f : 1.f / lt;
#pragma unroll
    for (int x = 0; x < kAttnMaxD / 64; ++x)
        if (lane + 64 * x < a.D)
            ((R *)a.out)[((b * a.Tq + t) * a.Hq + h) * a.D + lane + 64 * x] =
                T::narrow(o[x] * inv);
    if (lane == 0)
        a.lse[(b * a.Hq + h) * a.Tq + t] = lt == 0.f ? kNegInf : (mt + log2f(lt)) * kLn2;
}

template <typename T, int DP>
void run(const AttnArgs &a, hipStream_t s)
{
    const int64_t grid = (int64_t)a.nrb * a.Hk * a.B * a.nsplit;
    launch_kernel((attn_split_kernel<T, DP>), dim3((uint32_t)grid), dim3(64 * kSplitWaves),
                  (split_lds<T, DP>()), s, a);
}

}  // namespace

// The split form where the other one would leave most of the card idle.
bool attn_split_wanted(const AttnArgs &a)
{
    const int64_t blocks = (int64_t)a.B * a.Hq * ((a.Tq + kAttnRows - 1) / kAttnRows);
    return (int64_t)a.Tq * a.G <= 32 || (blocks < device_cus() && a.Tk >= 1024 && a.Tq < 256);
}

size_t plan_attn_split(AttnArgs *a)
{
    const int64_t rows = (int64_t)a->Tq * a->G;
    a->nrb = (int32_t)((rows + 31) / 32);
    const int64_t base = (int64_t)a->nrb * a->Hk * a->B, want = 8 * device_cus();
    const int64_t unit = kSplitWaves * kSplitKeys;         // one tile for each wave
    const int64_t most = a->Tk > 0 ? (a->Tk + unit - 1) / unit : 1;
    int64_t n = (want + base - 1) / base;
    n = n > most ? most : n;
    const int64_t chunk = ((most + n - 1) / n) * unit;
    a->chunk = (int32_t)chunk;
    a->nsplit = a->Tk > 0 ? (int32_t)((a->Tk + chunk - 1) / chunk) : 1;
    if (a->nsplit == 1) return 0;
    return (size_t)a->nsplit * a->B * a->Hk * rows * (a->D + 2) * sizeof(float);
}

void place_attn_split(AttnArgs *a, void *workspace)
{
    a->part_ml = (float *)workspace;
    a->part_o = a->part_ml + (int64_t)a->nsplit * a->B * a->Hk * a->Tq * a->G * 2;
}

template <typename T>
hipError_t launch_attn_split(const AttnArgs &a, hipStream_t s)
{
    if (a.D <= 64) run<T, 64>(a, s);
    else run<T, 128>(a, s);
    const int64_t all = (int64_t)a.B * a.Hk * a.Tq * a.G;
    if (a.nsplit > 1)
        launch_kernel((attn_join_kernel<T>), dim3((uint32_t)((all + 3) / 4)), dim3(256), 0, s, a);
    return hipGetLastError();
}

template hipError_t launch_attn_split<F32>(const AttnArgs &, hipStream_t);
template hipError_t launch_attn_split<F16>(const AttnArgs &, hipStream_t);
template hipError_t launch_attn_split<BF16>(const AttnArgs &, hipStream_t);

}  // namespace mp3d
