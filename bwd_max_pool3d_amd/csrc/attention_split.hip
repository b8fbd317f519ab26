// attention_split.hip -- attention forward for few queries over many keys
// (single new tokens, short chunks, few heads), split over the keys and joined.
//
// Bound: HBM (the keys and values are read once; 4 G flop for each 2 bytes
// of them).  All query heads that share a key head, and all new tokens, are
// rows of one block of up to 32, so a key is read once for all of them.  A
// workgroup takes one block of rows and one chunk of keys; its four waves
// take tiles of 32 keys in turn, each through a part of LDS of its own, so
// no wave waits for another until the end.  A tile's keys, and its values,
// go to registers as soon as they are in LDS, and the next tile's take their
// place there: loads are in flight all the time, with one tile of LDS a
// wave, and two workgroups fit on a CU.  Every wave keeps its own running
// maximum and sum; the four are joined in LDS, the chunks by a second
// kernel.  Chunks have a fixed length whatever the sequence's: those past a
// short sequence's end return at once, so long and short caches balance.
//
// Measured: 16 bfloat16 caches of 9728 to 32768, 32 heads of 128 on 8, one
// new token each: 250 us and 5 for the join, 5.5 TB/s (a copy reaches 5.0),
// where tiles by way of registers took 310 and the kernel for many queries
// takes 1048.  777 float16 keys, 16 heads on 4: 10 and 3.5 us (35).
#include "attention.hpp"

namespace mp3d {

namespace {

constexpr int kSplitWaves = 4;
constexpr int kSplitKeys = 32;             // keys of a wave's tile
constexpr int kSplitPad = 4;               // floats between the rows of the join
constexpr int kJoinGroups = 8;
constexpr float kRaise = 8.f;

// floats between a chunk's rows, for loads of 4
__host__ __device__ inline int split_stride(int D) { return (D + 3) & ~3; }

template <typename T, int DP>
constexpr uint32_t split_tiles()
{
    const uint32_t tiles = kSplitWaves * 2 * kSplitKeys * DP * sizeof(typename T::raw);
    const uint32_t join = kSplitWaves * 32 * (DP + kSplitPad) * sizeof(float);
    return tiles > join ? tiles : join;
}
template <typename T, int DP>
constexpr uint32_t split_lds()
{
    return split_tiles<T, DP>() + kSplitWaves * (2 * 3 * kSplitKeys + 64) * sizeof(float);
}

template <typename T, int DP, int DU, bool GEN>
__global__ __launch_bounds__(64 * kSplitWaves, (sizeof(typename T::raw) * DP > 256 ? 1 : 2))
void attn_split_kernel(AttnArgs a)
{
    using R = typename T::raw;
    constexpr int KB = kSplitKeys, NC = DU / 16, ND = DU / 32, NW = kSplitWaves;
    constexpr bool ALL = DU == DP;         // whole tiles with all their channels
    extern __shared__ __align__(16) unsigned char smem[];
    const int axes = GEN ? a.axes : 0;
    const int tid = threadIdx.x, wave = uniform(tid >> 6), lane = tid & 63, col = lane & 31,
              half = lane >> 5;
    R *const kt = (R *)smem + wave * 2 * KB * DP, *const vt = kt + KB * DP;
    int *const pk = (int *)(smem + split_tiles<T, DP>()) + wave * 2 * 3 * KB;   // [2][3][KB]
    float *const ml = (float *)(smem + split_tiles<T, DP>()) + NW * 2 * 3 * KB;  // [NW][32][2]

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
        TileDirect<T, DP, KB, 64> kd, vd;
        kd.init(lane, a.ks[1], a.D);
        vd.init(lane, a.vs[1], a.D);
        const bool usable = kd.usable(a.vec, a.ks[1], a.D) && vd.usable(a.vec, a.vs[1], a.D);
        const bool whole = usable && (!ALL || a.D == DP);
        if (a.D < DP) {                        // channels that no direct load writes
            for (int x = lane; x < 2 * KB * DP * (int)sizeof(R) / 16; x += 64)
                ((u32x4 *)kt)[x] = u32x4{0u, 0u, 0u, 0u};
            reads_done();                      // (these writes are)
        }
        const uint32_t lds_k = lds_address(kt), lds_v = lds_address(vt), lds_p = lds_address(pk);
        auto fetch = [&](const TileDirect<T, DP, KB, 64> &d, const R *p, int64_t stride, int k0,
                         uint32_t lds) {
            if (whole && glo <= k0 && k0 + KB <= ghi) d.template load<ALL>(p + k0 * stride, lds);
            else if (usable) d.load_edge(p, stride, k0, glo, ghi, lds);
        };
        auto place = [&](const R *p, int64_t stride, int k0, R *tile) {
            TileRegs<T, DP, KB, 64> r;
            r.load(p, stride, k0, glo, ghi, a.D, a.vec, lane);
            r.store(tile, lane);
            wait_all();
        };
        // three axes or none, so that what is in flight can be counted
        auto fetch_pos = [&](int k0, int buf) {
            if (axes > 0 && lane < KB)
#pragma unroll
                for (int x = 0; x < 3; ++x)
                    direct4(a.pos_k + ((int64_t)min(x, axes - 1) * a.B + b) * a.Tk + k0,
                            (uint32_t)min(lane, a.Tk - 1 - k0) * 4,
                            lds_p + (buf * 3 + x) * KB * 4);
        };
        const int kbeg = glo / KB * KB + wave * KB;
        if (kbeg < ghi) {
            fetch_pos(kbeg, 0);
            fetch(kd, kp, a.ks[1], kbeg, lds_k);
            fetch(vd, vp, a.vs[1], kbeg, lds_v);
        }

        const R *qp = (const R *)a.q + b * a.qs[0] + h * a.qs[2] + (int64_t)t * a.qs[1];
        Frag<T> qf[NC];
#pragma unroll
        for (int c = 0; c < NC; ++c) qf[c] = load8<T>(qp, c * 16 + half * 8, a.D, a.vec);
        const Scores sc = scores(a);
        int pq[3];
        float sl[3];
#pragma unroll
        for (int x = 0; x < 3; ++x) {
            if (x >= axes) break;
            pq[x] = a.pos_q[((int64_t)x * a.B + b) * a.Tq + t];
            sl[x] = a.slopes[h * axes + x] * sc.slope;
            arrived(pq[x]);
            arrived(sl[x]);
        }
        arrived(qf);
        constexpr int kTile = TileDirect<T, DP, KB, 64>::LOADS;
        int buf = 0;
        for (int k0 = kbeg; k0 < ghi; k0 += NW * KB, buf ^= 1) {
            const bool part = !(alo <= k0 && k0 + KB <= ahi), more = k0 + NW * KB < ghi;
            // keys: in flight after them are this tile's values.  (A wave's
            // LDS operations keep their order: no barrier)
            wait_loads<kTile>(usable);
            if (!usable) place(kp, a.ks[1], k0, kt);
            Frag<T> kf[NC], vf[ND][2];
#pragma unroll
            for (int c = 0; c < NC; ++c) kf[c] = row_frag<T, DP>(kt, col, c * 16 + half * 8);
            reads_done();
            if (more) {
                fetch_pos(k0 + NW * KB, buf ^ 1);
                fetch(kd, kp, a.ks[1], k0 + NW * KB, lds_k);
            }
            f32x16 s = f32x16(0.f);
#pragma unroll
            for (int c = 0; c < NC; ++c) s = mma<T>(kf[c], qf[c], s);
            // values: in flight after them are the next tile's keys
            if (axes > 0) wait_loads<kTile + 3>(more && usable);
            else wait_loads<kTile>(more && usable);
            if (!usable) place(vp, a.vs[1], k0, vt);
            if (part) {
                dropped |= vd.scrub(vt, k0, glo, ghi, true, nullptr, 0);
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            }
#pragma unroll
            for (int d = 0; d < ND; ++d)
#pragma unroll
                for (int c = 0; c < 2; ++c) vf[d][c] = col_frag<T, DP>(vt, c, d * 32, lane);
            reads_done();
            if (more) fetch(vd, vp, a.vs[1], k0 + NW * KB, lds_v);

            if (GEN) multiply_scores(s, sc);
            if (GEN && a.cap > 0.f) cap_scores<T>(s, sc, part);
#pragma unroll
            for (int x = 0; x < 3; ++x) {
                if (x >= axes) break;
                const int *p = pk + (buf * 3 + x) * KB + 4 * half;
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const int k = p[acc_row(e, 0)];        // (up to 2^32 apart)
                    s[e] = fmaf(-sl[x], (float)((uint32_t)max(k, pq[x]) - (uint32_t)min(k, pq[x])),
                                s[e]);
                }
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
                // (each query by itself: its sums do not depend on its neighbours')
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
                o[d] = mma<T>(vf[d][0], p0, o[d]);
                o[d] = mma<T>(vf[d][1], p1, o[d]);
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
            if (d < split_stride(a.D)) a.part_o[at * split_stride(a.D) + d] = ot;
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

// Joins the chunks: a workgroup per row, 8 groups of 32 lanes with 4 channels
// a lane.  The groups take the chunks in turn, each with a running maximum of
// its own, and are joined in LDS in a fixed order.
template <typename T>
__global__ __launch_bounds__(32 * kJoinGroups) void attn_join_kernel(AttnArgs a)
{
    using R = typename T::raw;
    constexpr int NG = kJoinGroups;
    __shared__ __align__(16) float jo[NG][kAttnMaxD];
    __shared__ float jm[NG], jl[NG];
    const int tid = threadIdx.x, g = tid >> 5, d0 = (tid & 31) * 4, rows = a.Tq * a.G;
    const int64_t all = (int64_t)a.B * a.Hk * rows, row = blockIdx.x;
    const int ds = split_stride(a.D);
    float m = kNegInf, l = 0.f;
    f32x4 o = f32x4(0.f);
#pragma unroll 4
    for (int s = g; s < a.nsplit; s += NG) {
        const int64_t at = s * all + row;
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
    const int64_t bh = row / rows;
    const int r = (int)(row - bh * rows), t = r / a.G;
    const int64_t b = bh / a.Hk;
    const int h = (int)(bh - b * a.Hk) * a.G + (r - t * a.G);
    if (tid < a.D)
        ((R *)a.out)[((b * a.Tq + t) * a.Hq + h) * a.D + tid] =
            T::narrow(lt == 0.f ? 0.f : ot / lt);
    if (tid == 0)
        a.lse[(b * a.Hq + h) * a.Tq + t] = lt == 0.f ? kNegInf : (mt + log2f(lt)) * kLn2;
}

template <typename T, int DP, int DU>
void run(const AttnArgs &a, hipStream_t s)
{
    const int64_t grid = (int64_t)a.nrb * a.Hk * a.B * a.nsplit;
    if (attn_general(a))
        launch_kernel((attn_split_kernel<T, DP, DU, true>), dim3((uint32_t)grid),
                      dim3(64 * kSplitWaves), (split_lds<T, DP>()), s, a);
    else
        launch_kernel((attn_split_kernel<T, DP, DU, false>), dim3((uint32_t)grid),
                      dim3(64 * kSplitWaves), (split_lds<T, DP>()), s, a);
}

}  // namespace

// The split form for rows that fit one block (the other kernel has 128 rows
// a workgroup; figures above), for short chunks where the other one would
// leave most of the card idle (64 queries of 8 heads, 8192 keys: 36 us, 160
// by the other; 200 of 8 on 2: 57 and 163; 250 over 1024 keys: 15 and 20), and
// for long ones of few heads.  There the waves do not share their keys, which
// costs 16-bit types more than float32, whose matrix instructions are 16 times
// slower: it pays from 4096 keys and a quarter of the CUs on (4096 tokens, 2
// heads of 128: 68 to 73 us, 84 by the other; 2048, 4 heads: 62 and 45), in
// float32 from 512 (512, 8 heads of 64: 21 and 42; 4096, 2 heads of 128: 202 to
// 256 and 574), and to five eighths of the CUs from 2048 (3 x 3302, 2 heads of
// 128: 311 to 470 and 472; 1024, 16 heads: 184 and 152).
bool attn_split_wanted(const AttnArgs &a, bool f32)
{
    const int64_t blocks = (int64_t)a.B * a.Hq * ((a.Tq + kAttnRows - 1) / kAttnRows);
    const int64_t cus = device_cus();
    if ((int64_t)a.Tq * a.G <= 32) return true;
    if (a.Tk >= 1024 && a.Tq < 256) return blocks < cus;
    if (f32) return a.Tk >= 512 && blocks * 8 <= cus * (a.Tk >= 2048 ? 5 : 2);
    return a.Tk >= 4096 && blocks * 4 <= cus;
}

// Eight workgroups a CU: 4, 12 and 16 measured 2 % more on long caches, 32
// (with tiles by way of registers) 17 %, a chunk's start being about 6 us.
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
    const size_t all = (size_t)a->nsplit * a->B * a->Hk * rows;
    return ((2 * all + 3) / 4 * 4 + all * split_stride(a->D)) * sizeof(float);
}

void place_attn_split(AttnArgs *a, void *workspace)
{
    a->part_ml = (float *)workspace;
    const int64_t all = (int64_t)a->nsplit * a->B * a->Hk * a->Tq * a->G;
    a->part_o = a->part_ml + (2 * all + 3) / 4 * 4;
}

template <typename T>
hipError_t launch_attn_split(const AttnArgs &a, hipStream_t s)
{
    if (a.D <= 32) run<T, 64, 32>(a, s);
    else if (a.D <= 64) run<T, 64, 64>(a, s);
    else if (a.D <= 96) run<T, 128, 96>(a, s);
    else run<T, 128, 128>(a, s);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;         // the join would read what was not written
    const int64_t all = (int64_t)a.B * a.Hk * a.Tq * a.G;
    if (a.nsplit > 1)
        launch_kernel((attn_join_kernel<T>), dim3((uint32_t)all),
                      dim3(32 * kJoinGroups), 0, s, a);
    return hipGetLastError();
}

template hipError_t launch_attn_split<F32>(const AttnArgs &, hipStream_t);
template hipError_t launch_attn_split<F16>(const AttnArgs &, hipStream_t);
template hipError_t launch_attn_split<BF16>(const AttnArgs &, hipStream_t);

}  // namespace mp3d
