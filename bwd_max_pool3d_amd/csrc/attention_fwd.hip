// attention_fwd.hip -- attention forward for many queries.
//
//   out_i = sum_j p_ij v_j,  p_ij = exp(s_ij - lse_i),  lse_i = log sum_j exp(s_ij)
// over the keys j that query i sees, in one pass with a running maximum and
// sum per query.  A workgroup takes 32 queries of one head for each of its
// waves, and walks the keys that any of its queries sees in tiles of 64, read
// once into LDS for all waves (attention.hpp has the layout).  The scores are formed as (keys x queries), so a query's scores
// lie in two lanes: its maximum and sum are sums over registers and one
// exchange between the wave's halves, and the weights go into the second
// product where they are.
//
// The running maximum is only raised when a score exceeds it by 2^8 (the
// weights then stay under 2^8, and the sums' relative error is the same);
// raising it costs a pass over the accumulators.  Weights are rounded to the
// storage type for the second product (its matrix instruction takes no
// other), their sum is not: the rounding errors are independent and as
// small as that of the output itself.
//
// Bound: the matrix unit and, with a cap, a bias or 64 channels, the vector
// unit, which a wave's two kinds of work take in turn: two waves on a SIMD
// overlap them in part.  Four waves share a tile so that LDS and L2 are read
// once for 128 queries; two waves a workgroup (64 queries) measured 293 us
// where four took 168, three waves on a SIMD spill.
//
// Measured: 10935 causal bfloat16 tokens, 16 heads of 128 on 4, cap 50:
// 605 to 675 us by the card's clock (730 to 810 TFLOP/s of visible pairs; 70 %
// of the cycles the vector unit is busy, 39 % the matrix unit).  8192 packed
// tokens in 9 documents, 16 heads of 64, bias on 3 axes: 125 us (of which
// the bias was 40 on the vector unit alone).  2 x 2047 float16, prefix, 16
// heads of 128 on 2: 64 us.
#include "attention.hpp"

namespace mp3d {

namespace {

constexpr int kFwdWaves = kAttnRows / 32;
constexpr int kFwdKeys = 64;               // one for each lane
constexpr int kFwdPos = kFwdKeys + 33;     // places of a tile's positions on one axis
constexpr float kRaise = 8.f;

// float32 tiles of 128 channels take twice the LDS and the registers: one
// workgroup on a CU
template <typename T, int DP>
constexpr int fwd_occupancy()
{
    return sizeof(typename T::raw) * DP > 256 ? 1 : 2;
}

template <typename T, int DP, int DU, bool GEN>
__global__ __launch_bounds__(64 * kFwdWaves, (fwd_occupancy<T, DP>())) void attn_fwd_kernel(AttnArgs a)
{
    using R = typename T::raw;
    const int axes = GEN ? a.axes : 0;
    constexpr int NW = kFwdWaves, NT = 64 * NW, KB = kFwdKeys, NC = DU / 16, ND = DU / 32;
    constexpr bool ALL = DU == DP;         // whole tiles with all their channels
    extern __shared__ __align__(16) unsigned char smem[];
    R *const kt = (R *)smem;                               // [2][KB * DP]
    R *const vt = kt + 2 * KB * DP;                        // [2][KB * DP]
    // [2][3][KB keys' positions, and ones 32 apart]
    u32x2 *const pk = (u32x2 *)(vt + 2 * KB * DP);
    int *const flag = (int *)(pk + 2 * 3 * kFwdPos);       // an infinity or a NaN was dropped
    int *const ends = flag + 1;                            // [4][NW]
    int *const fars = ends + 4 * NW;                       // a position is far

    const int nq = (a.Tq + 32 * NW - 1) / (32 * NW);
    const Block blk = block_of(blockIdx.x, a.B * a.Hq, nq);
    const int bh = blk.head;
    const int b = bh / a.Hq, h = bh - b * a.Hq, hk = h / a.G;
    // (without documents the last queries see the most, if causal)
    const int qt = a.order_q ? uniform(a.order_q[(int64_t)b * nq + blk.no]) : nq - 1 - blk.no;
    const int tid = threadIdx.x, wave = uniform(tid >> 6), lane = tid & 63, col = lane & 31, half = lane >> 5;
    const int q0 = qt * 32 * NW, i = q0 + wave * 32 + col;
    const int ic = min(i, a.Tq - 1);
    const Span sp = row_span(a, b, ic);

    // the wave's and the workgroup's keys: union, and the part all rows see
    int wlo = sp.hi > sp.lo ? sp.lo : 0x7fffffff, whi = sp.hi, alo = sp.lo, ahi = sp.hi;
#pragma unroll
    for (int m = 16; m; m >>= 1) {
        wlo = min(wlo, __shfl_xor(wlo, m));
        whi = max(whi, __shfl_xor(whi, m));
        alo = max(alo, __shfl_xor(alo, m));
        ahi = min(ahi, __shfl_xor(ahi, m));
    }
    wlo = __builtin_amdgcn_readfirstlane(wlo);
    whi = __builtin_amdgcn_readfirstlane(whi);
    alo = __builtin_amdgcn_readfirstlane(alo);
    ahi = __builtin_amdgcn_readfirstlane(ahi);
    if ((tid & 63) == 0) {
        ends[wave] = wlo;
        ends[NW + wave] = whi;
        ends[2 * NW + wave] = alo;
        ends[3 * NW + wave] = ahi;
    }
    if (tid == 0) *flag = *fars = 0;
    if (axes > 0 && tid < 2 * 3 * 2)
        pk[(tid >> 1) * kFwdPos + KB + (tid & 1) * 32] = u32x2{kOnes, kOnes};
    __syncthreads();
    int glo = ends[0], ghi = ends[NW], galo = ends[2 * NW], gahi = ends[3 * NW];
#pragma unroll
    for (int w = 1; w < NW; ++w) {
        glo = min(glo, ends[w]);
        ghi = max(ghi, ends[NW + w]);
        galo = max(galo, ends[2 * NW + w]);
        gahi = min(gahi, ends[3 * NW + w]);
    }

    glo = uniform(glo);
    ghi = uniform(ghi);
    galo = uniform(galo);
    gahi = uniform(gahi);

    const R *kp = (const R *)a.k + b * a.ks[0] + hk * a.ks[2];
    const R *vp = (const R *)a.v + b * a.vs[0] + hk * a.vs[2];
    const R *qp = (const R *)a.q + b * a.qs[0] + h * a.qs[2] + (int64_t)ic * a.qs[1];
    Frag<T> qf[NC];
#pragma unroll
    for (int c = 0; c < NC; ++c) qf[c] = load8<T>(qp, c * 16 + half * 8, a.D, a.vec);

    const Scores sc = scores(a);
    u32x2 pq[3];
    float sl[3];
    bool far = false;                      // a query's or a key's position is
#pragma unroll
    for (int x = 0; x < 3; ++x) {
        if (x >= axes) break;
        const u32x2 p = position_parts(a.pos_q[((int64_t)x * a.B + b) * a.Tq + ic]);
        far |= is_far_position(p);
        pq[x] = position_cols(p, half);
        sl[x] = a.slopes[h * axes + x] * sc.slope;
        arrived(sl[x]);
    }

    arrived(qf);
    f32x16 o[ND];
#pragma unroll
    for (int d = 0; d < ND; ++d) o[d] = f32x16(0.f);
    float m = kNegInf, l = 0.f;            // l: this half's sum

    const int kbeg = ghi > 0 ? glo / KB * KB : 0, kend = ghi;
    TileDirect<T, DP, KB, NT> kd, vd;
    kd.init(tid, a.ks[1], a.D);
    vd.init(tid, a.vs[1], a.D);
    const bool usable = kd.usable(a.vec, a.ks[1], a.D) && vd.usable(a.vec, a.vs[1], a.D);
    if (a.D < DP) {                        // channels that no direct load writes
        for (int x = tid; x < 4 * KB * DP * (int)sizeof(R) / 16; x += NT)
            ((u32x4 *)kt)[x] = u32x4{0u, 0u, 0u, 0u};
        __syncthreads();
    }
    // Positions go by way of a register, one axis a wave.  (It is not touched
    // before place: that would wait for it)
    const int32_t *pos = a.pos_k + ((int64_t)min(wave, 2) * a.B + b) * a.Tk;
    int32_t pr = 0;
    const uint32_t lds = lds_address(smem) + wave * 1024;
    const bool whole = usable && (!ALL || a.D == DP);
    const R *fk = kp + (int64_t)kbeg * a.ks[1], *fv = vp + (int64_t)kbeg * a.vs[1];
    auto fetch = [&](int k0, int buf) {
        const uint32_t at = lds + buf * KB * DP * (int)sizeof(R);
        constexpr uint32_t v0 = 2 * KB * DP * sizeof(R);
        if (whole && glo <= k0 && k0 + KB <= ghi) {
            kd.template load<ALL>(fk, at);
            vd.template load<ALL>(fv, at + v0);
        } else if (usable) {
            kd.load_edge(kp, a.ks[1], k0, glo, ghi, at);
            vd.load_edge(vp, a.vs[1], k0, glo, ghi, at + v0);
        }
        fk += KB * a.ks[1];
        fv += KB * a.vs[1];
        if (wave < axes) pr = pos[min(k0 + lane, a.Tk - 1)];
    };
    auto place = [&](int k0, int buf) {
        const bool edge = k0 < glo || k0 + KB > ghi;
        const bool drop = !(galo <= k0 && k0 + KB <= gahi);
        R *const ks = kt + buf * KB * DP, *const vs = vt + buf * KB * DP;
        wait_loads<0>(false);
        if (!usable) {
            const int t = opaque(threadIdx.x);
            TileRegs<T, DP, KB, NT> r;
            r.load(vp, a.vs[1], k0, glo, ghi, a.D, a.vec, t);
            if (drop && r.drop()) *flag = 1;
            r.store(vs, t);
            r.load(kp, a.ks[1], k0, glo, ghi, a.D, a.vec, t);
            r.store(ks, t);
            wait_all();
        } else if (edge || drop) {
            if (vd.scrub(vs, k0, glo, ghi, drop, nullptr, 0)) *flag = 1;
            if (edge) kd.scrub(ks, k0, glo, ghi, false, nullptr, 0);
        }
        if (wave < axes)
            pk[(buf * 3 + wave) * kFwdPos + lane] = position_parts(pr);
        hand_over();
    };
    int signed_axes = axes;                // negative with a far position (add_bias)
    if (kbeg < kend) {
        fetch(kbeg, 0);
        if (axes > 0) {                    // (while the first tile is on its way)
            const int32_t *p = a.pos_k + (int64_t)b * a.Tk;
            const int64_t y = axes > 1 ? (int64_t)a.B * a.Tk : 0, z = axes > 2 ? 2 * y : 0;
#pragma unroll 4
            for (int k = glo + tid; k < ghi; k += NT) {
                far |= is_far_position(p[k]);
                far |= is_far_position(p[k + y]);
                far |= is_far_position(p[k + z]);
            }
            if (far) *fars = 1;
        }
        place(kbeg, 0);
        if (axes > 0 && uniform(*fars)) signed_axes = -axes;
    }
int n = 0;
    for (int k0 = kbeg; k0 < kend; k0 += KB, ++n) {
        const int buf = n & 1;
        const bool more = k0 + KB < kend;
        if (more) fetch(k0 + KB, buf ^ 1);
        // (a wave none of whose queries sees the tile goes along: it would wait
        // for the others anyway)
        const R *kb = kt + buf * KB * DP, *vb = vt + buf * KB * DP;
        Frag<T> kf[NC][2], vf[ND][4], pf[4];
        f32x16 s[2] = {f32x16(0.f), f32x16(0.f)};
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int u = 0; u < 2; ++u)
                kf[c][u] = row_frag<T, DP>(kb, u * 32 + col, c * 16 + half * 8);
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int u = 0; u < 2; ++u) s[u] = mma<T>(kf[c][u], qf[c], s[u]);
#pragma unroll
        for (int d = 0; d < ND / 2; ++d)
#pragma unroll
            for (int c = 0; c < 4; ++c) vf[d][c] = col_frag<T, DP>(vb, c, d * 32, lane);
        reads_ahead<T, NC>();
        products_and_reads<T, NC, 1>();
        products_and_reads<T, NC, 2>();
        issued<T>();
        const bool part = !(alo <= k0 && k0 + KB <= ahi);
        if (GEN) {
            multiply_scores(s[0], sc);
            multiply_scores(s[1], sc);
        }
        if (GEN && a.cap > 0.f) {
#pragma unroll
            for (int u = 0; u < 2; ++u) cap_scores<T>(s[u], sc, part);
        }
        if (GEN && signed_axes != 0) {
            const u32x2 *const rows = pk + buf * 3 * kFwdPos + (half ? KB : col);
#pragma unroll
            for (int u = 0; u < 2; ++u)
                add_bias(s[u], rows + u * 32, kFwdPos, signed_axes, pq, sl);
        }
        if (part) {
            const uint32_t at = k0 + 4 * half - sp.lo, len = sp.hi - sp.lo;
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    s[u][r] = at + (u * 32 + acc_row(r, 0)) < len ? s[u][r] : kNegInf;
        }
        float mx = s[0][0];
#pragma unroll
        for (int r = 1; r < 16; ++r) mx = fmaxf(mx, s[0][r]);
#pragma unroll
        for (int r = 0; r < 16; ++r) mx = fmaxf(mx, s[1][r]);
        mx = halves_max(mx) * sc.mul;
        if (__any(mx > m + kRaise)) {
            // (each query by itself: its sums do not depend on its neighbours')
            const float mn = mx > m + kRaise ? mx : m;
            const float al = __builtin_amdgcn_exp2f(m - (mn == kNegInf ? 0.f : mn));
            l *= al;
#pragma unroll
            for (int d = 0; d < ND; ++d)
#pragma unroll
                for (int r = 0; r < 16; ++r) o[d][r] *= al;
            m = mn;
        }
        const float ms = m == kNegInf ? 0.f : m;
        auto weights = [&](int u) {
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                s[u][r] = __builtin_amdgcn_exp2f(fmaf(s[u][r], sc.mul, -ms));
                l += s[u][r];
            }
            pf[2 * u] = pack8<T>(s[u], 0);
            pf[2 * u + 1] = pack8<T>(s[u], 1);
        };
        weights(0);
        weights(1);
#pragma unroll
        for (int d = ND / 2; d < ND; ++d)
#pragma unroll
            for (int c = 0; c < 4; ++c) vf[d][c] = col_frag<T, DP>(vb, c, d * 32, lane);
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int d = 0; d < ND / 2; ++d) o[d] = mma<T>(vf[d][c], pf[c], o[d]);
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int d = ND / 2; d < ND; ++d) o[d] = mma<T>(vf[d][c], pf[c], o[d]);
        products_and_reads<T, 2 * ND, 2>();
        products_and_reads<T, 2 * ND, 0>();
        issued<T>();
        if (more) place(k0 + KB, buf ^ 1);
    }

    if (*flag) {                           // (set before the last barrier)
        for (int key = kbeg; key < kend; ++key) {
            const int k0 = key / KB * KB;
            if ((galo <= k0 && k0 + KB <= gahi) || key < sp.lo || key >= sp.hi) continue;
            const R *p = vp + (int64_t)key * a.vs[1];
#pragma unroll
            for (int d = 0; d < ND; ++d)
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    const int e = d * 32 + acc_row(r, half);
                    const float v = e < a.D ? T::widen(p[e]) : 0.f;
                    if (!(fabsf(v) < __builtin_huge_valf())) o[d][r] += v;
                }
        }
    }

    if (i >= a.Tq) return;
    l = halves_sum(l);
    const float inv = l == 0.f ? 0.f : 1.f / l;
    if (half == 0)
        a.lse[((int64_t)b * a.Hq + h) * a.Tq + i] = l == 0.f ? kNegInf : (m + log2f(l)) * kLn2;
    store_cols<T, ND>((R *)a.out + (((int64_t)b * a.Tq + i) * a.Hq + h) * a.D, o, inv, a.D, half);
}

template <typename T, int DP, int DU, bool GEN>
hipError_t run(const AttnArgs &a, hipStream_t s)
{
    constexpr int NW = kFwdWaves;
    constexpr uint32_t lds = 4 * kFwdKeys * DP * sizeof(typename T::raw) +
                             2 * 3 * kFwdPos * sizeof(u32x2) + (2 + 4 * NW) * sizeof(int);
    const int64_t nq = (a.Tq + 32 * NW - 1) / (32 * NW);
    launch_attn_order(a, false, s);
    // (none that reads the order follows a failed launch)
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    launch_kernel((attn_fwd_kernel<T, DP, DU, GEN>), dim3((uint32_t)(nq * a.B * a.Hq)),
                  dim3(64 * NW), lds, s, a);
    return hipGetLastError();
}

template <typename T, bool GEN>
hipError_t run_width(const AttnArgs &a, hipStream_t s)
{
    if (a.D <= 32) return run<T, 64, 32, GEN>(a, s);
    if (a.D <= 64) return run<T, 64, 64, GEN>(a, s);
    if (a.D <= 96) return run<T, 128, 96, GEN>(a, s);
    return run<T, 128, 128, GEN>(a, s);
}

}  // namespace

template <typename T>
hipError_t launch_attn_forward(const AttnArgs &a, hipStream_t s)
{
    return attn_general(a) ? run_width<T, true>(a, s) : run_width<T, false>(a, s);
}

template hipError_t launch_attn_forward<F32>(const AttnArgs &, hipStream_t);
template hipError_t launch_attn_forward<F16>(const AttnArgs &, hipStream_t);
template hipError_t launch_attn_forward<BF16>(const AttnArgs &, hipStream_t);

}  // namespace mp3d
