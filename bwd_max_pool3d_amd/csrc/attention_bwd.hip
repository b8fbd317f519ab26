// attention_bwd.hip -- attention backward.
//
// With the weights p_ij = exp(s_ij - lse_i) formed again from the forward's
// log-sum-exp, and delta_i = sum_j p_ij (do_i . v_j) = do_i . out_i:
//   dv_j = sum_i p_ij do_i
//   e_ij = p_ij (do_i . v_j - delta_i) (1 - tanh^2(scale q_i . k_j / cap))
//   dq_i = scale sum_j e_ij k_j        dk_j = scale sum_i e_ij q_i
// (the last factor of e only with a cap; the bias has no gradient).
//
// Three launches: the rows' constants (delta, the spans of keys, and their
// unions over 32 queries); dk and dv, a workgroup per 128 keys of one key
// head, walking the queries of the heads that share it; dq, a workgroup per
// 128 queries, walking their keys.  Scores and do . v are
// formed in both (7 products where 5 would do), and in exchange every sum
// is kept by one wave in registers and written once: no atomics, the same
// bits on every run.  Where one pass over a key head's query heads would
// leave the card idle they are dealt to several workgroups, whose binary32
// sums a fourth launch adds in a fixed order.
//
// p and e are rounded to the storage type for the second products, as the
// forward's weights are.  Range: float16 ends at 65504 and has its full bits
// down to 2^-14 only.  Over many keys p and e are below that, and gradients
// scaled against just this take e beyond 65504 while dq and dk are not.  So in
// float16 p is rounded times 2^12, and e over 2^x, taken out where dq, dk and
// dv are stored.  |do . v_j| and |delta| are at most |do|_1 max |v|, so with
//   x = 1 + exponent of |do|_1 max |v| - 15
// no |e| 2^-x reaches 2^15.  dq takes each query's x (in the exponential, at no
// cost); dk is a sum over queries, and takes the largest x of those that the
// workgroup walks (one operation a score).  The first kernel leaves |do|_1
// and its and |v|'s maxima over small groups, and the others join them as they
// start (2 x 2047 tokens, 16 heads of 128 on 2, forward and backward: 352 -> 361
// us; max |v| by a launch of its own 372).
//
// Bound: with 64 channels and a bias the vector unit and the waits between
// its work and the matrix unit's (vector 41 %, matrix 25 % of the cycles busy
// in dk, dv; 43 and 29 % in dq), with 128 the waits.  Measured: 8192 packed
// bfloat16 tokens in 9 documents, 16 heads of 64, bias on 3 axes: constants
// 13 us, dk and dv 208, dq 137.  2 x 2047 float16, causal with a prefix, 16
// heads of 128 on 2: 12, 175 and its parts' sum 15.5, 122.  32 x 245 float32,
// 4 heads of 64, bias on 3 axes: 8, 76, 47.
#include <type_traits>

#include "attention.hpp"

// (lambdas that two branches call are not always inlined otherwise, and
// their values would go through memory)
#define MP3D_INLINE __attribute__((always_inline))

namespace mp3d {

namespace {

constexpr int kBwdWaves = kAttnRows / 32;
constexpr int kStep = 32;                  // keys (dq) or queries (dk, dv) per step
constexpr int kPos = kStep + 2;            // places of a step's positions on one axis (16 bytes)
constexpr int kSmall = 16 * kStep + 3 * 8 * kPos;      // bytes of a step's constants, spans, positions
constexpr float kInf = __builtin_huge_valf();
constexpr int64_t kRowsGrid = (int64_t)1 << 23;        // workgroups of the constants along x

// ------------------------------------------------------------ constants

// delta from the scores, as sum_j p_ij (do_i . v_j), for the 32 queries of
// tile qt where together they see at most kFew keys; false elsewhere.  out is
// rounded to the storage type, and do . out with it; with few keys do . v and
// delta nearly cancel in e, and dq and dk would show it (16 to 100 causal
// tokens: 1.6 to 1.75 times the error of gradients rounded once, against 1.4
// with these sums; with many keys the rounding of e itself is larger).  Each
// wave takes 32 keys.
constexpr int kFew = 32 * 4;

template <typename T>
__device__ __forceinline__ bool few_keys_delta(const AttnArgs &a, int b, int h, int qt,
                                               float (*sums)[32])
{
    using R = typename T::raw;
    const int wave = uniform(threadIdx.x >> 6), lane = threadIdx.x & 63, col = lane & 31,
              half = lane >> 5;
    const int i = min(qt * 32 + col, a.Tq - 1);
    const Span sp = row_span(a, b, i);
    int lo = sp.hi > sp.lo ? sp.lo : 0x7fffffff, hi = sp.hi;
#pragma unroll
    for (int m = 16; m; m >>= 1) {
        lo = min(lo, __shfl_xor(lo, m));
        hi = max(hi, __shfl_xor(hi, m));
    }
    lo = uniform(lo);
    hi = uniform(hi);
    if (lo >= hi || hi - lo > kFew) return false;

    float sum = 0.f;
    const int k0 = lo + 32 * wave;
    if (k0 < hi) {
        const int hk = h / a.G, kc = min(k0 + col, hi - 1);
        const R *q = (const R *)a.q + b * a.qs[0] + h * a.qs[2] + (int64_t)i * a.qs[1];
        const R *g = (const R *)a.dout + b * a.gs[0] + h * a.gs[2] + (int64_t)i * a.gs[1];
        const R *k = (const R *)a.k + b * a.ks[0] + hk * a.ks[2] + (int64_t)kc * a.ks[1];
        const R *v = (const R *)a.v + b * a.vs[0] + hk * a.vs[2] + (int64_t)kc * a.vs[1];
        f32x16 s = f32x16(0.f), dp = f32x16(0.f);
#pragma unroll 1
        for (int c = 0; c < a.D; c += 16) {
            s = mma<T>(load8<T>(k, c + half * 8, a.D, a.vec), load8<T>(q, c + half * 8, a.D, a.vec),
                       s);
            dp = mma<T>(load8<T>(v, c + half * 8, a.D, a.vec),
                        load8<T>(g, c + half * 8, a.D, a.vec), dp);
        }
        const Scores sc = scores(a);
        multiply_scores(s, sc);
        if (a.cap > 0.f) cap_scores<T>(s, sc, true);
        for (int x = 0; x < a.axes; ++x) {
            const int64_t row = (int64_t)x * a.B + b;
            const double pq = a.pos_q[row * a.Tq + i];
            const int32_t *pk = a.pos_k + row * a.Tk;
            const float sl = a.slopes[h * a.axes + x] * sc.slope;
#pragma unroll
            for (int r = 0; r < 16; ++r)
                s[r] = fmaf(-sl,
                            fabsf((float)((double)pk[min(k0 + acc_row(r, half), hi - 1)] - pq)),
                            s[r]);
        }
        const float l = a.lse[((int64_t)b * a.Hq + h) * a.Tq + i];
        const float l2 = l == kNegInf ? kInf : l * kLog2e;
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            const int key = k0 + acc_row(r, half);
            const float p = __builtin_amdgcn_exp2f(fmaf(s[r], sc.mul, -l2));
            if (key >= sp.lo && key < sp.hi) sum = fmaf(p, dp[r], sum);
        }
    }
    sum = halves_sum(sum);
    if (half == 0) sums[wave][col] = sum;
    __syncthreads();
    return true;
}

// float16: what p is rounded times.
constexpr int kWeightBits = 12;

template <typename T>
constexpr bool ranged() { return T::code == F16::code; }

// The largest of 64 lanes' numbers, none negative, without LDS.
template <int CTRL>
__device__ __forceinline__ float dpp_max(float v)
{
    return fmaxf(v, __builtin_bit_cast(
                        float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xf,
                                                           0xf, true)));
}
__device__ __forceinline__ float wave_max(float v)
{
    v = dpp_max<0xb1>(v);                  // quads: lane ^ 1
    v = dpp_max<0x4e>(v);                  // lane ^ 2
    v = dpp_max<0x141>(v);                 // the other quad of 8 lanes (mirrored)
    v = dpp_max<0x140>(v);                 // the other 8 of 16 lanes (mirrored)
    const uint32_t a = __builtin_bit_cast(uint32_t, v);
    const auto x = __builtin_amdgcn_permlane16_swap(a, a, false, false);
    const uint32_t x0 = x[0], x1 = x[1];
    return halves_max(fmaxf(__builtin_bit_cast(float, x0), __builtin_bit_cast(float, x1)));
}

// What e is rounded over, its exponent: of norms of up to `norm` against
// values of up to `most`.  0 where there is no gradient, or one that is not
// finite.
__device__ __forceinline__ int range_exponent(float norm, float most)
{
    const float bound = norm * most;
    return bound > 0.f && bound < kInf ? __builtin_amdgcn_frexp_expf(bound) + 1 - 15 : 0;
}

// Keys whose positions a workgroup of the constants prepares.
__device__ __forceinline__ int keys_share(const AttnArgs &a)
{
    const int nt = (a.Tq + 31) / 32;
    return max((a.Tk + nt - 1) / nt, 1);
}

// float16: keys whose |v| a workgroup of the constants looks at, and how many
// of a key head's workgroups do.  (Not fewer than it has rows of threads for:
// the other kernels read one number for each.)
__device__ __forceinline__ int value_share(const AttnArgs &a)
{
    const int shares = (a.Tq + 31) / 32 * a.G;
    return max((a.Tk + shares - 1) / shares, 16);
}
__device__ __forceinline__ int value_parts(const AttnArgs &a)
{
    const int per = value_share(a);
    return (a.Tk + per - 1) / per;
}

// One workgroup per 32 queries of one head: 8 threads per row.
template <typename T>
__global__ __launch_bounds__(256, 6) void attn_rows_kernel(AttnArgs a)
{
    using R = typename T::raw;
    const int nt = (a.Tq + 31) / 32;
    const int64_t id = (int64_t)blockIdx.y * gridDim.x + blockIdx.x, bh = id / nt;
    if (bh >= (int64_t)a.B * a.Hq) return;
    const int qt = (int)(id - bh * nt);
    const int b = (int)(bh / a.Hq), h = (int)(bh - (int64_t)b * a.Hq);
    const int row = threadIdx.x >> 3, sub = threadIdx.x & 7, i = qt * 32 + row;
    const float l = a.lse[bh * a.Tq + min(i, a.Tq - 1)];
    float s = 0.f, norm = 0.f, value = 0.f;    // norm: |do|_1; value: |v| of a share of the keys
    if constexpr (ranged<T>()) {
        const int hk = h / a.G, per = value_share(a);
        const int L = a.kv_len ? min(a.kv_len[b], a.Tk) : a.Tk;        // (past it: nobody's)
        const int64_t first = ((int64_t)(h - hk * a.G) * nt + qt) * per;
        const int c = (threadIdx.x & 15) * 8;
        const R *v = (const R *)a.v + b * a.vs[0] + hk * a.vs[2];
#pragma unroll 2
        for (int64_t k = first + (threadIdx.x >> 4); k < min(first + per, (int64_t)L); k += 16) {
            struct alignas(16) {
                R e[8];
            } x = __builtin_bit_cast(decltype(x),
                                     load8<T>(v + k * a.vs[1], c, a.D, a.vec));
#pragma unroll
            for (int n = 0; n < 8; ++n) {
                const float y = fabsf(T::widen(x.e[n]));
                value = fmaxf(value, y < kInf ? y : 0.f);
            }
        }
    }
    if (i < a.Tq) {
        const R *o = (const R *)a.out + (((int64_t)b * a.Tq + i) * a.Hq + h) * a.D;
        const R *g = (const R *)a.dout + b * a.gs[0] + (int64_t)i * a.gs[1] + h * a.gs[2];
        const bool ovec = (int64_t)a.D * sizeof(R) % 16 == 0;
#pragma unroll
        for (int d = sub * 8; d < kAttnMaxD; d += 64) {
            struct alignas(16) {
                R e[8];
            } x = __builtin_bit_cast(decltype(x), load8<T>(o, d, a.D, ovec)),
              y = __builtin_bit_cast(decltype(y), load8<T>(g, d, a.D, a.vec));
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                s = fmaf(T::widen(x.e[k]), T::widen(y.e[k]), s);
                if (ranged<T>()) norm += fabsf(T::widen(y.e[k]));
            }
        }
    }
#pragma unroll
    for (int m = 4; m; m >>= 1) {
        s += __shfl_xor(s, m);
        if (ranged<T>()) norm += __shfl_xor(norm, m);
    }
    if constexpr (ranged<T>()) {
        // (what is not finite has no bound; a query that sees nothing no say)
        const bool some = i < a.Tq && norm < kInf && l != kNegInf;
        norm = some ? norm : 0.f;
        if (sub == 0 && i < a.Tq) a.norms[bh * a.Tq + i] = norm;
        __shared__ float most[2][4];
        norm = wave_max(norm);
        value = wave_max(value);
        if ((threadIdx.x & 63) == 0) {
            most[0][threadIdx.x >> 6] = norm;
            most[1][threadIdx.x >> 6] = value;
        }
        __syncthreads();
        if (threadIdx.x < 2) {
            const float *m = most[threadIdx.x];
            (threadIdx.x ? a.v_most : a.norm_most)[bh * nt + qt] =
                fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
        }
    }
    if (sizeof(R) == 2) {
        __shared__ float few[4][32];
        if (few_keys_delta<T>(a, b, h, qt, few)) {
            const float f = few[0][row] + few[1][row] + few[2][row] + few[3][row];
            if (fabsf(f) < kInf) s = f;
        }
    }
    if (sub == 0 && i < a.Tq) {
        const int64_t at = bh * a.Tq + i;
        // a row without weights: its exponents become -inf
        *(float2 *)(a.rowd + 2 * at) = make_float2(
            l == kNegInf ? kInf : fmaf(l, kLog2e, ranged<T>() ? -(float)kWeightBits : 0.f), -s);
    }
    if (h == 0 && a.axes > 0) {
        // this workgroup's share of the positions, and whether one is far
        __shared__ int far[2];
        if (threadIdx.x < 2) far[threadIdx.x] = 0;
        __syncthreads();
        const int per_q = 32, per_k = keys_share(a);
        for (int x = 0; x < a.axes; ++x) {
            const int64_t row = (int64_t)x * a.B + b;
            const int32_t *pk = a.pos_k + row * a.Tk, *pq = a.pos_q + row * a.Tq;
            for (int k = qt * per_k + threadIdx.x; k < min((qt + 1) * per_k, a.Tk); k += 256) {
                const u32x2 p = position_parts(pk[k]);
                ((u32x2 *)a.parts_k)[row * a.Tk + k] = p;
                if (is_far_position(p)) far[1] = 1;
            }
            const int k = qt * per_q + threadIdx.x;
            if (threadIdx.x < per_q && k < a.Tq) {
                const u32x2 p = position_parts(pq[k]);
                ((u32x2 *)a.parts_q)[row * a.Tq + k] = p;
                if (is_far_position(p)) far[0] = 1;
            }
        }
        __syncthreads();
        if (threadIdx.x == 0)
            *(int2 *)(a.fars + 2 * ((int64_t)b * nt + qt)) = make_int2(far[0], far[1]);
    }
    if (h == 0 && threadIdx.x < 64) {
        const int j = qt * 32 + (threadIdx.x & 31);
        Span sp = {0, 0};                  // (past the last query: none)
        if (j < a.Tq) sp = row_span(a, b, j);
        if (threadIdx.x < 32 && j < a.Tq)
            *(int2 *)(a.spans + 2 * ((int64_t)b * a.Tq + j)) = make_int2(sp.lo, sp.hi);
        int lo = sp.hi > sp.lo ? sp.lo : 0x7fffffff, hi = sp.hi, alo = sp.lo, ahi = sp.hi;
#pragma unroll
        for (int m = 16; m; m >>= 1) {
            lo = min(lo, __shfl_xor(lo, m));
            hi = max(hi, __shfl_xor(hi, m));
            alo = max(alo, __shfl_xor(alo, m));
            ahi = min(ahi, __shfl_xor(ahi, m));
        }
        if (threadIdx.x == 0)
            *(int4 *)(a.tiles + 4 * ((int64_t)b * nt + qt)) = make_int4(lo, hi, alo, ahi);
    }
}

// ------------------------------------------------------------------- dq

template <typename T, int DP>
constexpr int bwd_occupancy()
{
    return sizeof(typename T::raw) * DP > 256 ? 1 : 2;
}

template <typename T, int DP, int DU, bool GEN>
__global__ __launch_bounds__(64 * kBwdWaves, (bwd_occupancy<T, DP>())) void attn_dq_kernel(AttnArgs a)
{
    using R = typename T::raw;
    const int axes = GEN ? a.axes : 0;
    constexpr int kStages = stages<T, DP>();
    constexpr int NW = kBwdWaves, NT = 64 * NW, KB = kStep, NC = DU / 16, ND = DU / 32;
    constexpr bool ALL = DU == DP;         // whole tiles with all their channels
    extern __shared__ __align__(16) unsigned char smem[];
    constexpr int TS = KB * DP;                            // elements of a tile
    R *const kt = (R *)smem;                               // [kStages][K tile, V tile]
    // [kStages][3][KB keys' positions, and ones]
    u32x2 *const pk = (u32x2 *)(kt + kStages * 2 * TS);
    int *const bad = (int *)(pk + kStages * 3 * kPos);     // [kStages][KB] 1 + last step whose key
                                                           // held an infinity or a NaN
    int *const flag = bad + kStages * KB;                  // there was one
    int *const ends = flag + 1;                            // [4][NW]

    const int nq = (a.Tq + 32 * NW - 1) / (32 * NW);
    const Block blk = block_of(blockIdx.x, a.B * a.Hq, nq);
    const int bh = blk.head;
    const int b = bh / a.Hq, h = bh - b * a.Hq, hk = h / a.G;
    const int qt = a.order_q ? uniform(a.order_q[(int64_t)b * nq + blk.no]) : nq - 1 - blk.no;
    const int tid = threadIdx.x, wave = uniform(tid >> 6), lane = tid & 63, col = lane & 31,
              half = lane >> 5;
    const int q0 = qt * 32 * NW, i = q0 + wave * 32 + col;
    const int ic = min(i, a.Tq - 1);
    const int2 sp = *(const int2 *)(a.spans + 2 * ((int64_t)b * a.Tq + ic));
    const int nt = (a.Tq + 31) / 32, wt = min(qt * NW + wave, nt - 1);
    const int4 wu = *(const int4 *)(a.tiles + 4 * ((int64_t)b * nt + wt));
    const int wlo = __builtin_amdgcn_readfirstlane(wu.x), whi = __builtin_amdgcn_readfirstlane(wu.y);
    const int alo = __builtin_amdgcn_readfirstlane(wu.z), ahi = __builtin_amdgcn_readfirstlane(wu.w);
    if (lane == 0) {
        ends[wave] = wlo;
        ends[NW + wave] = whi;
        ends[2 * NW + wave] = alo;
        ends[3 * NW + wave] = ahi;
    }
    if (tid < kStages * KB) bad[tid] = 0;
    if (axes > 0 && tid < kStages * 3) pk[tid * kPos + KB] = u32x2{kOnes, kOnes};
    if (tid == 0) *flag = 0;
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
    const R *gp = (const R *)a.dout + b * a.gs[0] + h * a.gs[2] + (int64_t)ic * a.gs[1];
    Frag<T> qf[NC], gf[NC];
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        qf[c] = load8<T>(qp, c * 16 + half * 8, a.D, a.vec);
        gf[c] = load8<T>(gp, c * 16 + half * 8, a.D, a.vec);
    }
    const float2 rd = *(const float2 *)(a.rowd + 2 * ((int64_t)bh * a.Tq + ic));
    const Scores sc = scores(a);
    u32x2 pq[3];
    float sl[3];
    bool far = false;                      // a query's or a key's position is
    if (axes > 0) {
        const int per = keys_share(a);
        for (int t = max(glo, 0) / per + lane; t * (int64_t)per < ghi; t += 64)
            far |= a.fars[2 * ((int64_t)b * nt + t) + 1] != 0;
    }
#pragma unroll
    for (int x = 0; x < 3; ++x) {
        if (x >= axes) break;
        const u32x2 p = ((const u32x2 *)a.parts_q)[((int64_t)x * a.B + b) * a.Tq + ic];
        far |= is_far_position(p);
        pq[x] = position_cols(p, half);
        sl[x] = a.slopes[h * axes + x] * sc.slope;
        arrived(sl[x]);
    }
    const int signed_axes = __any(far) ? -axes : axes;     // (add_bias)

    float lse2 = rd.x, delta = rd.y;       // (delta negated)
    int xq = 0;                            // what e is rounded over, its exponent
    if constexpr (ranged<T>()) {
        const float norm = a.norms[(int64_t)bh * a.Tq + ic];
        const float *v = a.v_most + ((int64_t)b * a.Hq + hk * a.G) * nt;
        const int parts = value_parts(a);
        float most = 0.f;
#pragma unroll 4
        for (int t = lane; t < parts; t += 64) most = fmaxf(most, v[t]);
        xq = range_exponent(norm, wave_max(most));
        lse2 += (float)(kWeightBits + xq);
    }
    arrived(qf);
    arrived(gf);
    arrived(lse2);
    arrived(delta);
    f32x16 o[ND];
#pragma unroll
    for (int d = 0; d < ND; ++d) o[d] = f32x16(0.f);

    const int kbeg = ghi > 0 ? glo / KB * KB : 0, kend = ghi;
    const int steps = kend > kbeg ? (kend - kbeg + KB - 1) / KB : 0;
    TileDirect<T, DP, KB, NT> kd, vd;
    kd.init(tid, a.ks[1], a.D);
    vd.init(tid, a.vs[1], a.D);
    const bool usable = kd.usable(a.vec, a.ks[1], a.D) && vd.usable(a.vec, a.vs[1], a.D);
    if (a.D < DP)                          // channels that no direct load writes
        for (int x = tid; x < kStages * 2 * TS * (int)sizeof(R) / 16; x += NT)
            ((u32x4 *)kt)[x] = u32x4{0u, 0u, 0u, 0u};
    __syncthreads();
    const bool whole = usable && (!ALL || a.D == DP);
    // the next fetch: its step, its stage and where it reads
    const uint32_t lds = lds_address(smem) + wave * 1024,
                   lds_pk = lds_address(pk) + wave * kPos * 8;
    int fn = 0, fst = 0;
    const R *fk = kp + (int64_t)kbeg * a.ks[1], *fv = vp + (int64_t)kbeg * a.vs[1];
    const uint32_t *fpos =
        wave < axes ? a.parts_k + 2 * (((int64_t)wave * a.B + b) * a.Tk + kbeg) : nullptr;
    auto fetch = [&]() {
        const int k0 = kbeg + fn * KB;
        const uint32_t at = lds + fst * 2 * TS * (int)sizeof(R);
        if (whole && glo <= k0 && k0 + KB <= ghi) {
            kd.template load<ALL>(fk, at);
            vd.template load<ALL>(fv, at + TS * (int)sizeof(R));
        } else if (usable) {
            kd.load_edge(kp, a.ks[1], k0, glo, ghi, at);
            vd.load_edge(vp, a.vs[1], k0, glo, ghi, at + TS * (int)sizeof(R));
        }
        if (wave < axes)
            direct4(fpos, (uint32_t)(2 * min(lane >> 1, a.Tk - 1 - k0) + (lane & 1)) * 4,
                    lds_pk + fst * 3 * kPos * 8);
        ++fn;
        fst = fst + 1 < kStages ? fst + 1 : 0;
        fk += KB * a.ks[1];
        fv += KB * a.vs[1];
        fpos += 2 * KB;
    };
    auto clean = [&](int n, int st) {
        const int k0 = kbeg + n * KB;
        const bool edge = k0 < glo || k0 + KB > ghi;
        const bool drop = !(galo <= k0 && k0 + KB <= gahi);
        R *const ks = kt + st * 2 * TS;
        if (!usable) {
            const int t = opaque(threadIdx.x);
            TileRegs<T, DP, KB, NT> r;
            r.load(kp, a.ks[1], k0, glo, ghi, a.D, a.vec, t);
            if (drop && r.drop(bad + st * KB, n + 1, t)) *flag = 1;
            r.store(ks, t);
            r.load(vp, a.vs[1], k0, glo, ghi, a.D, a.vec, t);
            r.store(ks + TS, t);
            wait_all();
        } else if (edge || drop) {
            if (kd.scrub(ks, k0, glo, ghi, drop, bad + st * KB, n + 1)) *flag = 1;
            if (edge) vd.scrub(ks + TS, k0, glo, ghi, false, nullptr, 0);
        }
    };
    // Hands steps n and n + 1 over, which are in stages st and st + 1.
    constexpr int kLater = (kStages - 4) * 2 * TileDirect<T, DP, KB, NT>::LOADS;
    auto arrive = [&](int n, int st) {
        // (all of the later loads are there to be counted only if no step is
        // the last)
        wait_loads<kLater>(usable && n + kStages - 2 <= steps);
#pragma unroll 1
        for (int u = 0; u < 2 && n + u < steps; ++u) clean(n + u, st + u);
        hand_over();
    };
#pragma unroll 1
    while (fn < min(steps, kStages - 2)) fetch();
    if (steps > 0) arrive(0, 0);
    for (int n = 0, st = 0; n < steps; ++n) {
        const int k0 = kbeg + n * KB;
        if (fn < steps) fetch();
        {
            const R *kb = kt + st * 2 * TS, *vb = kb + TS;
            Frag<T> kr[NC], vr[NC], kc[ND][2];
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                kr[c] = row_frag<T, DP>(kb, col, c * 16 + half * 8);
                vr[c] = row_frag<T, DP>(vb, col, c * 16 + half * 8);
            }
            // (16 registers of delta, where they are there)
            constexpr bool kept = DP * sizeof(R) <= 128;
            f32x16 s = f32x16(0.f), dp = f32x16(kept ? delta : 0.f);
#pragma unroll
            for (int c = 0; c < NC; ++c) s = mma<T>(kr[c], qf[c], s);
#pragma unroll
            for (int c = 0; c < NC; ++c) dp = mma<T>(vr[c], gf[c], dp);
#pragma unroll
            for (int d = 0; d < ND; ++d)
#pragma unroll
                for (int c = 0; c < 2; ++c) kc[d][c] = col_frag<T, DP>(kb, c, d * 32, lane);
            reads_ahead<T, NC>();
            products_and_reads<T, NC, 1>();
            products_and_reads<T, NC, 2>();
            issued<T>();
            if constexpr (!kept) {
#pragma unroll
                for (int r = 0; r < 16; ++r) dp[r] += delta;
            }
            const bool part = !(alo <= k0 && k0 + KB <= ahi);
            if (GEN) multiply_scores(s, sc);
            if (GEN && a.cap > 0.f) {
                cap_scores<T>(s, sc, part);
#pragma unroll
                for (int r = 0; r < 16; ++r) dp[r] *= cap_slope(s[r], sc);
            }
            if (GEN && signed_axes != 0)
                add_bias(s, pk + st * 3 * kPos + (half ? KB : col), kPos, signed_axes, pq, sl);
            // (rows were dropped for the whole workgroup: a wave that sees all
            // of the tile meets them too)
            if (!(galo <= k0 && k0 + KB <= gahi) && *flag) {
                const auto x = acc_rows(bad + st * KB, half);
#pragma unroll
                for (int r = 0; r < 16; ++r) s[r] = x[r] == n + 1 ? kNegInf : s[r];
            }
#pragma unroll
            for (int r = 0; r < 16; ++r)
                s[r] = __builtin_amdgcn_exp2f(fmaf(s[r], sc.mul, -lse2)) * dp[r];
            if (part) {
                const uint32_t at = k0 + 4 * half - sp.x, len = sp.y - sp.x;
#pragma unroll
                for (int r = 0; r < 16; ++r) s[r] = at + acc_row(r, 0) < len ? s[r] : 0.f;
            }
            const Frag<T> e0 = pack8<T>(s, 0), e1 = pack8<T>(s, 1);
#pragma unroll
            for (int d = 0; d < ND; ++d) {
                o[d] = add_step<T>(kc[d][0], e0, kc[d][1], e1, o[d]);
            }
        }
        st = st + 1 < kStages ? st + 1 : 0;
        if ((n & 1) && n + 1 < steps) arrive(n + 1, st);
    }
    if (i >= a.Tq) return;
    store_cols<T, ND>((R *)a.dq + (((int64_t)b * a.Tq + i) * a.Hq + h) * a.D, o,
                      ranged<T>() ? ldexpf(a.scale, xq) : a.scale, a.D, half);
}

// -------------------------------------------------------------- dk and dv

// Where one wave cannot hold keys, values and both sums in the registers
// that leave room for a second wave on its SIMD, two waves share 32 keys:
// one sums dv, the other dk (and both form the scores: 5 products where 4
// would do, but the matrix unit is not left waiting for a wave by itself).
// 2 x 2047 float16 tokens, heads of 128: 172 us, one wave a SIMD 206.  With
// 64 channels of 16 bits two waves fit as they are.
template <typename T, int DP>
constexpr bool dkv_pairs()
{
    return sizeof(typename T::raw) * DP > 128 && sizeof(typename T::raw) * DP <= 256;
}
// (with pairs the CU holds one workgroup)
template <typename T, int DP>
constexpr int dkv_stages() { return dkv_pairs<T, DP>() ? 6 : stages<T, DP>(); }

template <typename T, int DP, int DU, bool GEN>
__global__ __launch_bounds__(64 * kBwdWaves * (dkv_pairs<T, DP>() ? 2 : 1),
                             (sizeof(typename T::raw) * DP > 256 ? 1 : 2))
void attn_dkv_kernel(AttnArgs a)
{
    using R = typename T::raw;
    const int axes = GEN ? a.axes : 0;
    constexpr bool PAIRS = dkv_pairs<T, DP>();
    constexpr int kStages = dkv_stages<T, DP>();
    constexpr int NW = kBwdWaves, NT = 64 * NW * (PAIRS ? 2 : 1), QB = kStep, NC = DU / 16,
                  ND = DU / 32;
    constexpr bool ALL = DU == DP;         // whole tiles with all their channels
    extern __shared__ __align__(16) unsigned char smem[];
    constexpr int TS = QB * DP;                            // elements of a tile
    R *const qt = (R *)smem;                               // [kStages][Q tile, dO tile]
    // [kStages] of: [2][QB] lse * log2 e and -delta, [QB][2] spans of keys,
    // [3][QB positions, and ones]
    unsigned char *const small = (unsigned char *)(qt + kStages * 2 * TS);
    auto rc = [&](int st) { return (float *)(small + st * kSmall); };
    auto sp = [&](int st) { return (int *)(small + st * kSmall + 8 * QB); };
    auto pq = [&](int st) { return (u32x2 *)(small + st * kSmall + 16 * QB); };
    int *const flag = (int *)(small + kStages * kSmall);   // an infinity or a NaN was dropped
    int *const ends = flag + 1;                            // [2] first and last tile
    int *const fars = ends + 2;                            // a query's position is far
    int *const most = fars + 1;                            // [2] bits of |do|_1's and |v|'s maxima

    const int nk = (a.Tk + 32 * NW - 1) / (32 * NW);
    const Block blk = block_of(blockIdx.x, a.B * a.Hk * a.gsplit, nk);
    const int gpart = blk.head % a.gsplit, bhk = blk.head / a.gsplit;
    const int b = bhk / a.Hk, hk = bhk - b * a.Hk;
    // (without documents the first keys are seen by the most queries, if causal)
    const int kb = a.order_k ? uniform(a.order_k[(int64_t)b * nk + blk.no]) : blk.no;
    const int g0 = (int)((int64_t)a.G * gpart / a.gsplit);
    const int g1 = (int)((int64_t)a.G * (gpart + 1) / a.gsplit);
    const int tid = threadIdx.x, wave = uniform(tid >> 6), lane = tid & 63, col = lane & 31,
              half = lane >> 5;
    const int k0 = kb * 32 * NW, kw = k0 + wave % NW * 32, key = kw + col;
    const bool second = PAIRS && wave >= NW;              // sums dk
    const int kc = min(key, a.Tk - 1);
    const int nt = (a.Tq + QB - 1) / QB;
    const int32_t *tiles = a.tiles + 4 * (int64_t)b * nt;

    // the tiles of queries that see a key of this block
    if (tid == 0) {
        *flag = *fars = 0;
        most[0] = most[1] = 0;
    }
    if (tid < 2) ends[tid] = tid ? -1 : nt;
    if (axes > 0 && tid < kStages * 3)
        pq(tid / 3)[tid % 3 * kPos + QB] = u32x2{kOnes, kOnes};
    __syncthreads();
    {
        int first = nt, last = -1;
        float norm = 0.f, value = 0.f;
        if constexpr (ranged<T>()) {
            const float *v = a.v_most + ((int64_t)b * a.Hq + hk * a.G) * nt;
            const int parts = nt > 0 ? value_parts(a) : 0;
            for (int t = tid; t < parts; t += NT) value = fmaxf(value, v[t]);
        }
        for (int t = tid; t < nt; t += NT) {
            float here = 0.f;
            if constexpr (ranged<T>())
                for (int g = g0; g < g1; ++g)
                    here = fmaxf(here, a.norm_most[((int64_t)b * a.Hq + hk * a.G + g) * nt + t]);
            const int4 u = *(const int4 *)(tiles + 4 * (int64_t)t);
            const int far = axes > 0 ? a.fars[2 * ((int64_t)b * nt + t)] : 0;
            if (u.x < k0 + 32 * NW && u.y > k0) {
                first = min(first, t);
                last = t;
                if (far) *fars = 1;
                norm = fmaxf(norm, here);
            }
        }
        if constexpr (ranged<T>()) {       // (not negative: their bits are in their order)
            norm = wave_max(norm);
            value = wave_max(value);
            if (lane == 0) {
                atomicMax(most, __builtin_bit_cast(int, norm));
                atomicMax(most + 1, __builtin_bit_cast(int, value));
            }
        }
        if (last >= 0) {
            atomicMin(ends, first);
            atomicMax(ends + 1, last);
        }
    }
    __syncthreads();
    const int first = uniform(ends[0]), last = uniform(ends[1]), span = last - first + 1;
    const int steps = span > 0 ? span * (g1 - g0) : 0;
    // (float16: p is there times 2^kWeightBits)
    const int xk = ranged<T>() ? uniform(range_exponent(__builtin_bit_cast(float, most[0]),
                                                        __builtin_bit_cast(float, most[1])))
                               : 0;
    const float e_unit = ranged<T>() ? ldexpf(1.f, -xk - kWeightBits) : 1.f;

    const R *kp = (const R *)a.k + b * a.ks[0] + hk * a.ks[2] + (int64_t)kc * a.ks[1];
    const R *vp = (const R *)a.v + b * a.vs[0] + hk * a.vs[2] + (int64_t)kc * a.vs[1];
    Frag<T> kf[NC], vf[NC];
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        kf[c] = load8<T>(kp, c * 16 + half * 8, a.D, a.vec);
        vf[c] = load8<T>(vp, c * 16 + half * 8, a.D, a.vec);
    }
    u32x2 pk[3];
    bool far = axes > 0 && *fars;          // a query's or a key's position is
#pragma unroll
    for (int x = 0; x < 3; ++x) {
        if (x >= axes) break;
        const u32x2 p = ((const u32x2 *)a.parts_k)[((int64_t)x * a.B + b) * a.Tk + kc];
        far |= is_far_position(p);
        pk[x] = position_cols(p, half);
    }
    const int signed_axes = __any(far) ? -axes : axes;     // (add_bias)
    const Scores sc = scores(a);
    arrived(kf);
    arrived(vf);
    f32x16 dv[ND], more[PAIRS ? 1 : ND];   // (the second wave's sums are in dv too)
    f32x16 *const dk = PAIRS ? dv : more;
#pragma unroll
    for (int d = 0; d < ND; ++d) dk[d] = dv[d] = f32x16(0.f);

    TileDirect<T, DP, QB, NT> qd, gd;
    qd.init(tid, a.qs[1], a.D);
    gd.init(tid, a.gs[1], a.D);
    const bool usable = qd.usable(a.vec, a.qs[1], a.D) && gd.usable(a.vec, a.gs[1], a.D);
    if (a.D < DP)                          // channels that no direct load writes
        for (int x = tid; x < kStages * 2 * TS * (int)sizeof(R) / 16; x += NT)
            ((u32x4 *)qt)[x] = u32x4{0u, 0u, 0u, 0u};
    __syncthreads();
    const bool whole = usable && (!ALL || a.D == DP);
    const R *const qbase = (const R *)a.q + b * a.qs[0], *const gbase =
        (const R *)a.dout + b * a.gs[0];
    // The next fetch: its step, stage, head and tile, and where it reads.
    // Of the first waves each reads 256 bytes with the tile: the rows'
    // constants, the spans, the positions on two axes (wave 3 those on the
    // third too).
    int fn = 0, fst = 0, fh = hk * a.G + g0, ft = first;
    const uint32_t lds = lds_address(smem) + wave * 1024,
                   lds_small = lds_address(small) +
                               (wave < 2 ? wave * 8 * QB : 16 * QB + (wave % NW - 2) * kPos * 8);
    const R *fq, *fg;
    const char *fs;
    auto rewind = [&]() MP3D_INLINE {                  // to tile ft of head fh
        const int64_t at = (int64_t)ft * QB;
        fq = qbase + fh * a.qs[2] + at * a.qs[1];
        fg = gbase + fh * a.gs[2] + at * a.gs[1];
        if (wave == 0) fs = (const char *)(a.rowd + 2 * (((int64_t)b * a.Hq + fh) * a.Tq + at));
        else if (wave == 1) fs = (const char *)(a.spans + 2 * ((int64_t)b * a.Tq + at));
        else fs = (const char *)(a.parts_q + 2 * (((int64_t)(wave % NW - 2) * a.B + b) * a.Tq + at));
    };
    rewind();
    const uint32_t pair_of = lane * 4, parted = (2 * col + half) * 4;
    const uint32_t mine = wave == 0 ? parted : pair_of;    // (constants are parted on the way)
    const int64_t third = (int64_t)a.B * a.Tq * 8;
    auto fetch = [&]() MP3D_INLINE {
        const int q0 = ft * QB;
        const uint32_t at = lds + fst * 2 * TS * (int)sizeof(R), as = lds_small + fst * kSmall;
        uint32_t off = mine;
        if (whole && q0 + QB <= a.Tq) {
            qd.template load<ALL>(fq, at);
            gd.template load<ALL>(fg, at + TS * (int)sizeof(R));
        } else {
            if (usable) {
                qd.load_edge(qbase + fh * a.qs[2], a.qs[1], q0, 0, a.Tq, at);
                gd.load_edge(gbase + fh * a.gs[2], a.gs[1], q0, 0, a.Tq, at + TS * (int)sizeof(R));
            }
            // (the last query's for those past it)
            off = min(mine, (uint32_t)(a.Tq - 1 - q0) * 8 + (mine & 4));
        }
        if (wave < 2 + min(axes, 2)) direct4(fs, off, as);
        if (wave == 3 && axes == 3) direct4(fs + third, off, as + kPos * 8);
        ++fn;
        fst = fst + 1 < kStages ? fst + 1 : 0;
        if (++ft > last) {
            ft = first;
            ++fh;
            rewind();
        } else {
            fq += QB * a.qs[1];
            fg += QB * a.gs[1];
            fs += 8 * QB;
        }
    };
    // What the 32 queries of a tile see together, for 64 tiles in the lanes.
    int all_lo = 0, all_hi = 0, have = 0x7fffffff;
    auto seen_by_all = [&](int t, int *lo, int *hi) MP3D_INLINE {
        if (t < have || t >= have + 64) {
            have = t;
            const int2 u = *(const int2 *)(tiles + 4 * (int64_t)min(t + lane, nt - 1) + 2);
            all_lo = u.x;
            all_hi = u.y;
            arrived(all_lo);
            arrived(all_hi);
        }
        *lo = __builtin_amdgcn_readlane(all_lo, t - have);
        *hi = __builtin_amdgcn_readlane(all_hi, t - have);
    };
    struct Step {
        int h, t;                          // head and tile
        int lo, hi;                        // the keys that all of its queries see
    };
    auto following = [&](Step x) MP3D_INLINE {
        Step y = {x.t < last ? x.h : x.h + 1, x.t < last ? x.t + 1 : first, 0, 0};
        seen_by_all(y.t, &y.lo, &y.hi);
        return y;
    };
    auto clean = [&](const Step &x, int st) MP3D_INLINE {
        const int q0 = x.t * QB;
        const bool edge = q0 + QB > a.Tq, drop = !(x.lo <= k0 && k0 + 32 * NW <= x.hi);
        R *const qs = qt + st * 2 * TS;
        if (!usable && second) {
            // the other half of the workgroup does it
        } else if (!usable) {
            const int t = opaque(threadIdx.x);
            TileRegs<T, DP, QB, 64 * NW> r;
            r.load(qbase + x.h * a.qs[2], a.qs[1], q0, 0, a.Tq, a.D, a.vec, t);
            if (drop && r.drop()) *flag = 1;
            r.store(qs, t);
            r.load(gbase + x.h * a.gs[2], a.gs[1], q0, 0, a.Tq, a.D, a.vec, t);
            if (drop && r.drop()) *flag = 1;
            r.store(qs + TS, t);
            wait_all();
        } else if (edge || drop) {
            if (qd.scrub(qs, q0, 0, a.Tq, drop, nullptr, 0)) *flag = 1;
            if (gd.scrub(qs + TS, q0, 0, a.Tq, drop, nullptr, 0)) *flag = 1;
        }
        if (edge) {                        // past the last query: no weight, no keys
            const int i = opaque(lane);
            if (wave == 0 && q0 + (i & 31) >= a.Tq) rc(st)[i] = i < QB ? kInf : 0.f;
            if (wave == 1 && q0 + (i >> 1) >= a.Tq) sp(st)[i] = 0;
        }
    };
    // Hands steps n (x) and n + 1 over, which are in stages st and st + 1.
    constexpr int kLater = (kStages - 4) * 2 * TileDirect<T, DP, QB, NT>::LOADS;
    auto arrive = [&](int n, int st, Step x) MP3D_INLINE {
        // (all of the later loads are there to be counted only if no step is
        // the last)
        wait_loads<kLater>(usable && n + kStages - 2 <= steps);
#pragma unroll 1
        for (int u = 0; u < 2 && n + u < steps; ++u) {
            clean(x, st + u);
            x = following(x);
        }
        hand_over();
    };
    float sl[3] = {0.f, 0.f, 0.f};
    int sl_of = -1;                        // the head they are of
    // A step's part of dv, of dk, or of both.
    auto sums = [&](auto want_v, auto want_k, const Step &x, int st) MP3D_INLINE {
        constexpr bool V = decltype(want_v)::value, K = decltype(want_k)::value;
        const R *qb = qt + st * 2 * TS, *gb = qb + TS;
        const bool part = !(x.lo <= kw && kw + 32 <= x.hi);
        Frag<T> qr[NC], gr[NC], qc[ND][2], gc[ND][2];
        f32x16 s = f32x16(0.f), dp;
#pragma unroll
        for (int c = 0; c < NC; ++c) qr[c] = row_frag<T, DP>(qb, col, c * 16 + half * 8);
#pragma unroll
        for (int c = 0; c < NC; ++c) s = mma<T>(qr[c], kf[c], s);
        if constexpr (K) {
            dp = acc_rows(rc(st) + QB, half);
#pragma unroll
            for (int c = 0; c < NC; ++c) gr[c] = row_frag<T, DP>(gb, col, c * 16 + half * 8);
#pragma unroll
            for (int c = 0; c < NC; ++c) dp = mma<T>(gr[c], vf[c], dp);
        }
        const f32x16 lr = acc_rows(rc(st), half);
        if constexpr (V) {
#pragma unroll
            for (int d = 0; d < ND; ++d)
#pragma unroll
                for (int c = 0; c < 2; ++c) gc[d][c] = col_frag<T, DP>(gb, c, d * 32, lane);
        }
        reads_ahead<T, NC>();
        if constexpr (K) products_and_reads<T, NC, 1>();
        products_and_reads<T, NC, V ? 2 + 8 / NC : 8 / NC>();
        issued<T>();
        if (GEN) multiply_scores(s, sc);
        if (GEN && a.cap > 0.f) {
            cap_scores<T>(s, sc, part);
            if constexpr (K) {
#pragma unroll
                for (int r = 0; r < 16; ++r) dp[r] *= cap_slope(s[r], sc);
            }
        }
        if (GEN && signed_axes != 0)
            add_bias(s, pq(st) + (half ? QB : col), kPos, signed_axes, pk, sl);
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            s[r] = __builtin_amdgcn_exp2f(fmaf(s[r], sc.mul, -lr[r]));
            if constexpr (K) dp[r] *= ranged<T>() ? s[r] * e_unit : s[r];
        }
        if (part) {
            i32x16 lo, hi;
            acc_pairs(sp(st), half, &lo, &hi);
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const bool see = key >= lo[r] && key < hi[r];
                if constexpr (V) s[r] = see ? s[r] : 0.f;
                if constexpr (K) dp[r] = see ? dp[r] : 0.f;
            }
        }
        Frag<T> p0, p1, e0, e1;
        if constexpr (V) {
            p0 = pack8<T>(s, 0);
            p1 = pack8<T>(s, 1);
        }
        if constexpr (K) {
            e0 = pack8<T>(dp, 0);
            e1 = pack8<T>(dp, 1);
        }
#pragma unroll
        for (int d = 0; d < ND; ++d) {
            if constexpr (V) {
                dv[d] = add_step<T>(gc[d][0], p0, gc[d][1], p1, dv[d]);
            }
            if constexpr (K) {
                qc[d][0] = col_frag<T, DP>(qb, 0, d * 32, lane);
                qc[d][1] = col_frag<T, DP>(qb, 1, d * 32, lane);
            }
        }
        if constexpr (K) {
#pragma unroll
            for (int d = 0; d < ND; ++d) {
                dk[d] = add_step<T>(qc[d][0], e0, qc[d][1], e1, dk[d]);
            }
        }
        if constexpr (V && K) products_and_reads<T, 2 * ND, 2>();
        else if constexpr (K) reads_ahead<T, 4>();
        if constexpr (V) products_and_reads<T, 2 * ND, 0>();
        else products_and_reads<T, 2 * ND, 2>();
        issued<T>();
    };
    auto walk = [&](auto want_v, auto want_k) MP3D_INLINE {
#pragma unroll 1
        while (fn < min(steps, kStages - 2)) fetch();
        Step x = {hk * a.G + g0, first, 0, 0};
        if (steps > 0) {
            seen_by_all(x.t, &x.lo, &x.hi);
            arrive(0, 0, x);
        }
        for (int n = 0, st = 0; n < steps; ++n) {
            if (fn < steps) fetch();
            if (axes > 0 && x.h != sl_of) {
                sl_of = x.h;
#pragma unroll
                for (int c = 0; c < 3; ++c) {
                    sl[c] = uniform_load(a.slopes + x.h * axes + min(c, axes - 1)) * sc.slope;
                    arrived(sl[c]);
                }
            }
            sums(want_v, want_k, x, st);
            x = following(x);
            st = st + 1 < kStages ? st + 1 : 0;
            if ((n & 1) && n + 1 < steps) arrive(n + 1, st, x);
        }
    };
    if constexpr (!PAIRS) walk(std::true_type(), std::true_type());
    else if (second) walk(std::false_type(), std::true_type());
    else walk(std::true_type(), std::false_type());
    if (*flag && !second) {                // (the loop's last barrier is behind us)
        // infinities and NaN of do that were dropped, for the keys they reach
        // (in dk they are there already: e is NaN with them)
        for (int n = 0; n < steps; ++n) {
            const int32_t *u = tiles + 4 * (int64_t)(first + n % span);
            if (u[2] <= k0 && k0 + 32 * NW <= u[3]) continue;
            const int h = hk * a.G + g0 + n / span, q0 = (first + n % span) * QB;
            for (int i = q0; i < min(q0 + QB, a.Tq); ++i) {
                const int2 span2 = *(const int2 *)(a.spans + 2 * ((int64_t)b * a.Tq + i));
                const R *g = (const R *)a.dout + b * a.gs[0] + (int64_t)i * a.gs[1] + h * a.gs[2];
                if (key < span2.x || key >= span2.y) continue;
#pragma unroll
                for (int d = 0; d < ND; ++d)
#pragma unroll
                    for (int r = 0; r < 16; ++r) {
                        const int e = d * 32 + acc_row(r, half);
                        const float v = e < a.D ? T::widen(g[e]) : 0.f;
                        if (!(fabsf(v) < kInf)) dv[d][r] += v;
                    }
            }
        }
    }
    if (key >= a.Tk) return;
    const int64_t at = (((int64_t)b * a.Tk + key) * a.Hk + hk) * a.D;
    const int64_t part = gpart * (int64_t)a.B * a.Tk * a.Hk * a.D + at;
    if (!PAIRS || second) {
        const float f = ranged<T>() ? ldexpf(a.scale, xk) : a.scale;
        if (a.gsplit == 1) store_cols<T, ND>((R *)a.dk + at, dk, f, a.D, half);
        else store_cols<F32, ND>(a.part_dk + part, dk, f, a.D, half);
    }
    if (!second) {
        constexpr float f = ranged<T>() ? 1.f / (1 << kWeightBits) : 1.f;
        if (a.gsplit == 1) store_cols<T, ND>((R *)a.dv + at, dv, f, a.D, half);
        else store_cols<F32, ND>(a.part_dv + part, dv, f, a.D, half);
    }
}

// Adds the parts of dk and dv (blockIdx.y) in order.
template <typename T>
__global__ __launch_bounds__(256) void attn_parts_kernel(AttnArgs a)
{
    using R = typename T::raw;
    const int64_t all = (int64_t)a.B * a.Tk * a.Hk * a.D;
    const float *p = blockIdx.y ? a.part_dv : a.part_dk;
    R *out = (R *)(blockIdx.y ? a.dv : a.dk);
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < all;
         i += (int64_t)gridDim.x * 256) {
        float s = 0.f;
        for (int g = 0; g < a.gsplit; ++g) s += p[g * all + i];
        out[i] = T::narrow(s);
    }
}

template <typename T, int DP, int DU, bool GEN>
hipError_t run(const AttnArgs &a, hipStream_t s)
{
    constexpr int NW = kBwdWaves;
    hipError_t e;
    constexpr uint32_t tile = 2 * kStep * DP * sizeof(typename T::raw);
    constexpr int sq = stages<T, DP>(), sk = dkv_stages<T, DP>();
    const int64_t nq = (a.Tq + 32 * NW - 1) / (32 * NW);
    const int64_t nk = (a.Tk + 32 * NW - 1) / (32 * NW);
    if (nk > 0) {
        launch_kernel((attn_dkv_kernel<T, DP, DU, GEN>), dim3((uint32_t)(nk * a.B * a.Hk * a.gsplit)),
                      dim3(64 * NW * (dkv_pairs<T, DP>() ? 2 : 1)), sk * (tile + kSmall) + 6 * 4, s, a);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    if (nk > 0 && a.gsplit > 1) {
        const int64_t need = ((int64_t)a.B * a.Tk * a.Hk * a.D + 255) / 256;
        launch_kernel((attn_parts_kernel<T>),
                      dim3((uint32_t)(need < kMaxTileGrid ? need : kMaxTileGrid), 2), dim3(256), 0,
                      s, a);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    if (nq > 0)
        launch_kernel((attn_dq_kernel<T, DP, DU, GEN>), dim3((uint32_t)(nq * a.B * a.Hq)),
                      dim3(64 * NW), sq * (tile + 3 * kPos * 8 + kStep * 4) + (1 + 4 * NW) * 4, s, a);
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

int64_t round16(int64_t bytes) { return (bytes + 15) & ~(int64_t)15; }

}  // namespace

// A key head's query heads are dealt out until two workgroups a CU are there
// (2 x 2047 with 8 heads a key head: dk, dv 175 us and 15.5 for the sum of the
// parts, 740 without).  Workspace: tiles, spans, rowd, the blocks' orders, the
// positions and what is far of them, float16's bounds, then the parts (each
// at a multiple of 16 bytes).
size_t plan_attn_backward(AttnArgs *a)
{
    const int64_t blocks = (int64_t)((a->Tk + kAttnRows - 1) / kAttnRows) * a->B * a->Hk;
    const int64_t want = 2 * device_cus();
    int64_t g = blocks > 0 ? (want + blocks - 1) / blocks : 1;
    a->gsplit = (int32_t)(g < 1 ? 1 : g > a->G ? a->G : g);
    const int64_t nt = (a->Tq + 31) / 32, rows = (int64_t)a->B * a->Tq;
    int64_t n = round16(rows * a->Hq * 8) + round16(rows * 8) + (int64_t)a->B * nt * 16 +
                attn_order_bytes(*a, false) + attn_order_bytes(*a, true) +
                round16((int64_t)a->axes * rows * 8) +
                round16((int64_t)a->axes * a->B * a->Tk * 8) +
                round16(a->axes > 0 ? a->B * nt * 8 : 0);
    if (a->f16) n += round16(rows * a->Hq * 4) + 2 * round16(a->B * nt * a->Hq * 4);
    if (a->gsplit > 1)
        n += 2 * round16((int64_t)a->gsplit * a->B * a->Tk * a->Hk * a->D * 4);
    return (size_t)n;
}

void place_attn_backward(AttnArgs *a, void *workspace)
{
    const int64_t nt = (a->Tq + 31) / 32, rows = (int64_t)a->B * a->Tq;
    char *p = (char *)workspace;
    a->tiles = (int32_t *)p;
    p += (int64_t)a->B * nt * 16;
    a->spans = (int32_t *)p;
    p += round16(rows * 8);
    a->rowd = (float *)p;
    p += round16(rows * a->Hq * 8);
    const int64_t oq = attn_order_bytes(*a, false), ok = attn_order_bytes(*a, true);
    a->order_q = oq ? (int32_t *)p : nullptr;
    p += oq;
    a->order_k = ok ? (int32_t *)p : nullptr;
    p += ok;
    a->parts_q = (uint32_t *)p;
    p += round16((int64_t)a->axes * rows * 8);
    a->parts_k = (uint32_t *)p;
    p += round16((int64_t)a->axes * a->B * a->Tk * 8);
    a->fars = (int32_t *)p;
    p += round16(a->axes > 0 ? a->B * nt * 8 : 0);
    if (a->f16) {
        a->norm_most = (float *)p;
        p += round16(a->B * nt * a->Hq * 4);
        a->v_most = (float *)p;
        p += round16(a->B * nt * a->Hq * 4);
        a->norms = (float *)p;
        p += round16(rows * a->Hq * 4);
    }
    a->part_dk = (float *)p;
    p += round16((int64_t)a->gsplit * a->B * a->Tk * a->Hk * a->D * 4);
    a->part_dv = (float *)p;
}

template <typename T>
hipError_t launch_attn_backward(const AttnArgs &a, hipStream_t s)
{
    const int64_t nt = (a.Tq + 31) / 32;
    // (a kernel reads what the one before it wrote: none follows a failed launch)
    hipError_t e;
    if (nt > 0) {
        // four times the workgroups of the other kernels, which may pass the
        // 2^32 threads of a launch along x
        const int64_t blocks = nt * a.B * a.Hq, x = blocks < kRowsGrid ? blocks : kRowsGrid;
        launch_kernel((attn_rows_kernel<T>), dim3((uint32_t)x, (uint32_t)((blocks + x - 1) / x)),
                      dim3(256), 0, s, a);
        if ((e = hipGetLastError()) != hipSuccess) return e;
        launch_attn_order(a, true, s);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    return attn_general(a) ? run_width<T, true>(a, s) : run_width<T, false>(a, s);
}

template hipError_t launch_attn_backward<F32>(const AttnArgs &, hipStream_t);
template hipError_t launch_attn_backward<F16>(const AttnArgs &, hipStream_t);
template hipError_t launch_attn_backward<BF16>(const AttnArgs &, hipStream_t);

}  // namespace mp3d
