// rope.hip -- rotary positions with three axes over q and k in one launch.
//
// Pair i < P of a head's first 2P channels (channels i and P + i, or 2i and
// 2i + 1 when interleaved) turns by theta = pos[axis(i)] * inv_freq[i]:
//   (u, v) -> (u cos - v sin, u sin + v cos).
// The map is orthogonal, so its backward is the same kernel with -theta.
//
// Bound: HBM (each element read and written once, about six operations per
// pair and head).  The angle depends on the token and the pair only, so a
// thread computes the sines of its few pairs once and walks the heads with
// them.  theta is formed in binary64 turns: the product pos * inv_freq in
// binary32 is off by theta * 2^-24 radians, which at positions in the
// thousands is already more than a binary32 output's last place.
//
// Measured: 4 x 8 x 56 x 56 bfloat16 tokens of 16 + 4 heads of 128 (1.03 GB)
// 214 us, 4.8 TB/s, where a copy reaches 5.0; 7840 float32 tokens of 12 + 12
// heads of 80, interleaved, backward (121 MB) 23.7 us, 5.1 TB/s; one token of
// each of 32 sequences 6 us, of which the launch and the sines are nearly all.
#include "dtype.hpp"
#include "tokens.hpp"

namespace mp3d {

namespace {

constexpr int kHeadBatch = 4;              // heads loaded before the first is stored

template <int BYTES> struct Wide;
template <> struct Wide<16> { using type = u32x4; };
template <> struct Wide<8> { using type = u32x2; };
template <> struct Wide<4> { using type = uint32_t; };
template <> struct Wide<2> { using type = uint16_t; };

template <typename R, int V>
struct alignas(sizeof(R) * V) Pack {
    R e[V];
};

template <typename R, int V>
__device__ __forceinline__ Pack<R, V> ld(const R *p)
{
    using W = typename Wide<sizeof(R) * V>::type;
    return __builtin_bit_cast(Pack<R, V>, *(const W *)p);
}

template <typename R, int V>
__device__ __forceinline__ void st(R *p, Pack<R, V> v)
{
    using W = typename Wide<sizeof(R) * V>::type;
    *(W *)p = __builtin_bit_cast(W, v);
}

// sine and cosine of 2 pi t: reduced to the nearest quarter turn in
// binary64, then the Taylor polynomials on [-pi/4, pi/4] (the first term
// left out is under 2e-9)
__device__ __forceinline__ void sincos_turns(double t, float *sn, float *cs)
{
    const double f = 4.0 * (t - rint(t)), q = rint(f);
    const float r = (float)((f - q) * 1.5707963267948966);
    const float r2 = r * r;
    float s = 1.f / 362880.f;
    s = fmaf(s, r2, -1.f / 5040.f);
    s = fmaf(s, r2, 1.f / 120.f);
    s = fmaf(s, r2, -1.f / 6.f);
    s = fmaf(s * r2, r, r);
    float c = -1.f / 3628800.f;
    c = fmaf(c, r2, 1.f / 40320.f);
    c = fmaf(c, r2, -1.f / 720.f);
    c = fmaf(c, r2, 1.f / 24.f);
    c = fmaf(c, r2, -0.5f);
    c = fmaf(c, r2, 1.f);
    const int k = (int)q;                  // -2 .. 2
    const float a = (k & 1) ? c : s, b = (k & 1) ? s : c;
    *sn = (k & 2) ? -a : a;
    *cs = ((k + 1) & 2) ? -b : b;
}

// One thread: one unit of one token (V channels of each half, or V adjacent
// channels when interleaved, or V channels that do not turn) over the heads
// [h0, h1) of q and k.
template <typename T, int V, bool IL>
__global__ __launch_bounds__(kBlock) void rope_kernel(RopePlan p)
{
    using R = typename T::raw;
    constexpr int NP = IL ? (V > 1 ? V / 2 : 1) : V;     // pairs per unit
    const int lt = threadIdx.x / p.units, u = threadIdx.x - lt * p.units;
    if (lt >= p.tpb) return;
    const int nh = p.heads[0] + p.heads[1];
    const int h0 = blockIdx.y * p.hpt, h1 = min(nh, h0 + p.hpt);
    const int64_t tokens = p.B * p.T, step = (int64_t)gridDim.x * p.tpb;
    for (int64_t tok = (int64_t)blockIdx.x * p.tpb + lt; tok < tokens; tok += step) {
        const int64_t b = p.B == 1 ? 0 : tok / p.T, t = tok - b * p.T;
        for (int uu = u; uu < p.units; uu += kBlock) {
            const bool turn = uu < p.rot_units;
            float sn[NP], cs[NP];
            int c0, c1;                    // channels of the first and the second vector
            if (turn) {
                const int i0 = uu * NP;
                int32_t at[3];
                if (p.pos) {
#pragma unroll
                    for (int a = 0; a < 3; ++a) at[a] = p.pos[a * tokens + tok];
                } else {
                    const int32_t c = (int32_t)t, r = c / p.gw;
                    at[0] = r / p.gh;
                    at[1] = r - at[0] * p.gh;
                    at[2] = c - r * p.gw;
                }
#pragma unroll
                for (int j = 0; j < NP; ++j) {
                    const int i = i0 + j;
                    const int32_t w = i < p.e0 ? at[0] : i < p.e1 ? at[1] : at[2];
                    sincos_turns((double)w * ((double)p.freq[i] * 0.15915494309189535), &sn[j],
                                 &cs[j]);
                    sn[j] *= p.sign;
                }
                c0 = IL ? 2 * i0 : i0;
                c1 = IL ? 2 * i0 + 1 : p.P + i0;
            } else {
                c0 = c1 = 2 * p.P + (uu - p.rot_units) * V;
            }
            for (int h = h0; h < h1; h += kHeadBatch) {
                Pack<R, V> a[kHeadBatch], c[kHeadBatch];
#pragma unroll
                for (int n = 0; n < kHeadBatch; ++n) {
                    const int hh = h + n < h1 ? h + n : h1 - 1;
                    const int which = hh >= p.heads[0];
                    const R *src = (const R *)p.src[which] + b * p.ss[which][0] +
                                   t * p.ss[which][1] +
                                   (hh - (which ? p.heads[0] : 0)) * p.ss[which][2];
                    a[n] = ld<R, V>(src + c0);
                    if (!(IL && V > 1)) c[n] = ld<R, V>(src + c1);
                }
#pragma unroll
                for (int n = 0; n < kHeadBatch; ++n) {
                    if (h + n >= h1) break;
                    if (turn) {
#pragma unroll
                        for (int j = 0; j < NP; ++j) {
                            R &eu = IL && V > 1 ? a[n].e[(2 * j) % V] : a[n].e[j];
                            R &ev = IL && V > 1 ? a[n].e[(2 * j + 1) % V] : c[n].e[j];
                            const float x = T::widen(eu), y = T::widen(ev);
                            eu = T::narrow(x * cs[j] - y * sn[j]);
                            ev = T::narrow(x * sn[j] + y * cs[j]);
                        }
                    }
                    const int hh = h + n, which = hh >= p.heads[0];
                    R *dst = (R *)p.dst[which] + b * p.ds[which][0] + t * p.ds[which][1] +
                             (hh - (which ? p.heads[0] : 0)) * p.ds[which][2];
                    st<R, V>(dst + c0, a[n]);
                    if (!(IL && V > 1) && turn) st<R, V>(dst + c1, c[n]);
                }
            }
        }
    }
}

template <typename T, int V>
void launch_v(const RopePlan &p, dim3 grid, hipStream_t s)
{
    if (p.interleaved)
        launch_kernel((rope_kernel<T, V, true>), grid, dim3(kBlock), 0, s, p);
    else
        launch_kernel((rope_kernel<T, V, false>), grid, dim3(kBlock), 0, s, p);
}

}  // namespace

// All heads of a token per thread where there are threads enough to fill the
// card without splitting the heads; else as few as a batch of loads.
void plan_rope_heads(RopePlan *p)
{
    const int nh = p->heads[0] + p->heads[1];
    const int64_t want = 8 * kBlock * (int64_t)device_cus();
    const int64_t threads = p->B * p->T * p->units;
    int64_t parts = (want + threads - 1) / threads;
    int64_t hpt = (nh + parts - 1) / parts;
    hpt = (hpt + kHeadBatch - 1) / kHeadBatch * kHeadBatch;
    p->hpt = (int32_t)hpt;
}

template <typename T>
hipError_t launch_rope(const RopePlan &p, hipStream_t s)
{
    const int64_t tokens = p.B * p.T, blocks = (tokens + p.tpb - 1) / p.tpb;
    const int nh = p.heads[0] + p.heads[1];
    const dim3 grid((uint32_t)(blocks < (1 << 18) ? blocks : (1 << 18)),
                    (uint32_t)((nh + p.hpt - 1) / p.hpt));
    switch (p.vec) {
    case 8:
        if constexpr (sizeof(typename T::raw) == 2) launch_v<T, 8>(p, grid, s);
        break;
    case 4:
        if constexpr (sizeof(typename T::raw) == 4) launch_v<T, 4>(p, grid, s);
        break;
    case 2: launch_v<T, 2>(p, grid, s); break;
    default: launch_v<T, 1>(p, grid, s); break;
    }
    return hipGetLastError();
}

template hipError_t launch_rope<F32>(const RopePlan &, hipStream_t);
template hipError_t launch_rope<F16>(const RopePlan &, hipStream_t);
template hipError_t launch_rope<BF16>(const RopePlan &, hipStream_t);

}  // namespace mp3d
