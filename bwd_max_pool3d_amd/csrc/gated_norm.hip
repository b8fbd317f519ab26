// gated_norm.hip -- the norm after a block, its gate and residual scale, the
// residual sum and the norm before the next block, in one pass; backward.
//
//   y = x + rs * gate * post * n(h)         z = pre * n(y)
//   n(a) = (a - mean) * r,  r = 1 / sqrt(mean((a - mean)^2) + eps)
// (mean is 0 for the RMS norm).  With a gradient d at n(a), the gradient at
// a is r * (d - mean(d) - n * mean(d n)), without mean(d) for the RMS norm.
//
// Bound: HBM.  A row lives in registers between its reductions, so x and h
// are read once and y and z written once; the mean is taken before the
// squares, so no cancellation.  The backward forms y again from x and h in
// binary32 (the stored y is rounded) and reads no stored y.
//
// The sums over rows (gradients of the weights and of the gate) are kept by
// a fixed number of workgroups that walk the rows, one partial row each in
// the workspace, then added in a fixed order: no atomics, the same bits on
// every run.
//
// Measured, 43740 x 1024 bfloat16, RMS: forward 72 us (5.0 TB/s), backward
// 94 us (5.7 TB/s), its join 6 us; 7840 x 1001 float32, layer norm, rows not
// aligned to 16 bytes: 26 and 37 us (4.1 TB/s in all).  A copy reaches
// 5.0 TB/s.
#include "dtype.hpp"
#include "tokens.hpp"

namespace mp3d {

namespace {

constexpr int kNormWg = 768;               // backward workgroups of 256 threads to aim for

// The elements of a thread: V adjacent ones of every TPR * V, so that a
// wave reads whole lines.
template <typename T, int TPR, int EPT, int V>
struct Row {
    using R = typename T::raw;
    float e[EPT];

    __device__ __forceinline__ void load(const R *p, int t, int C)
    {
#pragma unroll
        for (int j = 0; j < EPT / V; ++j) {
            const int c = (j * TPR + t) * V;
            if (c < C) {
                if constexpr (V == 1) {
                    e[j] = T::widen(p[c]);
                } else {
                    T::unpack(*(const u32x4 *)(p + c), e + j * V);
                }
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i) e[j * V + i] = 0.f;
            }
        }
    }
    __device__ __forceinline__ void fill(float v)
    {
#pragma unroll
        for (int i = 0; i < EPT; ++i) e[i] = v;
    }
    __device__ __forceinline__ void load_or(const void *p, int64_t off, int t, int C, float v)
    {
        if (p) load((const R *)p + off, t, C);
        else fill(v);
    }
    __device__ __forceinline__ void store(R *p, int t, int C) const
    {
#pragma unroll
        for (int j = 0; j < EPT / V; ++j) {
            const int c = (j * TPR + t) * V;
            if (c < C) {
                if constexpr (V == 1) {
                    p[c] = T::narrow(e[j]);
                } else {
                    struct alignas(16) { R r[V]; } o;
#pragma unroll
                    for (int i = 0; i < V; ++i) o.r[i] = T::narrow(e[j * V + i]);
                    st_stream((u32x4 *)(p + c), __builtin_bit_cast(u32x4, o));
                }
            }
        }
    }
    __device__ static __forceinline__ int col(int k, int t)
    {
        return ((k / V) * TPR + t) * V + k % V;
    }
};

// The same elements as they are stored: in flight, or kept, in half the
// registers for 16-bit types.
template <typename T, int TPR, int EPT, int V>
struct RawRow {
    using R = typename T::raw;
    struct alignas(V > 1 ? 16 : sizeof(R)) Pack {
        R r[V];
    } q[EPT / V];

    __device__ __forceinline__ void load(const void *p, int64_t off, int t, int C)
    {
#pragma unroll
        for (int j = 0; j < EPT / V; ++j) {
            const int c = (j * TPR + t) * V;
            const R *s = (const R *)p + off + c;
            if (c < C) {
                if constexpr (V == 1) q[j].r[0] = *s;
                else q[j] = __builtin_bit_cast(Pack, *(const u32x4 *)s);
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i) q[j].r[i] = 0;
            }
        }
    }
    __device__ __forceinline__ void fill(float v)
    {
#pragma unroll
        for (int k = 0; k < EPT; ++k) q[k / V].r[k % V] = T::narrow(v);
    }
    __device__ __forceinline__ void load_or(const void *p, int64_t off, int t, int C, float v)
    {
        if (p) load(p, off, t, C);
        else fill(v);
    }
    __device__ __forceinline__ float operator[](int k) const { return T::widen(q[k / V].r[k % V]); }
};

// Sum over the 64 lanes, in every lane (each step adds the same two values in
// both of a pair's lanes, so all get the same bits), without LDS.
template <int CTRL>
__device__ __forceinline__ float dpp_add(float v)
{
    return v + __builtin_bit_cast(
                   float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xf,
                                                      0xf, true));
}
__device__ __forceinline__ float wave_sum(float v)
{
    v = dpp_add<0xb1>(v);                  // quads: lane ^ 1
    v = dpp_add<0x4e>(v);                  // lane ^ 2
    v = dpp_add<0x141>(v);                 // the other quad of 8 lanes (mirrored)
    v = dpp_add<0x140>(v);                 // the other 8 of 16 lanes (mirrored)
    const uint32_t a = __builtin_bit_cast(uint32_t, v);
    const auto x = __builtin_amdgcn_permlane16_swap(a, a, false, false);
    const uint32_t x0 = x[0], x1 = x[1];
    v = __builtin_bit_cast(float, x0) + __builtin_bit_cast(float, x1);
    const uint32_t b = __builtin_bit_cast(uint32_t, v);
    const auto y = __builtin_amdgcn_permlane32_swap(b, b, false, false);
    const uint32_t y0 = y[0], y1 = y[1];
    return __builtin_bit_cast(float, y0) + __builtin_bit_cast(float, y1);
}

// Sum over the TPR threads of a row; every thread gets it.
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float *red)
{
    v = wave_sum(v);
    if constexpr (TPR > 64) {
        __syncthreads();                   // the last sum's readers are done
        if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
        __syncthreads();
        v = red[0];
#pragma unroll
        for (int i = 1; i < TPR / 64; ++i) v += red[i];
    }
    return v;
}

// Mean (0 for the RMS norm) and reciprocal deviation of a row.
template <typename RowT, int TPR, int EPT>
__device__ __forceinline__ void statistics(const RowT &a, int t, const NormPlan &p, float *red,
                                           float *mean, float *r)
{
    float m = 0.f;
    if (p.layer) {
        float s = 0.f;
#pragma unroll
        for (int k = 0; k < EPT; ++k) s += a.e[k];       // zero past the row's end
        m = row_sum<TPR>(s, red) / (float)p.C;
    }
    float q = 0.f;
#pragma unroll
    for (int k = 0; k < EPT; ++k) {
        const float d = RowT::col(k, t) < p.C ? a.e[k] - m : 0.f;
        q = fmaf(d, d, q);
    }
    *mean = m;
    *r = 1.f / sqrtf(row_sum<TPR>(q, red) / (float)p.C + p.eps);
}

template <typename T, int TPR, int EPT, int V>
__global__ __launch_bounds__(TPR == 64 ? 256 : TPR) void norm_fwd_kernel(NormPlan p)
{
    using R = typename T::raw;
    using RowT = Row<T, TPR, EPT, V>;
    __shared__ float red[TPR / 64];
    const int t = threadIdx.x % TPR;
    const int64_t per = TPR == 64 ? 4 : 1;
    // TPR == 64: the waves of a workgroup leave on their own (no barrier inside)
    for (int64_t row = (int64_t)blockIdx.x * per + threadIdx.x / TPR; row < p.rows;
         row += (int64_t)gridDim.x * per) {
        const int64_t off = row * p.C;
        RowT x;
        x.load((const R *)p.x + off, t, p.C);
        float st[4] = {0.f, 0.f, 0.f, 0.f};
        if (p.h) {
            RowT h, w;
            h.load((const R *)p.h + off, t, p.C);
            float m = 0.f, r = 1.f;
            if (p.has_post) {
                statistics<RowT, TPR, EPT>(h, t, p, red, &m, &r);
                st[0] = m;
                st[1] = r;
            }
#pragma unroll
            for (int k = 0; k < EPT; ++k) h.e[k] = (h.e[k] - m) * r * p.rs;
            if (p.post) {
                w.load((const R *)p.post, t, p.C);
#pragma unroll
                for (int k = 0; k < EPT; ++k) h.e[k] *= w.e[k];
            }
            if (p.gate) {
                w.load((const R *)p.gate + (row / p.rpg) * p.C, t, p.C);
#pragma unroll
                for (int k = 0; k < EPT; ++k) h.e[k] *= w.e[k];
            }
#pragma unroll
            for (int k = 0; k < EPT; ++k)
                x.e[k] = RowT::col(k, t) < p.C ? x.e[k] + h.e[k] : 0.f;
            x.store((R *)p.y + off, t, p.C);
        }
        if (p.has_pre) {
            float m, r;
            statistics<RowT, TPR, EPT>(x, t, p, red, &m, &r);
            st[2] = m;
            st[3] = r;
            RowT w;
            w.load_or(p.pre, 0, t, p.C, 1.f);
#pragma unroll
            for (int k = 0; k < EPT; ++k) w.e[k] *= (x.e[k] - m) * r;
            w.store((R *)p.z + off, t, p.C);
        }
        if (p.stats && t == 0)
            *(float4 *)(p.stats + 4 * row) = make_float4(st[0], st[1], st[2], st[3]);
    }
}

// Each workgroup walks rows of one gate row's group after another (of one
// group only when wpg > 1) and keeps its columns' sums in registers.
template <typename T, int TPR, int EPT, int V>
__global__ __launch_bounds__(TPR == 64 ? 256 : TPR) void norm_bwd_kernel(NormPlan p)
{
    using R = typename T::raw;
    using RowT = Row<T, TPR, EPT, V>;
    constexpr int NW = TPR == 64 ? 4 : 1;  // rows in flight per workgroup
    __shared__ float red[TPR / 64];
    __shared__ float join[NW > 1 ? TPR * EPT : 1];
    const int t = threadIdx.x % TPR, wv = threadIdx.x / TPR;
    float dpost[EPT], dpre[EPT], dgate[EPT];
#pragma unroll
    for (int k = 0; k < EPT; ++k) dpost[k] = dpre[k] = 0.f;

    // the workgroup's sum of a column array, in the threads of wave 0
    // (rows are dealt to the waves in a fixed way and added in wave order)
    auto combine = [&](float *v) {
        if constexpr (NW > 1) {
            for (int w = 1; w < NW; ++w) {
                __syncthreads();
                if (wv == w) {
#pragma unroll
                    for (int k = 0; k < EPT; ++k) join[k * TPR + t] = v[k];
                }
                __syncthreads();
                if (wv == 0) {
#pragma unroll
                    for (int k = 0; k < EPT; ++k) v[k] += join[k * TPR + t];
                }
            }
        }
    };

    // (kept as stored, and the next row loaded while one is worked on: a wave
    // has only its own loads to cover their latency with)
    RawRow<T, TPR, EPT, V> wpost, wpre, wgate, rx, rh, ry, rz;
    wpost.load_or(p.post, 0, t, p.C, 1.f);
    wpre.load_or(p.pre, 0, t, p.C, 1.f);
    const int64_t g0 = p.wpg > 1 ? blockIdx.x / p.wpg : blockIdx.x;
    const int64_t gstep = p.wpg > 1 ? p.groups : gridDim.x;
    const int sub = p.wpg > 1 ? blockIdx.x % p.wpg : 0;
    const int64_t istep = (int64_t)p.wpg * NW;
    for (int64_t g = g0; g < p.groups; g += gstep) {
#pragma unroll
        for (int k = 0; k < EPT; ++k) dgate[k] = 0.f;
        wgate.load_or(p.gate, g * p.C, t, p.C, 1.f);
        float4 rst;
        auto fetch = [&](int64_t i) {
            const int64_t row = g * p.rpg + i, off = row * p.C;
            rst = *(const float4 *)(p.stats + 4 * row);
            rx.load(p.x, off, t, p.C);
            if (p.h) rh.load(p.h, off, t, p.C);
            ry.load_or(p.dy, off, t, p.C, 0.f);
            if (p.has_pre) rz.load(p.dz, off, t, p.C);
        };
        int64_t i = (int64_t)sub * NW + wv;
        if (i < p.rpg) fetch(i);
        for (; i < p.rpg; i += istep) {
            const int64_t off = (g * p.rpg + i) * p.C;
            const float4 st = rst;
            RowT y, nh, d, a;              // x then y; h then n(h); dy then dx; dz
#pragma unroll
            for (int k = 0; k < EPT; ++k) {
                y.e[k] = rx[k];
                nh.e[k] = p.h ? rh[k] : 0.f;
                d.e[k] = ry[k];
                a.e[k] = p.has_pre ? rz[k] : 0.f;
            }
            if (i + istep < p.rpg) fetch(i + istep);
            if (p.h) {
#pragma unroll
                for (int k = 0; k < EPT; ++k) {
                    if (p.has_post) nh.e[k] = (nh.e[k] - st.x) * st.y;
                    y.e[k] = fmaf(wpost[k] * wgate[k] * p.rs, nh.e[k], y.e[k]);
                }
            }
            if (p.has_pre) {
                float s1 = 0.f, s2 = 0.f;
#pragma unroll
                for (int k = 0; k < EPT; ++k) {
                    y.e[k] = RowT::col(k, t) < p.C ? (y.e[k] - st.z) * st.w : 0.f;
                    dpre[k] = fmaf(a.e[k], y.e[k], dpre[k]);
                    a.e[k] *= wpre[k];
                    s1 = fmaf(a.e[k], y.e[k], s1);
                    s2 += a.e[k];
                }
                s1 = row_sum<TPR>(s1, red) / (float)p.C;
                s2 = p.layer ? row_sum<TPR>(s2, red) / (float)p.C : 0.f;
#pragma unroll
                for (int k = 0; k < EPT; ++k)
                    d.e[k] = fmaf(a.e[k] - fmaf(y.e[k], s1, s2), st.w, d.e[k]);
            }
            d.store((R *)p.dx + off, t, p.C);
            if (p.h) {
                float s1 = 0.f, s2 = 0.f;
#pragma unroll
                for (int k = 0; k < EPT; ++k) {
                    if (RowT::col(k, t) >= p.C) d.e[k] = 0.f;
                    const float u = d.e[k] * nh.e[k] * p.rs, w = wpost[k], wg = wgate[k];
                    dgate[k] = fmaf(u, w, dgate[k]);
                    dpost[k] = fmaf(u, wg, dpost[k]);
                    d.e[k] *= w * wg * p.rs;
                    s1 = fmaf(d.e[k], nh.e[k], s1);
                    s2 += d.e[k];
                }
                if (p.has_post) {
                    s1 = row_sum<TPR>(s1, red) / (float)p.C;
                    s2 = p.layer ? row_sum<TPR>(s2, red) / (float)p.C : 0.f;
#pragma unroll
                    for (int k = 0; k < EPT; ++k)
                        d.e[k] = (d.e[k] - fmaf(nh.e[k], s1, s2)) * st.y;
                }
                d.store((R *)p.dh + off, t, p.C);
            }
        }
        if (p.gate) {
            combine(dgate);
            float *out = p.wpg > 1 ? p.part + ((int64_t)blockIdx.x * 3 + 2) * p.C
                                   : p.dgate + g * p.C;
            if (wv == 0) {
#pragma unroll
                for (int k = 0; k < EPT; ++k)
                    if (RowT::col(k, t) < p.C) out[RowT::col(k, t)] = dgate[k];
            }
        }
    }
    if (p.dpost) {
        combine(dpost);
        float *out = p.part + (int64_t)blockIdx.x * 3 * p.C;
        if (wv == 0) {
#pragma unroll
            for (int k = 0; k < EPT; ++k)
                if (RowT::col(k, t) < p.C) out[RowT::col(k, t)] = dpost[k];
        }
    }
    if (p.dpre) {
        combine(dpre);
        float *out = p.part + ((int64_t)blockIdx.x * 3 + 1) * p.C;
        if (wv == 0) {
#pragma unroll
            for (int k = 0; k < EPT; ++k)
                if (RowT::col(k, t) < p.C) out[RowT::col(k, t)] = dpre[k];
        }
    }
}

// Adds the workgroups' partial rows: blockIdx.y 0 dpost, 1 dpre, 2 + g the
// gate row g (over its wpg workgroups).  64 columns by 16 slices of rows.
__global__ __launch_bounds__(1024) void norm_join_kernel(NormPlan p)
{
    __shared__ float sum[16][64];
    const int job = blockIdx.y;
    float *out = job == 0 ? p.dpost : job == 1 ? p.dpre : p.dgate + (int64_t)(job - 2) * p.C;
    if (job < 2 ? !out : !p.dgate) return;
    const int64_t first = job < 2 ? 0 : (int64_t)(job - 2) * p.wpg;
    const int n = job < 2 ? p.nwg : p.wpg;
    const float *part = p.part + (first * 3 + (job < 2 ? job : 2)) * p.C;
    const int c = blockIdx.x * 64 + threadIdx.x % 64, sl = threadIdx.x / 64;
    float s = 0.f;
    if (c < p.C) {
#pragma unroll 8
        for (int i = sl; i < n; i += 16) s += part[(int64_t)i * 3 * p.C + c];
    }
    sum[sl][threadIdx.x % 64] = s;
    __syncthreads();
    if (sl == 0 && c < p.C) {
        for (int i = 1; i < 16; ++i) s += sum[i][threadIdx.x];
        out[c] = s;
    }
}

// Zeros to one of the sums: blockIdx.y 0 dpost, 1 dpre, 2 dgate.
__global__ __launch_bounds__(256) void norm_zero_kernel(NormPlan p)
{
    float *out = blockIdx.y == 0 ? p.dpost : blockIdx.y == 1 ? p.dpre : p.dgate;
    if (!out) return;
    const int64_t n = blockIdx.y == 2 ? p.gate_rows * p.C : p.C;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256)
        out[i] = 0.f;
}

template <typename T, int TPR, int EPT>
void forward_v(const NormPlan &p, hipStream_t s)
{
    constexpr int V = 16 / sizeof(typename T::raw);
    const int64_t per = TPR == 64 ? 4 : 1;
    const int64_t need = (p.rows + per - 1) / per;
    const dim3 grid((uint32_t)(need < kMaxTileGrid ? need : kMaxTileGrid));
    const dim3 block(TPR == 64 ? 256 : TPR);
    if (p.vec)
        launch_kernel((norm_fwd_kernel<T, TPR, EPT, V>), grid, block, 0, s, p);
    else
        launch_kernel((norm_fwd_kernel<T, TPR, EPT, 1>), grid, block, 0, s, p);
}

template <typename T, int TPR, int EPT>
void backward_v(const NormPlan &p, hipStream_t s)
{
    constexpr int V = 16 / sizeof(typename T::raw);
    const dim3 grid((uint32_t)p.nwg), block(TPR == 64 ? 256 : TPR);
    if (p.vec)
        launch_kernel((norm_bwd_kernel<T, TPR, EPT, V>), grid, block, 0, s, p);
    else
        launch_kernel((norm_bwd_kernel<T, TPR, EPT, 1>), grid, block, 0, s, p);
}

}  // namespace

// Forward: a wave by itself for rows of up to 1024, 16 elements a thread, so
// that no sum needs a barrier (1024 bfloat16: 72 us, with 256 threads of 8 98;
// 1001 float32: 26 and 33 us); longer rows do not fit a wave's registers.
void plan_norm(NormPlan *p, int es, bool aligned16)
{
    p->vec = aligned16 && (int64_t)p->C * es % 16 == 0;
    p->threads = p->C <= 1024 ? 64 : p->C <= 4096 ? 256 : 1024;
    p->ept = p->C <= 8 * p->threads ? 8 : 16;
}

// The backward keeps three sums and four rows in registers, so a thread takes
// 8 elements wherever a workgroup can hold the row with that (16 a thread:
// over 256 registers, one wave on a SIMD: 43740 x 1024 240 us, with 8 and the
// next row in flight 94).
size_t plan_norm_backward(NormPlan *p)
{
    p->threads = 64;
    while (p->threads < 1024 && 8 * p->threads < p->C) p->threads *= 2;
    p->ept = p->C <= 8 * p->threads ? 8 : 16;
    const int64_t target = p->threads <= 128 ? 1024 : (int64_t)kNormWg * 256 / p->threads;
    const int64_t per = p->threads == 64 ? 4 : 1;
    p->groups = p->gate_rows > 0 ? p->gate_rows : 1;
    p->rpg = p->rows / p->groups;
    if (p->groups >= target) {
        p->wpg = 1;
        p->nwg = (int32_t)target;
    } else {
        const int64_t most = (p->rpg + per - 1) / per;    // at least one row for each wave
        int64_t w = target / p->groups;
        if (w > most) w = most;
        p->wpg = (int32_t)(w < 1 ? 1 : w);
        p->nwg = (int32_t)(p->groups * p->wpg);
    }
    return (size_t)p->nwg * 3 * p->C * sizeof(float);
}

template <typename T>
hipError_t launch_norm_forward(const NormPlan &p, hipStream_t s)
{
    if (p.threads == 64) {
        if (p.ept == 8) forward_v<T, 64, 8>(p, s);
        else forward_v<T, 64, 16>(p, s);
    } else if (p.threads == 256) {
        if (p.ept == 8) forward_v<T, 256, 8>(p, s);
        else forward_v<T, 256, 16>(p, s);
    } else if (p.ept == 8) {
        forward_v<T, 1024, 8>(p, s);
    } else {
        forward_v<T, 1024, 16>(p, s);
    }
    return hipGetLastError();
}

template <typename T>
hipError_t launch_norm_backward(const NormPlan &p, hipStream_t s)
{
    switch (p.threads) {
    case 64: backward_v<T, 64, 8>(p, s); break;
    case 128: backward_v<T, 128, 8>(p, s); break;
    case 256: backward_v<T, 256, 8>(p, s); break;
    case 512: backward_v<T, 512, 8>(p, s); break;
    default:
        if (p.ept == 8) backward_v<T, 1024, 8>(p, s);
        else backward_v<T, 1024, 16>(p, s);
    }
    const int64_t jobs = 2 + (p.gate && p.wpg > 1 ? p.groups : 0);
    if (p.dpost || p.dpre || jobs > 2)
        launch_kernel(norm_join_kernel, dim3((uint32_t)((p.C + 63) / 64), (uint32_t)jobs),
                      dim3(1024), 0, s, p);
    return hipGetLastError();
}

hipError_t launch_norm_no_rows(const NormPlan &p, hipStream_t s)
{
    if (!p.dpost && !p.dpre && !p.dgate) return hipSuccess;
    const int64_t n = p.dgate && p.gate_rows > 1 ? p.gate_rows * p.C : p.C;
    const int64_t blocks = (n + 255) / 256;
    launch_kernel(norm_zero_kernel,
                  dim3((uint32_t)(blocks < kMaxTileGrid ? blocks : kMaxTileGrid), 3), dim3(256), 0, s,
                  p);
    return hipGetLastError();
}

#define MP3D_NORM(T)                                                     \
    template hipError_t launch_norm_forward<T>(const NormPlan &, hipStream_t); \
    template hipError_t launch_norm_backward<T>(const NormPlan &, hipStream_t);
MP3D_NORM(F32)
MP3D_NORM(F16)
MP3D_NORM(BF16)

}  // namespace mp3d
