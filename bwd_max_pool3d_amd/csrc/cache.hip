// cache.hip -- keys and values into a cache of 8 or 4 bits, and back.
//
//   write: s = least integer with max |x| <= M 2^s over a group of 32 channels
//          (M = 448 or 6), not under -126; code = the format's number nearest
//          to x / 2^s (ties to the even last bit)
//   read:  code 2^s, rounded to the storage type
// x / 2^s is exact, so a code is the right one for every x.  The scale is
// never too small for the group's largest channel, which a scale taken from
// its exponent alone would clip by up to an eighth (448 of 512) or a third
// (6 of 8).  Where code 2^s would be past the storage type's largest number
// (a group within 2^-5 of it, of e4m3) the largest code that is not is taken.
//
// Bound: HBM; for new tokens of a few sequences, the launch.  A thread has 8
// adjacent channels (4 or 8 to read, 16 bytes of them), four threads share a
// group; k and v go in one launch.
#include "cache.hpp"

namespace mp3d {

namespace {

constexpr int kRowsAhead = 4;              // rows of a thread whose loads are in flight together

// A workgroup's rows of (tokens x heads), a thread's place among them.
struct Walk {
    int piece, t, h, dt, dh;
    bool idle;
    __device__ __forceinline__ Walk(int pieces, int H)
    {
        const int rows = blockDim.x / pieces, r = threadIdx.x / pieces;
        piece = threadIdx.x - r * pieces;
        idle = r >= rows;
        t = r / H;
        h = r - t * H;
        dt = rows / H;
        dh = rows - dt * H;
    }
    __device__ __forceinline__ void next(int H)
    {
        t += dt;
        h += dh;
        if (h >= H) {
            h -= H;
            ++t;
        }
    }
};

// Elements d0 .. d0 + 7 of a row, zero past D.
template <typename T, bool VEC>
__device__ __forceinline__ void load_row8(const typename T::raw *p, int d0, int D, float *x)
{
    if constexpr (VEC) {
        constexpr int PER = 16 / sizeof(typename T::raw);
        u32x4 w[8 / PER];
#pragma unroll
        for (int i = 0; i < 8 / PER; ++i)
            w[i] = d0 < D ? ((const u32x4 *)(p + d0))[i] : u32x4{0u, 0u, 0u, 0u};
#pragma unroll
        for (int i = 0; i < 8 / PER; ++i) T::unpack(w[i], x + i * PER);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = d0 + i < D ? T::widen(p[d0 + i]) : 0.f;
    }
}

// A group's scale byte, from the bits of its largest magnitude.
template <int FMT>
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax)
{
    // 1.75 2^8 = 448, 1.5 2^2 = 6
    constexpr int32_t kBinade = FMT == kE4M3 ? 8 : 2;
    constexpr uint32_t kFraction = FMT == kE4M3 ? 0x600000u : 0x400000u;
    if (amax >= 0x7f800000u) return 255u;
    const int32_t s = (int32_t)(amax >> 23) - kBinade + ((amax & 0x7fffffu) > kFraction);
    return (uint32_t)max(s, 1);
}

template <typename T, int FMT, bool VEC>
__global__ __launch_bounds__(256) void cache_write_kernel(CachePlan p)
{
    using R = typename T::raw;
    constexpr float kTop = FMT == kE4M3 ? 448.f : 6.f, kLast = FMT == kE4M3 ? 240.f : 3.f;
    // the scale under which the code of a group's binade is past the type
    constexpr uint32_t kPast = T::code == F16::code ? (FMT == kE4M3 ? 135u : 141u)
                                                    : (FMT == kE4M3 ? 247u : 253u);
    const int64_t id = blockIdx.x / p.tiles;
    const int tile = (int)(blockIdx.x - id * p.tiles), v = (int)(id & 1);
    const int64_t b = id >> 1;
    const int T0 = tile * p.per, Tn = min(p.per, p.T - T0);
    const int64_t first = p.start ? p.start[b] : 0;
    const int used = p.count ? p.count[b] : p.T;
    const R *src = (const R *)p.x[v] + b * p.xs[v][0] + T0 * p.xs[v][1];
    uint8_t *codes = p.codes[v] + b * p.cs[v][0], *scales = p.scales[v] + b * p.ss[v][0];
    Walk w(p.pieces, p.H);
    if (w.idle) return;
    const int d0 = w.piece * 8;
    while (w.t < Tn) {
        float x[kRowsAhead][8];
        int t[kRowsAhead], h[kRowsAhead];
#pragma unroll
        for (int i = 0; i < kRowsAhead; ++i) {
            t[i] = w.t;
            h[i] = w.h;
            // (the four threads of a group have the same row)
            if (t[i] < Tn) load_row8<T, VEC>(src + t[i] * p.xs[v][1] + h[i] * p.xs[v][2], d0, p.D, x[i]);
            w.next(p.H);
        }
#pragma unroll
        for (int i = 0; i < kRowsAhead; ++i) {
            if (t[i] >= Tn) break;
            const int64_t row = first + T0 + t[i];
            uint32_t amax = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e)
                amax = max(amax, __builtin_bit_cast(uint32_t, x[i][e]) & 0x7fffffffu);
            amax = max(amax, (uint32_t)__shfl_xor((int)amax, 1));
            amax = max(amax, (uint32_t)__shfl_xor((int)amax, 2));
            if (T0 + t[i] >= used || row < 0 || row >= p.rows) continue;
            const uint32_t s = scale_byte<FMT>(amax);
            // (a group with an infinity or a NaN: codes of 0)
            const float f = s == 255u ? 0.f : __builtin_bit_cast(float, (254u - s) << 23);
            const float lim = s == kPast ? kLast : kTop;
            float y[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)
                y[e] = s == 255u ? 0.f : fminf(fmaxf(x[i][e] * f, -lim), lim);
            uint8_t *c = codes + row * p.cs[v][1] + h[i] * p.cs[v][2];
            uint32_t q[2] = {0u, 0u};
            if constexpr (FMT == kE4M3) {
                q[0] = __builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], 0, false);
                q[0] = __builtin_amdgcn_cvt_pk_fp8_f32(y[2], y[3], q[0], true);
                q[1] = __builtin_amdgcn_cvt_pk_fp8_f32(y[4], y[5], 0, false);
                q[1] = __builtin_amdgcn_cvt_pk_fp8_f32(y[6], y[7], q[1], true);
            } else {
                q[0] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, y[0], y[1], 1.f, 0);
                q[0] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q[0], y[2], y[3], 1.f, 1);
                q[0] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q[0], y[4], y[5], 1.f, 2);
                q[0] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q[0], y[6], y[7], 1.f, 3);
            }
            if constexpr (VEC) {
                if (d0 < p.D) {
                    if constexpr (FMT == kE4M3) *(u32x2 *)(c + d0) = u32x2{q[0], q[1]};
                    else *(uint32_t *)(c + d0 / 2) = q[0];
                }
            } else {
                const int at = code_bytes<FMT>(d0), end = code_bytes<FMT>(p.D);
#pragma unroll
                for (int e = 0; e < code_bytes<FMT>(8); ++e)
                    if (at + e < end) c[at + e] = (uint8_t)(q[e / 4] >> (8 * (e % 4)));
            }
            if ((w.piece & 3) == 0)
                scales[row * p.ss[v][1] + h[i] * p.ss[v][2] + w.piece / 4] = (uint8_t)s;
        }
    }
}

// N = 16 / sizeof(element) channels a thread.
template <typename T, int FMT, bool VEC>
__global__ __launch_bounds__(256) void cache_read_kernel(CachePlan p)
{
    using R = typename T::raw;
    constexpr int N = 16 / sizeof(R);
    const int64_t id = blockIdx.x / p.tiles;
    const int tile = (int)(blockIdx.x - id * p.tiles), v = (int)(id & 1);
    const int64_t b = id >> 1;
    const int T0 = tile * p.per, Tn = min(p.per, p.T - T0);
    const int64_t first = p.start ? p.start[b] : 0;
    const int used = p.count ? p.count[b] : p.T;
    const uint8_t *codes = p.codes[v] + b * p.cs[v][0], *scales = p.scales[v] + b * p.ss[v][0];
    R *dst = (R *)p.x[v] + (b * p.T + T0) * p.H * (int64_t)p.D;
    Walk w(p.pieces, p.H);
    if (w.idle) return;
    const int d0 = w.piece * N;
    while (w.t < Tn) {
        uint32_t q[kRowsAhead][2], s[kRowsAhead];
        int t[kRowsAhead], h[kRowsAhead];
#pragma unroll
        for (int i = 0; i < kRowsAhead; ++i) {
            t[i] = w.t;
            h[i] = w.h;
            q[i][0] = q[i][1] = 0u;
            s[i] = 127u;
            const int64_t row = first + T0 + t[i];
            if (t[i] < Tn && T0 + t[i] < used && row >= 0 && row < p.rows) {
                const uint8_t *c = codes + row * p.cs[v][1] + h[i] * p.cs[v][2];
                s[i] = scales[row * p.ss[v][1] + h[i] * p.ss[v][2] + d0 / kGroup];
                if constexpr (VEC) {
                    if constexpr (FMT == kE4M3) {
                        if constexpr (N == 8) {
                            const u32x2 x = *(const u32x2 *)(c + d0);
                            q[i][0] = x.x;
                            q[i][1] = x.y;
                        } else {
                            q[i][0] = *(const uint32_t *)(c + d0);
                        }
                    } else if constexpr (N == 8) {
                        q[i][0] = *(const uint32_t *)(c + d0 / 2);
                    } else {
                        q[i][0] = *(const uint16_t *)(c + d0 / 2);
                    }
                } else {
                    const int at = code_bytes<FMT>(d0), end = code_bytes<FMT>(p.D);
#pragma unroll
                    for (int e = 0; e < code_bytes<FMT>(N); ++e)
                        if (at + e < end) q[i][e / 4] |= (uint32_t)c[at + e] << (8 * (e % 4));
                }
            }
            w.next(p.H);
        }
#pragma unroll
        for (int i = 0; i < kRowsAhead; ++i) {
            if (t[i] >= Tn) break;
            struct alignas(16) {
                u32x4 v[sizeof(R) * 8 / 16];
            } o;
            widen8<T, FMT>(q[i][0], q[i][1], scale_of(s[i]), o.v);
            R *out = dst + ((int64_t)t[i] * p.H + h[i]) * p.D + d0;
            if constexpr (VEC) {
                *(u32x4 *)out = o.v[0];
            } else {
                R e[8];
                __builtin_memcpy(e, &o, sizeof(e));
#pragma unroll
                for (int j = 0; j < N; ++j)
                    if (d0 + j < p.D) out[j] = e[j];
            }
        }
    }
}

template <typename T, int FMT>
hipError_t run(const CachePlan &p, bool read, hipStream_t s)
{
    const dim3 grid((uint32_t)(p.tiles * p.B * 2)), block(p.threads);
    if (read && p.vec) launch_kernel((cache_read_kernel<T, FMT, true>), grid, block, 0, s, p);
    else if (read) launch_kernel((cache_read_kernel<T, FMT, false>), grid, block, 0, s, p);
    else if (p.vec) launch_kernel((cache_write_kernel<T, FMT, true>), grid, block, 0, s, p);
    else launch_kernel((cache_write_kernel<T, FMT, false>), grid, block, 0, s, p);
    return hipGetLastError();
}

}  // namespace

// Threads that walk a row, tokens of a workgroup.  Rows of up to 256 pieces
// share a workgroup; longer ones (heads over 2048 channels) are refused.
void plan_cache(CachePlan *p, int elem_bytes, bool read)
{
    const int per = read ? 16 / elem_bytes : 8;
    p->pieces = read ? (p->D + per - 1) / per : (p->D + kGroup - 1) / kGroup * (kGroup / per);
    p->threads = 256;
    const int64_t rows = 256 / p->pieces;
    // kRowsAhead rows a thread where that still fills the card, else one
    const int64_t all = (int64_t)p->B * 2 * p->T * p->H;
    int64_t want = rows * kRowsAhead;
    if (all / want < 8 * device_cus()) want = rows;
    int64_t tokens = (want + p->H - 1) / p->H;
    p->per = (int32_t)(tokens < p->T ? tokens : p->T);
    p->tiles = (p->T + p->per - 1) / p->per;
}

template <typename T>
hipError_t launch_cache(const CachePlan &p, bool read, hipStream_t s)
{
    return p.format == kE4M3 ? run<T, kE4M3>(p, read, s) : run<T, kE2M1>(p, read, s);
}

template hipError_t launch_cache<F32>(const CachePlan &, bool, hipStream_t);
template hipError_t launch_cache<F16>(const CachePlan &, bool, hipStream_t);
template hipError_t launch_cache<BF16>(const CachePlan &, bool, hipStream_t);

}  // namespace mp3d
