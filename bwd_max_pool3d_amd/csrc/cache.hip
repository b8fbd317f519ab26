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
// group; k and v go in one launch.  A write of 4 x 10935 tokens of 4 heads of
// 128, bfloat16 to e4m3: 26.4 us, 5.1 TB/s; a read of 2 x 32768 of 8 heads: 64
// us, 6.3 TB/s, by stores that stay out of the caches (75 with plain ones); one
// token of 32 sequences: 4 us.
#include "cache.hpp"

namespace mp3d {

namespace {

constexpr int kRowsAhead = 4;              // rows of a thread whose loads are in flight together

typedef short s16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

// A workgroup's rows of (tokens x heads), and a thread's places among them: of
// the row that it is at, from the workgroup's first token, in each of the
// tensors that it walks.
struct Walk {
    int piece, t, h, dt, dh;
    bool idle;
    __device__ __forceinline__ Walk(int pieces, int H)
    {
        const uint32_t rows = blockDim.x / (uint32_t)pieces, r = threadIdx.x / (uint32_t)pieces;
        piece = threadIdx.x - r * pieces;
        idle = r >= rows;
        t = r / (uint32_t)H;
        h = r - t * H;
        dt = rows / (uint32_t)H;
        dh = rows - dt * H;
    }
    // true: the head went past the last, and back
    __device__ __forceinline__ bool next(int H)
    {
        t += dt;
        h += dh;
        const bool over = h >= H;
        h -= over ? H : 0;
        t += over;
        return over;
    }
};
struct Place {
    int64_t at, step, over;
    __device__ __forceinline__ Place(const Walk &w, int H, int64_t token, int64_t head)
        : at(w.t * token + w.h * head), step(w.dt * token + w.dh * head), over(step + token - H * head)
    {
    }
    __device__ __forceinline__ void next(bool past) { at += past ? over : step; }
};

// 8 elements of a row, as they are stored.
template <typename T>
struct Eight {
    using R = typename T::raw;
    static constexpr int N = sizeof(R) * 8 / 16;
    u32x4 w[N];

    // from d0 on, zero past D
    template <bool VEC>
    __device__ __forceinline__ void load(const R *p, int d0, int D)
    {
        if constexpr (VEC) {
#pragma unroll
            for (int i = 0; i < N; ++i)
                w[i] = d0 < D ? ((const u32x4 *)(p + d0))[i] : u32x4{0u, 0u, 0u, 0u};
        } else {
            struct alignas(16) {
                R e[8];
            } o;
#pragma unroll
            for (int i = 0; i < 8; ++i) o.e[i] = d0 + i < D ? p[d0 + i] : R(0);
            __builtin_memcpy(w, &o, sizeof(o));
        }
    }
    // The largest magnitude's bits, as binary32: patterns without their signs
    // are in the order of what they stand for, infinities and NaN last.
    __device__ __forceinline__ uint32_t largest() const
    {
        if constexpr (T::code == F32::code) {
            uint32_t m = 0;
#pragma unroll
            for (int i = 0; i < N; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) m = max(m, w[i][j] & 0x7fffffffu);
            return m;
        } else {
            typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
            u16x2 m = {0, 0};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t x = w[0][j] & 0x7fff7fffu;
                m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, x));
            }
            const uint16_t most = m[0] > m[1] ? m[0] : m[1];
            return __builtin_bit_cast(uint32_t, T::widen(most));
        }
    }
    // Codes under a scale.
    template <int FMT>
    __device__ __forceinline__ u32x2 codes(float scale) const
    {
        u32x2 q = {0u, 0u};
        if constexpr (T::code == F32::code) {
            float f[8];
#pragma unroll
            for (int i = 0; i < N; ++i) T::unpack(w[i], f + 4 * i);
            return codes_of<FMT>(f, scale);
        } else if constexpr (FMT == kE4M3) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                s16x2 c = {0, 0};
                const uint32_t a = w[0][2 * i], b = w[0][2 * i + 1];
                if constexpr (T::code == F16::code) {
                    c = __builtin_amdgcn_cvt_scalef32_pk_fp8_f16(c, __builtin_bit_cast(f16x2, a), scale, false);
                    c = __builtin_amdgcn_cvt_scalef32_pk_fp8_f16(c, __builtin_bit_cast(f16x2, b), scale, true);
                } else {
                    c = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(c, __builtin_bit_cast(bf16x2, a), scale, false);
                    c = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(c, __builtin_bit_cast(bf16x2, b), scale, true);
                }
                q[i] = __builtin_bit_cast(uint32_t, c);
            }
        } else {
            const uint32_t x[4] = {w[0].x, w[0].y, w[0].z, w[0].w};
            uint32_t c = 0;
            if constexpr (T::code == F16::code) {
                c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c, __builtin_bit_cast(f16x2, x[0]), scale, 0);
                c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c, __builtin_bit_cast(f16x2, x[1]), scale, 1);
                c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c, __builtin_bit_cast(f16x2, x[2]), scale, 2);
                c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c, __builtin_bit_cast(f16x2, x[3]), scale, 3);
            } else {
                c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2, x[0]), scale, 0);
                c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2, x[1]), scale, 1);
                c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2, x[2]), scale, 2);
                c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2, x[3]), scale, 3);
            }
            q.x = c;
        }
        return q;
    }
    // The same, no magnitude past lim.
    template <int FMT>
    __device__ __forceinline__ u32x2 codes_within(float scale, float lim) const
    {
        float f[8];
#pragma unroll
        for (int i = 0; i < N; ++i) T::unpack(w[i], f + 8 / N * i);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = fminf(fmaxf(f[i], -lim), lim);
        return codes_of<FMT>(f, scale);
    }
    template <int FMT>
    static __device__ __forceinline__ u32x2 codes_of(const float *f, float scale)
    {
        if constexpr (FMT == kE4M3) {
            s16x2 c[2] = {{0, 0}, {0, 0}};
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                c[i] = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(c[i], f[4 * i], f[4 * i + 1], scale, false);
                c[i] = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(c[i], f[4 * i + 2], f[4 * i + 3], scale, true);
            }
            return u32x2{__builtin_bit_cast(uint32_t, c[0]), __builtin_bit_cast(uint32_t, c[1])};
        } else {
            uint32_t c = 0;
            c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, f[0], f[1], scale, 0);
            c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, f[2], f[3], scale, 1);
            c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, f[4], f[5], scale, 2);
            c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, f[6], f[7], scale, 3);
            return u32x2{c, 0u};
        }
    }
};

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

// The largest of four adjacent lanes.
__device__ __forceinline__ uint32_t quad_max(uint32_t v)
{
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xb1, 0xf, 0xf, true));
    return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4e, 0xf, 0xf, true));
}

// What a workgroup has: `which` of k and v, a sequence's tokens [T0, T0 + Tn),
// and of these [from, to) those that are in use and have a row in the cache.
struct Tile {
    int v, T0, Tn, from, to;
    int64_t b, row;                        // row: of the first token
    __device__ __forceinline__ explicit Tile(const CachePlan &p)
    {
        const uint32_t id = blockIdx.x / (uint32_t)p.tiles, tile = blockIdx.x - id * p.tiles;
        v = id & 1;
        b = id >> 1;
        T0 = (int)tile * p.per;
        Tn = min(p.per, p.T - T0);
        row = (p.start ? p.start[b] : 0) + (int64_t)T0;
        const int used = (p.count ? p.count[b] : p.T) - min(T0, p.count ? p.count[b] : p.T);
        from = (int)min(max(-row, (int64_t)0), (int64_t)Tn);
        to = (int)min((int64_t)min(used, Tn), max(p.rows - row, (int64_t)0));
    }
};

template <typename T, int FMT, bool VEC>
__global__ __launch_bounds__(256) void cache_write_kernel(CachePlan p)
{
    using R = typename T::raw;
    constexpr float kLast = FMT == kE4M3 ? 240.f : 3.f;
    // the scale under which the code of a group's binade is past the type
    constexpr uint32_t kPast = T::code == F16::code ? (FMT == kE4M3 ? 135u : 141u)
                                                    : (FMT == kE4M3 ? 247u : 253u);
    Walk w(p.pieces, p.H);
    const Tile tile(p);
    if (w.idle || tile.from >= tile.to) return;
    const int v = tile.v;
    const R *src = (const R *)p.x[v] + tile.b * p.xs[v][0] + tile.T0 * p.xs[v][1];
    uint8_t *codes = p.codes[v] + tile.b * p.cs[v][0] + tile.row * p.cs[v][1];
    uint8_t *scales = p.scales[v] + tile.b * p.ss[v][0] + tile.row * p.ss[v][1] + w.piece / 4;
    Place x(w, p.H, p.xs[v][1], p.xs[v][2]), c(w, p.H, p.cs[v][1], p.cs[v][2]),
        s(w, p.H, p.ss[v][1], p.ss[v][2]);
    const int d0 = w.piece * 8;
    while (w.t < tile.to) {
        Eight<T> e[kRowsAhead];
        int64_t at[kRowsAhead], scale_at[kRowsAhead];
        bool there[kRowsAhead];
#pragma unroll
        for (int i = 0; i < kRowsAhead; ++i) {
            // (the four threads of a group have the same row)
            there[i] = w.t >= tile.from && w.t < tile.to;
            at[i] = c.at;
            scale_at[i] = s.at;
            if (there[i]) e[i].template load<VEC>(src + x.at, d0, p.D);
            const bool past = w.next(p.H);
            x.next(past);
            c.next(past);
            s.next(past);
        }
#pragma unroll
        for (int i = 0; i < kRowsAhead; ++i) {
            if (!there[i]) continue;
            const uint32_t byte = scale_byte<FMT>(quad_max(e[i].largest()));
            const float scale = scale_of(byte);
            u32x2 q = e[i].template codes<FMT>(scale);
            if (__builtin_expect(byte >= kPast, 0)) {
                if (byte == kPast) q = e[i].template codes_within<FMT>(scale, kLast * scale);
                else q = u32x2{0u, 0u};    // an infinity or a NaN
            }
            uint8_t *const out = codes + at[i];
            if constexpr (VEC) {
                if (d0 < p.D) {
                    if constexpr (FMT == kE4M3) *(u32x2 *)(out + d0) = q;
                    else *(uint32_t *)(out + d0 / 2) = q.x;
                }
            } else {
                const int first = code_bytes<FMT>(d0), end = code_bytes<FMT>(p.D);
                const uint32_t word[2] = {q.x, q.y};
#pragma unroll
                for (int j = 0; j < code_bytes<FMT>(8); ++j)
                    if (first + j < end) out[first + j] = (uint8_t)(word[j / 4] >> (8 * (j % 4)));
            }
            if ((w.piece & 3) == 0) scales[scale_at[i]] = (uint8_t)byte;
        }
    }
}

// N = 16 / sizeof(element) channels a thread.
template <typename T, int FMT, bool VEC>
__global__ __launch_bounds__(256) void cache_read_kernel(CachePlan p)
{
    using R = typename T::raw;
    constexpr int N = 16 / sizeof(R);
    Walk w(p.pieces, p.H);
    const Tile tile(p);
    if (w.idle) return;
    const int v = tile.v, d0 = w.piece * N;
    const uint8_t *codes = p.codes[v] + tile.b * p.cs[v][0] + tile.row * p.cs[v][1];
    const uint8_t *scales = p.scales[v] + tile.b * p.ss[v][0] + tile.row * p.ss[v][1] + d0 / kGroup;
    R *dst = (R *)p.x[v] + (tile.b * p.T + tile.T0) * p.H * (int64_t)p.D + d0;
    Place x(w, p.H, (int64_t)p.H * p.D, p.D), c(w, p.H, p.cs[v][1], p.cs[v][2]),
        s(w, p.H, p.ss[v][1], p.ss[v][2]);
    while (w.t < tile.Tn) {
        uint32_t q[kRowsAhead][2], byte[kRowsAhead];
        int64_t at[kRowsAhead];
        bool there[kRowsAhead];
#pragma unroll
        for (int i = 0; i < kRowsAhead; ++i) {
            there[i] = w.t < tile.Tn;
            at[i] = x.at;
            q[i][0] = q[i][1] = 0u;
            byte[i] = 127u;
            if (w.t >= tile.from && w.t < tile.to) {
                const uint8_t *in = codes + c.at;
                byte[i] = scales[s.at];
                if constexpr (VEC) {
                    if constexpr (FMT == kE4M3) {
                        if constexpr (N == 8) {
                            const u32x2 y = *(const u32x2 *)(in + d0);
                            q[i][0] = y.x;
                            q[i][1] = y.y;
                        } else {
                            q[i][0] = *(const uint32_t *)(in + d0);
                        }
                    } else if constexpr (N == 8) {
                        q[i][0] = *(const uint32_t *)(in + d0 / 2);
                    } else {
                        q[i][0] = *(const uint16_t *)(in + d0 / 2);
                    }
                } else {
                    const int first = code_bytes<FMT>(d0), end = code_bytes<FMT>(p.D);
#pragma unroll
                    for (int j = 0; j < code_bytes<FMT>(N); ++j)
                        if (first + j < end) q[i][j / 4] |= (uint32_t)in[first + j] << (8 * (j % 4));
                }
            }
            const bool past = w.next(p.H);
            x.next(past);
            c.next(past);
            s.next(past);
        }
#pragma unroll
        for (int i = 0; i < kRowsAhead; ++i) {
            if (!there[i]) break;
            struct alignas(16) {
                u32x4 v[sizeof(R) * 8 / 16];
            } o;
            widen8<T, FMT>(q[i][0], q[i][1], scale_of(byte[i]), o.v);
            R *const out = dst + at[i];
            if constexpr (VEC) {
                st_stream((u32x4 *)out, o.v[0]);
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

// Threads that walk a row, tokens of a workgroup.  A row has at most 256 pieces:
// a head of kCacheMaxD = 1024 channels of float32, read 4 a thread.
void plan_cache(CachePlan *p, int elem_bytes, bool read)
{
    const int per = read ? 16 / elem_bytes : 8;
    p->pieces = read ? (p->D + per - 1) / per : (p->D + kGroup - 1) / kGroup * (kGroup / per);
    p->threads = 256;
    // kRowsAhead rows a thread where that leaves two workgroups for a CU, else
    // one; whole tokens, so that no thread goes round again for the last few
    // (5 x 1330 tokens of 8 heads of 72, which did: 12.9 us)
    const int64_t rows = 256 / p->pieces, all = (int64_t)p->B * 2 * p->T * p->H;
    int64_t want = rows * kRowsAhead;
    if (all / want < 2 * device_cus()) want = rows;
    const int64_t tokens = want > p->H ? want / p->H : 1;
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
