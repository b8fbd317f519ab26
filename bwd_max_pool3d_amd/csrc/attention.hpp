// attention.hpp -- what the attention kernels share: their arguments, the
// keys a query sees, tiles in LDS and the matrix fragments read from them.
//
// Fragments.  All products run on 32x32 matrix instructions, 16 deep.  A
// fragment is 8 elements of one lane; lane l holds row (or column) l % 32
// and the half l / 32 of the depth.  The 32x32 result lies with column
// l % 32 in lane l and rows 8 (r / 4) + 4 (l / 32) + r % 4 in its registers
// r = 0 .. 15.  So the scores are formed transposed to what they feed: a
// result's registers 8c .. 8c + 7, rounded to the storage type, are the
// second operand of the next product over the rows 16c .. 16c + 15, taken
// in the order {0-3, 8-11} (lower half) and {4-7, 12-15} (upper half), with
// no exchange between lanes.  The first operand of that product is read
// from LDS in the same order: for 16-bit types by the transposing LDS read,
// which hands each of 16 lanes one column of a 4 x 16 block.
#pragma once

#include "dtype.hpp"
#include "tokens.hpp"

namespace mp3d {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kNegInf = -__builtin_huge_valf();

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int i32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

// 8 elements of a lane: 16 bytes, or 32 for float32
template <typename T>
struct Frag {
    static constexpr int NV = sizeof(typename T::raw) * 8 / 16;
    u32x4 w[NV];
    __device__ __forceinline__ void zero()
    {
#pragma unroll
        for (int i = 0; i < NV; ++i) w[i] = u32x4{0u, 0u, 0u, 0u};
    }
};

template <typename T>
__device__ __forceinline__ f32x16 mma(const Frag<T> &a, const Frag<T> &b, f32x16 c)
{
    if constexpr (T::code == BF16::code) {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a.w[0]),
                                                       __builtin_bit_cast(bf16x8, b.w[0]), c, 0, 0,
                                                       0);
    } else if constexpr (T::code == F16::code) {
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a.w[0]),
                                                      __builtin_bit_cast(f16x8, b.w[0]), c, 0, 0,
                                                      0);
    } else {
        // eight products 2 deep: the halves' elements i meet
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const u32x4 x = a.w[i / 4], y = b.w[i / 4];
            const uint32_t xe[4] = {x.x, x.y, x.z, x.w}, ye[4] = {y.x, y.y, y.z, y.w};
            c = __builtin_amdgcn_mfma_f32_32x32x2f32(__builtin_bit_cast(float, xe[i % 4]),
                                                     __builtin_bit_cast(float, ye[i % 4]), c, 0, 0,
                                                     0);
        }
        return c;
    }
}

// c plus a step's 32 products, a0 b0 the first 16.  float32, whose results
// show it: the step is summed by itself and then added, or a sum over
// thousands would be rounded every two products (gradients over 2 x 4000
// queries: 1.5e-6 off that way).  In 16-bit types the operands' own rounding
// is a thousand times that.
template <typename T>
__device__ __forceinline__ f32x16 add_step(const Frag<T> &a0, const Frag<T> &b0, const Frag<T> &a1,
                                           const Frag<T> &b1, f32x16 c)
{
    if constexpr (T::code == F32::code) return c + mma<T>(a1, b1, mma<T>(a0, b0, f32x16(0.f)));
    else return mma<T>(a1, b1, mma<T>(a0, b0, c));
}

// Registers 8c .. 8c + 7 of a result as an operand.
template <typename T>
__device__ __forceinline__ Frag<T> pack8(const f32x16 &s, int c)
{
    struct alignas(16) {
        typename T::raw e[8];
    } o;
#pragma unroll
    for (int i = 0; i < 8; ++i) o.e[i] = T::narrow(s[8 * c + i]);
    return __builtin_bit_cast(Frag<T>, o);
}

// The order in which a stretch of reads from LDS and matrix products is
// issued, up to issued(): `ahead` reads, then a product and `per` reads at a
// time.  Left to itself the compiler reads each fragment just before its use,
// and a wave waits for LDS 30 times a tile; read all at once, the fragments
// take registers that are not there.  float32 is left to the compiler (its
// fragments are several reads and products each).
template <typename T, int AHEAD>
__device__ __forceinline__ void reads_ahead()
{
    if constexpr (sizeof(typename T::raw) == 2) __builtin_amdgcn_sched_group_barrier(0x100, AHEAD, 0);
}
template <typename T, int PRODUCTS, int PER>
__device__ __forceinline__ void products_and_reads()
{
    if constexpr (sizeof(typename T::raw) == 2) {
#pragma unroll
        for (int i = 0; i < PRODUCTS; ++i) {
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
            if constexpr (PER > 0) __builtin_amdgcn_sched_group_barrier(0x100, PER, 0);
        }
    }
}
template <typename T>
__device__ __forceinline__ void issued()
{
    if constexpr (sizeof(typename T::raw) == 2) __builtin_amdgcn_sched_barrier(0);
}

// Row of a result's register r (see above).
__device__ __forceinline__ constexpr int acc_row(int r, int half)
{
    return 8 * (r / 4) + 4 * half + r % 4;
}

// Channels d of a result's column (one row of a tensor in memory, rows
// starting at multiples of 16 bytes times the row's number), times f.
template <typename T, int ND>
__device__ __forceinline__ void store_cols(typename T::raw *out, const f32x16 *o, float f, int D,
                                           int half)
{
    using R = typename T::raw;
    const bool wide = D % 4 == 0;          // rows then start at multiples of 4 elements
#pragma unroll
    for (int d = 0; d < ND; ++d)
#pragma unroll
        for (int r = 0; r < 16; r += 4) {
            const int e = d * 32 + acc_row(r, half);
            struct alignas(4 * sizeof(R)) {
                R v[4];
            } w;
#pragma unroll
            for (int x = 0; x < 4; ++x) w.v[x] = T::narrow(o[d][r + x] * f);
            if (wide) {
                if (e < D) *(decltype(w) *)(out + e) = w;
            } else {
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    if (e + x < D) out[e + x] = w.v[x];
            }
        }
}

// The values of a result's rows from an array of 32 in LDS (16-byte aligned).
template <typename E>
__device__ __forceinline__ auto acc_rows(const E *v, int half)
{
    typedef E e4 __attribute__((ext_vector_type(4)));
    typedef E e16 __attribute__((ext_vector_type(16)));
    e16 o;
#pragma unroll
    for (int r = 0; r < 16; r += 4) {
        const e4 x = *(const e4 *)(v + acc_row(r, half));
#pragma unroll
        for (int i = 0; i < 4; ++i) o[r + i] = x[i];
    }
    return o;
}

// The same from an array of 32 pairs.
template <typename E, typename E16>
__device__ __forceinline__ void acc_pairs(const E *v, int half, E16 *a, E16 *b)
{
    typedef E e4 __attribute__((ext_vector_type(4)));
#pragma unroll
    for (int r = 0; r < 16; r += 4)
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
            const e4 x = *(const e4 *)(v + 2 * (acc_row(r, half) + i));
            (*a)[r + i] = x[0];
            (*b)[r + i] = x[1];
            (*a)[r + i + 1] = x[2];
            (*b)[r + i + 1] = x[3];
        }
}

// The larger, and the sum, of the two halves' values.
__device__ __forceinline__ float halves_max(float v)
{
    const auto x = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, v),
                                                    __builtin_bit_cast(uint32_t, v), false, false);
    const uint32_t a = x[0], b = x[1];
    return fmaxf(__builtin_bit_cast(float, a), __builtin_bit_cast(float, b));
}
__device__ __forceinline__ float halves_sum(float v)
{
    const auto x = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, v),
                                                    __builtin_bit_cast(uint32_t, v), false, false);
    const uint32_t a = x[0], b = x[1];
    return __builtin_bit_cast(float, a) + __builtin_bit_cast(float, b);
}

// --- tiles in LDS: rows of DP elements in chunks of 8, the chunks of a row
// swapped by the row's number.  LDS has 64 banks of 4 bytes, and serves 16
// lanes of 16 bytes, or 32 of 8, at once.  So that they spread over all
// banks, the same chunk of 16 rows (row fragments) must take 16 places of
// 256 bytes, and so must 4 chunks of 4 rows (column fragments).  A row of
// 128 16-bit elements is 256 bytes, one of 64 half of that.
template <typename R, int DP>
__device__ __forceinline__ int tile_swap(int row)
{
    if constexpr (sizeof(R) == 2 && DP == 128) return ((row & 3) << 2) | ((row >> 2) & 3);
    if constexpr (sizeof(R) == 2) return ((row & 2) << 1) | ((row >> 2) & 3);
    return row & 7;
}

template <typename R, int DP>
__device__ __forceinline__ int tile_at(int row, int chunk)
{
    return row * DP + ((chunk ^ tile_swap<R, DP>(row)) << 3);
}

// Elements d0 .. d0 + 7 (d0 a multiple of 8) of a row.
template <typename T, int DP>
__device__ __forceinline__ Frag<T> row_frag(const typename T::raw *tile, int row, int d0)
{
    const u32x4 *p = (const u32x4 *)(tile + tile_at<typename T::raw, DP>(row, d0 >> 3));
    Frag<T> f;
#pragma unroll
    for (int i = 0; i < Frag<T>::NV; ++i) f.w[i] = p[i];
    return f;
}

// Column l % 32 of the 32 columns from d0, rows 16c .. 16c + 15 in the
// operand order above.
template <typename T, int DP>
__device__ __forceinline__ Frag<T> col_frag(const typename T::raw *tile, int c, int d0, int l)
{
    const int half = l >> 5;
    Frag<T> f;
    if constexpr (sizeof(typename T::raw) == 2) {
        const int col = d0 + (l & 16) + (l & 3) * 4;
        const int row = 16 * c + 4 * half + ((l & 15) >> 2);
        typedef __attribute__((address_space(3))) s16x4 lds_t;
        struct alignas(16) {
            s16x4 v[2];
        } o;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const typename T::raw *p =
                tile + tile_at<typename T::raw, DP>(row + 8 * k, col >> 3) + (col & 7);
            o.v[k] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_t *)p);
        }
        f = __builtin_bit_cast(Frag<T>, o);
    } else {
        const int col = d0 + (l & 31);
        struct alignas(16) {
            float e[8];
        } o;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int row = 16 * c + 4 * half + (i < 4 ? i : i + 4);
            o.e[i] = tile[tile_at<typename T::raw, DP>(row, col >> 3) + (col & 7)];
        }
        f = __builtin_bit_cast(Frag<T>, o);
    }
    return f;
}

// Infinities and NaN set to 0; true if there was one.
template <typename T>
__device__ __forceinline__ bool drop_nonfinite16(u32x4 &v)
{
    bool bad = false;
    uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if constexpr (T::code == F32::code) {
            if ((w[j] & 0x7f800000u) == 0x7f800000u) {
                bad = true;
                w[j] = 0;
            }
        } else {
            constexpr uint32_t e = T::code == F16::code ? 0x7c00u : 0x7f80u;
            if ((w[j] & e) == e) {
                bad = true;
                w[j] &= 0xffff0000u;
            }
            if ((w[j] & (e << 16)) == (e << 16)) {
                bad = true;
                w[j] &= 0xffffu;
            }
        }
    }
    v = u32x4{w[0], w[1], w[2], w[3]};
    return bad;
}

template <typename T>
__device__ __forceinline__ bool drop_nonfinite(Frag<T> &f)
{
    bool bad = false;
#pragma unroll
    for (int i = 0; i < Frag<T>::NV; ++i) bad |= drop_nonfinite16<T>(f.w[i]);
    return bad;
}

// A value that the compiler may not reason about: what depends on it stays
// inside a rarely taken branch of a loop (computed ahead of the loop, it
// would cost the common path its registers).
__device__ __forceinline__ int opaque(int v)
{
    asm volatile("" : "+v"(v));
    return v;
}

// Elements d0 .. d0 + 7 of a row of D in memory, zero past D.  vec: rows
// start at multiples of 16 bytes.
template <typename T>
__device__ __forceinline__ Frag<T> load8(const typename T::raw *p, int d0, int D, bool vec)
{
    Frag<T> f;
    f.zero();
    if (vec && d0 + 8 <= D) {
#pragma unroll
        for (int i = 0; i < Frag<T>::NV; ++i) f.w[i] = ((const u32x4 *)(p + d0))[i];
    } else if (d0 < D) {
        struct alignas(16) {
            typename T::raw e[8];
        } o = __builtin_bit_cast(decltype(o), f);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (d0 + i < D) o.e[i] = p[d0 + i];
        f = __builtin_bit_cast(Frag<T>, o);
    }
    return f;
}

// Waits for loaded fragments.  Those that live through a loop must be there
// before it: the compiler would otherwise wait for them in it, every time
// round, and with them for every later load.
template <typename T, int N>
__device__ __forceinline__ void arrived(Frag<T> (&f)[N])
{
#pragma unroll
    for (int c = 0; c < N; ++c)
#pragma unroll
        for (int i = 0; i < Frag<T>::NV; ++i) asm volatile("" : "+v"(f[c].w[i]));
}
__device__ __forceinline__ void arrived(float &v) { asm volatile("" : "+v"(v)); }

// A tile of ROWS rows on its way from memory to LDS, spread over NT threads.
template <typename T, int DP, int ROWS, int NT>
struct TileRegs {
    using R = typename T::raw;
    static constexpr int N = ROWS * (DP / 8) / NT;
    static_assert(N * NT == ROWS * (DP / 8), "whole chunks per thread");
    Frag<T> f[N];

    // rows r0 .. r0 + ROWS - 1 of base; rows outside [lo, hi) are zero and
    // are not read
    __device__ __forceinline__ void load(const R *base, int64_t stride, int r0, int lo, int hi,
                                         int D, bool vec, int t)
    {
        if (vec && D == DP && lo <= r0 && r0 + ROWS <= hi) {
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const int id = t + NT * j;
                const R *p = base + (int64_t)(r0 + id / (DP / 8)) * stride + (id % (DP / 8)) * 8;
#pragma unroll
                for (int i = 0; i < Frag<T>::NV; ++i) f[j].w[i] = ((const u32x4 *)p)[i];
            }
            return;
        }
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const int id = t + NT * j, row = r0 + id / (DP / 8);
            if (row >= lo && row < hi)
                f[j] = load8<T>(base + (int64_t)row * stride, (id % (DP / 8)) * 8, D, vec);
            else
                f[j].zero();
        }
    }
    __device__ __forceinline__ void store(R *tile, int t) const
    {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const int id = t + NT * j;
            u32x4 *p = (u32x4 *)(tile + tile_at<typename T::raw, DP>(id / (DP / 8), id % (DP / 8)));
#pragma unroll
            for (int i = 0; i < Frag<T>::NV; ++i) p[i] = f[j].w[i];
        }
    }
    __device__ __forceinline__ bool drop()
    {
        bool bad = false;
#pragma unroll
        for (int j = 0; j < N; ++j) bad |= drop_nonfinite<T>(f[j]);
        return bad;
    }
    // the same, with the rows that held one marked
    __device__ __forceinline__ bool drop(int *row_mark, int mark, int t)
    {
        bool bad = false;
#pragma unroll
        for (int j = 0; j < N; ++j)
            if (drop_nonfinite<T>(f[j])) {
                row_mark[(t + NT * j) / (DP / 8)] = mark;
                bad = true;
            }
        return bad;
    }
};

// 16 (or 4) bytes a lane from p + off to LDS, lane after lane from address
// `lds`; p and lds are the same in every lane.  Written as instructions with
// no result: through the builtin the compiler knows that LDS is written, and
// waits for all loads before each transposing read, whichever tile that is
// from.  The kernels count these loads themselves (wait_loads).  (m0 is the
// compiler's own only right around an instruction that takes it; these
// kernels have no other.)
__device__ __forceinline__ uint32_t lds_address(const void *p)
{
    typedef const __attribute__((address_space(3))) void lds_t;
    return __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(lds_t *)p);
}
__device__ __forceinline__ void direct16(const void *p, uint32_t off, uint32_t lds)
{
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
                 :
                 : "s"(lds), "v"(off), "s"(p)
                 : "memory");
}
__device__ __forceinline__ void direct4(const void *p, uint32_t off, uint32_t lds)
{
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, %2"
                 :
                 : "s"(lds), "v"(off), "s"(p)
                 : "memory");
}

// (The kernels' DU: channels that products are formed over, 32 to 128.  Tiles
// in LDS have DP = 64 or 128, with zeros past a tensor's D.  4 x 1330 tokens of
// 8 heads of 72, forward and backward: bfloat16 43 and 219 us, over all 128 53
// and 262; float32 308 and 1134, over 128 412 and 1572.)
//
// The same tile straight from memory to LDS, 16 bytes a lane, with nothing
// in registers meanwhile.  A wave's lanes fill 1 KiB of LDS in order, so the
// swap of the chunks is made on the memory side.  Rows outside [lo, hi) are
// read from the nearest row inside, and set to zero (with what else is to be
// dropped) in LDS once they are there, by the lanes that loaded them.
template <typename T, int DP, int ROWS, int NT>
struct TileDirect {
    using R = typename T::raw;
    static constexpr int PER = 16 / sizeof(R);             // elements of a lane's 16 bytes
    static constexpr int UNITS = DP / PER;                 // of a row
    static constexpr int STEP = NT / UNITS;                // rows of one round over the threads
    static constexpr int N = ROWS / STEP;
    static_assert(N * STEP == ROWS && (STEP & (STEP - 1)) == 0, "whole rounds over the threads");
    uint32_t row, ch;                                      // bytes from the round's first row
    int64_t step;                                          // bytes from round to round
    uint32_t end;                                          // bytes of a row's channels

    __device__ __forceinline__ void init(int t, int64_t stride, int D)
    {
        const int r = t / UNITS, u = t % UNITS, c = (u * PER / 8) ^ tile_swap<R, DP>(r);
        row = (uint32_t)(r * stride) * (uint32_t)sizeof(R);
        ch = (c * 8 + (u * PER) % 8) * (uint32_t)sizeof(R);
        step = STEP * stride * (int64_t)sizeof(R);
        end = D * (uint32_t)sizeof(R);
    }
    // The lane's channels in round j.  (The swap of a sum of rows without
    // common bits is the exclusive or of their swaps; with 16 rows or more a
    // round, all rounds swap alike.)
    __device__ __forceinline__ uint32_t channels(int j) const
    {
        return ch ^ (tile_swap<R, DP>(j * STEP) * 8 * (uint32_t)sizeof(R));
    }
    // A tile whose rows are all there, the first at p, and with ALL all DP
    // channels.  `lds`: the wave's first place in the tile.  Every wave waits for its loads before
    // the barrier that hands the tile over.  (What is left to do a tile is
    // little: a wave alone on its SIMD takes a scalar instruction every four
    // cycles, and a taken branch costs tens.)
    template <bool ALL>
    __device__ __forceinline__ void load(const R *p, uint32_t lds) const
    {
#pragma unroll
        for (int j = 0; j < N; ++j)
            if (ALL || channels(j) < end)  // (true in some lane: a load that counts)
                direct16((const char *)p + j * step, row + channels(j), lds + j * NT * 16);
    }
    // Any tile, from row r0 of base.
    __device__ __forceinline__ void load_edge(const R *base, int64_t stride, int r0, int lo, int hi,
                                              uint32_t lds) const
    {
        const int t = opaque(threadIdx.x % NT) / UNITS;
#pragma unroll
        for (int j = 0; j < N; ++j) {
            // (clamping keeps the order: no lane is before the first)
            const int first = r0 + j * STEP, at = min(max(first, lo), hi - 1);
            const int r = min(max(first + t, lo), hi - 1) - at;
            if (channels(j) < end)
                direct16(base + at * stride, (uint32_t)(r * stride) * (uint32_t)sizeof(R) + channels(j),
                         lds + j * NT * 16);
        }
    }
    // Rows outside [lo, hi) of a tile that has arrived to zero; with `drop`
    // infinities and NaN too (true if there was one; its row marked).
    __device__ __forceinline__ bool scrub(R *tile, int r0, int lo, int hi, bool drop,
                                          int *row_mark, int mark) const
    {
        bool bad = false;
        const int t = opaque(threadIdx.x % NT);
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const int id = j * NT + t, at = r0 + id / UNITS;
            u32x4 *p = (u32x4 *)(tile + id * PER);
            if (at < lo || at >= hi) {
                *p = u32x4{0u, 0u, 0u, 0u};
            } else if (drop) {
                u32x4 v = *p;
                if (drop_nonfinite16<T>(v)) {
                    *p = v;
                    if (row_mark) row_mark[id / UNITS] = mark;
                    bad = true;
                }
            }
        }
        return bad;
    }
    // Can tiles be loaded this way at all?  Whole chunks, and a row's offset
    // within 31 bits.
    __device__ static __forceinline__ bool usable(bool vec, int64_t stride, int D)
    {
        return vec && D % 8 == 0 && stride < (1 << 24);
    }
    // Loads that a wave has issued for a tile.
    static constexpr int LOADS = N;
};

// --- stages: LDS holds several tiles, filled all but two steps ahead of
// their use.  Steps go in pairs, with one wait and one barrier a pair.  A
// wave's loads return in order: when no more are outstanding than it issued
// for the later steps, the next pair is there.  (Its own waits, and a barrier
// that adds none: __syncthreads would wait for every load.)  Six stages, or
// four where six would not leave room for a second workgroup.
template <typename T, int DP>
constexpr int stages() { return sizeof(typename T::raw) * DP <= 128 ? 6 : 4; }

template <int OUTSTANDING>
__device__ __forceinline__ void wait_loads(bool later)
{
    if (later) asm volatile("s_waitcnt vmcnt(%0)" ::"n"(OUTSTANDING) : "memory");
    else asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
}

// After loads through registers in a loop: none is waited for later on.
__device__ __forceinline__ void wait_all() { __builtin_amdgcn_s_waitcnt(0x0f70); }  // vmcnt(0)

__device__ __forceinline__ void hand_over()
{
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// The reads from a part of LDS are done: loads may write there again.
__device__ __forceinline__ void reads_done() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

// A value that is the same in every lane, as a scalar.
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// A value in a vector or a scalar register that has been loaded, here and
// not where it is used (see arrived).
__device__ __forceinline__ void arrived(int &v) { asm volatile("" : "+v"(v)); }
__device__ __forceinline__ void arrived_scalar(float &v) { asm volatile("" : "+s"(v)); }

// A value that is the same in every lane, read through the scalar cache (a
// vector load would have to wait for the stages before it).
template <typename E>
__device__ __forceinline__ E uniform_load(const E *p)
{
    typedef const __attribute__((address_space(4))) E constant_t;
    return *(constant_t *)(uintptr_t)p;
}

// --- infinities and NaN in masked places
//
// 0 * inf is NaN, so a masked weight of 0 does not keep a key's value out of
// a matrix product.  Keys that no query of the workgroup sees are staged as
// zeros.  Where some see a key and others do not, its infinities and NaN are
// staged as zeros too, and added afterwards to the results of those who do
// see it: a positive weight times such a value is that value, so the weight
// itself is not needed.  In dq and dk nothing is added: there a weight's
// gradient is NaN with it already.  (A key that is not finite gives a query
// the score -infinity, and weight 0, or makes its lse NaN: dq sets the
// score of such a key to -infinity, which gives both.  A query that is not
// finite has no finite score, so its lse is NaN, or -infinity.)
//
// --- which block of which head a workgroup takes.  Heads go to the XCDs in
// contiguous runs (those that share keys share an L2).  Within an XCD the
// longest blocks of all its heads come first; every second round over the
// CUs runs backwards, so that where two rounds fit at once a CU gets a long
// and a short one.
struct Block {
    int head, no;                          // no: in order of falling length
};

__device__ __forceinline__ Block block_of(uint32_t id, int heads, int blocks)
{
    constexpr int kCus = 32;               // of an XCD
    const bool split = heads % 8 == 0;
    const int per = split ? heads / 8 : heads, round = split ? kCus : 8 * kCus;
    const int total = per * blocks;
    int j = split ? id / 8 : id;
    const int c = j / round;
    if (c & 1) {
        const int first = c * round;
        j = first + min(round, total - first) - 1 - (j - first);
    }
    return {(split ? (int)(id % 8) * per : 0) + j % per, j / per};
}

// --- the keys a query sees
struct Span {
    int lo, hi;                            // [lo, hi) within [0, Tk); {0, 0}: none
};

__device__ __forceinline__ Span row_span(const AttnArgs &a, int b, int i)
{
    int L = a.Tk;
    if (a.kv_len) L = min(max(a.kv_len[b], 0), a.Tk);
    const int p = i + L - a.Tq;
    int lo = 0, hi = L, pre = 0;
    if (a.docs) {
        const int32_t *o = a.docs + (int64_t)b * (a.ndocs + 1);
        if (p < o[0] || p >= o[a.ndocs]) return {0, 0};
        int d = 0, e = a.ndocs;            // o[d] <= p < o[e]
        while (e - d > 1) {
            const int m = (d + e) >> 1;
            if (o[m] <= p) d = m;
            else e = m;
        }
        lo = max(o[d], 0);
        hi = min(o[d + 1], L);
        if (a.prefix) pre = a.prefix[(int64_t)b * a.ndocs + d];
    } else if (a.prefix) {
        pre = a.prefix[b];
    }
    if (a.causal) hi = min(hi, max(p + 1, min(lo, a.Tk) + min(max(pre, 0), a.Tk)));
    return hi > lo ? Span{lo, hi} : Span{0, 0};
}

// --- scores: from the accumulated products q.k to exponents of 2.  The
// scale is left to the exponent's own multiply-add (exponent = score * mul -
// maximum) and divided out of the cap and of the bias' slopes, unless it is
// not positive: the largest score would not have the largest exponent.  With a
// cap it is left only where the cap in these units and its reciprocal (its
// sixth power, in cap_scores) are well within binary32; else the scores are
// multiplied by the scale, or for a small cap by scale / cap.
struct Scores {
    bool multiply;                         // by `scale` first
    float scale, mul;
    float slope;                           // factor of the bias' slopes
    float cap, per_cap;                    // the cap and its reciprocal, in these units
};

__device__ __forceinline__ Scores scores(const AttnArgs &a)
{
    if (a.cap > 0.f) {
        const float per = a.scale / a.cap;
        if (a.scale > 1e-6f && a.scale < 1e6f && per < 1e6f)
            return {false, a.scale, a.scale * kLog2e, 1.f / a.scale, a.cap / a.scale, per};
        if (a.cap < 1e-3f)                 // (past 1e38 a score is 0 or beyond the cap)
            return {true, fminf(fmaxf(per, -1e38f), 1e38f), a.cap * kLog2e, 1.f / a.cap, 1.f, 1.f};
        return {true, a.scale, kLog2e, 1.f, a.cap, 1.f / a.cap};
    }
    const bool multiply = !(a.scale > 1e-30f);
    const float unit = multiply ? 1.f : a.scale;
    return {multiply, a.scale, unit * kLog2e, 1.f / unit, 0.f, 0.f};
}

// (a branch: as a choice between two results it would be in every tile)
__device__ __forceinline__ void multiply_scores(f32x16 &s, const Scores &sc)
{
    if (!sc.multiply) return;
    asm volatile("");
    s *= sc.scale;
}

// --- distances of positions: the differences of 32 rows' and 32 columns'
// positions, as a matrix product.  A position is the sum of its four bytes
// p3 2^24 + p2 2^16 + p1 2^8 + p0, with its sign, each exact in bfloat16, so
//   p - k = (p3, p2, p1, p0, 1, 1, 1, 1) . (1, 1, 1, 1, -k3, -k2, -k1, -k0),
// eight products that one matrix instruction forms for all pairs.  Below 2^24
// (p3 and k3 are 0) the terms of a distance under 2^24 have no partial sum
// past it, in whatever order they are added: no error.  Else a first
// instruction forms the difference of the upper halves, 17 bits wide, and a
// second adds the lower ones: exact below 2^23, and the distance of any two
// int32 within a few units of 2^-24 of it.  The vector units, which bound these
// kernels at 64 channels, are left with one operation a score and axis where
// they had two, and LDS with one read where it had four.
constexpr uint32_t kOnes = 0x3f803f80u;    // two
constexpr uint32_t kUpper = 0x7fff0000u;   // p3's place, without its sign

// (p3 above p2, p1 above p0)
__device__ __forceinline__ u32x2 position_parts(int32_t p)
{
    const uint32_t m = p < 0 ? 0u - (uint32_t)p : (uint32_t)p;
    const uint32_t sign = (uint32_t)(p >> 31) & 0x80008000u;
    auto part = [](uint32_t byte, float unit) {
        return __builtin_bit_cast(uint32_t, (float)byte * unit);
    };
    return u32x2{(part(m >> 24, 16777216.f) | part(m >> 16 & 0xffu, 65536.f) >> 16) ^ sign,
                 (part(m >> 8 & 0xffu, 256.f) | part(m & 0xffu, 1.f) >> 16) ^ sign};
}

// The columns' operand: lanes 0 .. 31 ones, 32 .. 63 the parts, negated.
__device__ __forceinline__ u32x2 position_cols(u32x2 parts, int half)
{
    u32x2 c = half ? parts ^ 0x80008000u : u32x2{kOnes, kOnes};
    asm volatile("" : "+v"(c));
    return c;
}

__device__ __forceinline__ bool is_far_position(int32_t p)
{
    return (uint32_t)p + (1u << 24) - 1u > (2u << 24) - 2u;
}
__device__ __forceinline__ bool is_far_position(u32x2 parts) { return parts.x & kUpper; }

// The rows' is read from LDS: `lane` points to the lane's parts, for lanes
// 32 .. 63 to ones.  FAR: some position that the workgroup walks is 2^24 or
// more.
template <bool FAR>
__device__ __forceinline__ f32x16 differences(const u32x2 *lane, u32x2 cols)
{
    auto product = [&](u32x2 rows, f32x16 c) {
        return __builtin_amdgcn_mfma_f32_32x32x8bf16_1k(__builtin_bit_cast(s16x4, rows),
                                                        __builtin_bit_cast(s16x4, cols), c, 0, 0,
                                                        0);
    };
    const u32x2 rows = *lane;
    if constexpr (FAR)
        return product(u32x2{0u, rows.y}, product(u32x2{rows.x, 0u}, f32x16(0.f)));
    else return product(rows, f32x16(0.f));
}

// Minus slope times distance on each axis, from scores s: `rows` the tile's
// parts on the first axis, those of an axis `step` after it.  axes negative:
// the wave may meet a far position.  (Two branches without an else, on a
// number that is there anyway: as one with an else the kernels took 16
// registers more, and dk, dv of packed documents 290 us instead of 208; with
// both products in every step 216, and the forward 135 instead of 124.)
template <bool FAR>
__device__ __forceinline__ void add_axes(f32x16 &s, const u32x2 *rows, int step, int axes,
                                         const u32x2 *cols, const float *slopes)
{
#pragma unroll
    for (int x = 0; x < 3; ++x) {
        if (x >= axes) break;
        const f32x16 p = differences<FAR>(rows + x * step, cols[x]);
#pragma unroll
        for (int r = 0; r < 16; ++r) s[r] = fmaf(-slopes[x], fabsf(p[r]), s[r]);
        if constexpr (FAR) asm volatile("" : "+v"(s));
    }
}
__device__ __forceinline__ void add_bias(f32x16 &s, const u32x2 *rows, int step, int axes,
                                         const u32x2 *cols, const float *slopes)
{
    if (__builtin_expect_with_probability(axes < 0, 0, 1.0))
        add_axes<true>(s, rows, step, -axes, cols, slopes);
    add_axes<false>(s, rows, step, axes, cols, slopes);
}

// The 16 scores of a result to c tanh(s / c).  float32: the library's
// tanhf, for its relative accuracy near 0.  16-bit types, which keep 2^-9 or
// 2^-12 of a weight: 1 - 2 / (1 + e^2x), within 2e-7; and where no score of the
// wave passes c / 4, as with a cap well above the scores, the odd Taylor
// polynomial, within 1e-7, in 5 instructions instead of 5 of which two (the
// exponential and the reciprocal) take twice the time or more.  So a query's
// last bits depend on the scores of the wave's other queries, but not on what
// it does not see: a tile of which some is masked (`part`) takes the first form.
template <typename T>
__device__ __forceinline__ void cap_scores(f32x16 &s, const Scores &sc, bool part)
{
    const float f = sc.per_cap;
    if constexpr (T::code == F32::code) {
#pragma unroll
        for (int r = 0; r < 16; ++r) s[r] = sc.cap * tanhf(s[r] * f);
        return;
    }
    float big = fabsf(s[0]);
#pragma unroll
    for (int r = 1; r < 16; ++r) big = fmaxf(big, fabsf(s[r]));
    if (!part && !__any(!(big * f < 0.25f))) {
        const float f2 = f * f, c3 = -f2 / 3.f, c5 = f2 * f2 * (2.f / 15.f),
                    c7 = f2 * f2 * f2 * (-17.f / 315.f);
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            const float y = s[r] * s[r];
            s[r] = fmaf(fmaf(fmaf(c7, y, c5), y, c3) * y, s[r], s[r]);
        }
    } else {
        const float g = f * (2.f * kLog2e);
#pragma unroll
        for (int r = 0; r < 16; ++r)
            s[r] = fmaf(-2.f * sc.cap,
                        __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(s[r] * g)), sc.cap);
    }
}

// The derivative of a capped score by the score: 1 - tanh^2 (the square of the
// quotient: the cap's own may leave binary32).
__device__ __forceinline__ float cap_slope(float s, const Scores &sc)
{
    const float t = s * sc.per_cap;
    return fmaf(-t, t, 1.f);
}

}  // namespace mp3d
