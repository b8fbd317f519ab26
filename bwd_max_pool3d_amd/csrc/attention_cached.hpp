// attention_cached.hpp -- attention of new tokens over caches, plain or of 8
// or 4 bits, behind prefixes that sequences share: the kernel that walks
// them.
//
// One launch has two kinds of workgroups, over the shared prefixes and over
// the sequences' own caches; a chunk of keys of one cache and key head each.
// The rows of a block are the query heads that share the key head, of all
// new tokens, and over a prefix of all sequences that share it: so a prefix
// is read once for all of them (for each block of rows, see below), not once a
// sequence.  The chunks' sums are joined by a second kernel, which does not
// care which cache they came from.
//
// A tile is 32 keys and their values, as elements in LDS (attention.hpp has
// the layout and the products).  Codes are read 16 channels a lane into
// registers, a tile ahead, and widened as they are placed in LDS: values are
// exactly what a cache is read back as, in the queries' type.  (Widening the
// fragments instead would need a value's scale per key inside a lane's eight
// keys.)  Elements go to LDS directly.
//
// Few rows go in blocks of 16 (MB = 16): each wave has all 16 and tiles of its
// own, no wave waits for another.  More rows go in blocks of 128 (MB = 32): the
// waves have 32 each, and share two tiles that they bring in turn, a quarter
// each; codes are read and widened once for 128 rows, into the one half of LDS
// while the products run from the other.
//
// Bound, and what the kernel takes (the join's 4 to 10 us apart):
//   blocks of 16, long caches: HBM.  16 caches of 9728 to 32768, 32 heads on 8
//     of 128, e4m3: 135 us, 5.3 TB/s; every byte is fetched once.
//   blocks of 128, long prefixes: the matrix and the vector unit in turn, as a
//     wave's softmax waits for its scores.  4096 sequences on 8192 keys, 32 heads
//     on 8 of 128, no own keys: plain 591 us, 930 TFLOP/s, e4m3 646 us, 850, e2m1
//     591 us, 930 (with an own cache of one key each, 32768 workgroups more, 862,
//     950 and 893 us); 64 sequences on 32768 keys, e4m3, 69 us; a workgroup's
//     start and end (6 to 8 us) weigh the more the shorter the chunks are.
//   the same over 128 channels with a cap, a bias or a factor: registers too.
//     The compiler spills 63 of them (e2m1) or 73 (e4m3; plain 15, and without
//     these 2, 14 and none), and a reload in the loop waits behind the codes in
//     flight.  128 drafted rows on 6272 keys, e2m1, cap: 66 us.
//   a few hundred keys: the launch and one step's latency.  777 keys, e2m1: 9 us.
#pragma once

#include <type_traits>

#include "attention.hpp"
#include "cache.hpp"

namespace mp3d {

constexpr int kCachedWaves = 4;
constexpr int kCachedKeys = 32;            // keys of a tile
constexpr int kCachedPad = 4;              // floats between the rows of the join

// floats between the rows of a chunk's sums, for loads of 4
__host__ __device__ inline int cached_stride(int D) { return (D + 3) & ~3; }

// Tiles of LDS a wave: elements straight from memory need one for keys and one
// for values; codes of up to 16 rows take turns in one, so that three
// workgroups fit on a CU (16 caches of 9728 to 32768, e4m3: 137 us; the same
// with two workgroups that read two tiles ahead, for twice the registers).
template <int FMT, int MB>
constexpr int cached_slots() { return FMT == kPlain || MB == 32 ? 2 : 1; }
template <typename T, int FMT, int DP, int MB>
constexpr uint32_t cached_tiles()
{
    const uint32_t tiles = kCachedWaves * cached_slots<FMT, MB>() * kCachedKeys * DP *
                           sizeof(typename T::raw);
    const uint32_t join = kCachedWaves * MB * (DP + kCachedPad) * sizeof(float);
    return tiles > join ? tiles : join;
}
template <typename T, int FMT, int DP, int MB>
constexpr uint32_t cached_lds()
{
    return cached_tiles<T, FMT, DP, MB>() +
           (kCachedWaves * (2 * 3 * kCachedKeys + 2 * MB) + 4) * (uint32_t)sizeof(float);
}

// Workgroups on a CU: of tiles DP wide, of elements of `size` bytes; `general`: the
// kernels with GEN; mb: the most rows of a wave.
constexpr int cached_occupancy(int size, int format, int DP, bool general, int mb)
{
    if (size * DP > 256) return format == kPlain ? 1 : 2;
    return format != kPlain && mb == 16 && !general ? 3 : 2;
}

// --- products with MB columns (rows of the call, in lanes l % MB).  A lane's
// 8 elements of an operand are 8 deep at 8 (l / MB); register e of a result is
// its row group(e) + 4 (l / MB) + e % 4: with 16 columns a result has 16 rows,
// and a tile's keys are two results.  As with 32, registers 8c .. 8c + 7 of the
// scores are the next product's operand, 16 or 32 keys deep.
template <int MB>
struct Cols {
    static constexpr int PARTS = 64 / MB, DEPTH = 8 * PARTS, SCORES = kCachedKeys / PARTS;
    static constexpr int PER = MB == 32 ? 16 : 4;          // registers of a result
    typedef float acc __attribute__((ext_vector_type(MB == 32 ? 16 : 4)));
    typedef float scores __attribute__((ext_vector_type(MB == 32 ? 16 : 8)));
    // a key's place in the tile, or a channel's in its block, without 4 (l / MB)
    __device__ static constexpr int group(int e) { return (MB == 32 ? 8 : 16) * (e / 4) + e % 4; }
    __device__ static __forceinline__ float over_parts_max(float v)
    {
        if constexpr (MB == 16) {
            const auto x = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(uint32_t, v),
                                                            __builtin_bit_cast(uint32_t, v), false,
                                                            false);
            const uint32_t a = x[0], b = x[1];
            v = fmaxf(__builtin_bit_cast(float, a), __builtin_bit_cast(float, b));
        }
        return halves_max(v);
    }
    __device__ static __forceinline__ float over_parts_sum(float v)
    {
        if constexpr (MB == 16) {
            const auto x = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(uint32_t, v),
                                                            __builtin_bit_cast(uint32_t, v), false,
                                                            false);
            const uint32_t a = x[0], b = x[1];
            v = __builtin_bit_cast(float, a) + __builtin_bit_cast(float, b);
        }
        return halves_sum(v);
    }
};

template <typename T, int MB>
__device__ __forceinline__ typename Cols<MB>::acc mma_cols(const Frag<T> &a, const Frag<T> &b,
                                                           typename Cols<MB>::acc c)
{
    if constexpr (MB == 32) {
        return mma<T>(a, b, c);
    } else if constexpr (T::code == BF16::code) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a.w[0]),
                                                       __builtin_bit_cast(bf16x8, b.w[0]), c, 0, 0,
                                                       0);
    } else if constexpr (T::code == F16::code) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a.w[0]),
                                                      __builtin_bit_cast(f16x8, b.w[0]), c, 0, 0,
                                                      0);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const u32x4 x = a.w[i / 4], y = b.w[i / 4];
            const uint32_t xe[4] = {x.x, x.y, x.z, x.w}, ye[4] = {y.x, y.y, y.z, y.w};
            c = __builtin_amdgcn_mfma_f32_16x16x4f32(__builtin_bit_cast(float, xe[i % 4]),
                                                     __builtin_bit_cast(float, ye[i % 4]), c, 0, 0,
                                                     0);
        }
        return c;
    }
}

// Channel d0 + l % MB of the keys that registers 8c .. 8c + 7 are of.
template <typename T, int DP, int MB>
__device__ __forceinline__ Frag<T> value_frag(const typename T::raw *tile, int c, int d0, int l)
{
    using R = typename T::raw;
    if constexpr (MB == 32) {
        return col_frag<T, DP>(tile, c, d0, l);
    } else if constexpr (sizeof(R) == 2) {
        const int col = d0 + (l & 3) * 4, row = 4 * (l >> 4) + ((l & 15) >> 2);
        typedef __attribute__((address_space(3))) s16x4 lds_t;
        struct alignas(16) {
            s16x4 v[2];
        } o;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const R *p = tile + tile_at<R, DP>(row + 16 * k, col >> 3) + (col & 7);
            o.v[k] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_t *)p);
        }
        return __builtin_bit_cast(Frag<T>, o);
    } else {
        const int col = d0 + (l & 15);
        struct alignas(16) {
            float e[8];
        } o;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int row = 4 * (l >> 4) + Cols<16>::group(i);
            o.e[i] = tile[tile_at<R, DP>(row, col >> 3) + (col & 7)];
        }
        return __builtin_bit_cast(Frag<T>, o);
    }
}

// Weights 8c .. 8c + 7 as an operand of the second product, which has operands
// of the queries' type alone: each is off by up to half a step (2^-8 of it in
// bfloat16, 2^-11 in float16), as in mp3d_attention_forward.  Float32 weights would
// take the float32 instructions, at an eighth of the rate.  Out is off by 0.0023
// with it where one rounding of the output is 0.0017 (bfloat16; float16 0.00022 and
// 0.0002); the sums of weights are not rounded.
template <typename T, typename V>
__device__ __forceinline__ Frag<T> pack_scores(const V &s, int c)
{
    struct alignas(16) {
        typename T::raw e[8];
    } o;
#pragma unroll
    for (int i = 0; i < 8; ++i) o.e[i] = T::narrow(s[8 * c + i]);
    return __builtin_bit_cast(Frag<T>, o);
}

// The keys [0, end) of its own cache that new token t of sequence b sees, or
// of the prefix that it shares.
__device__ __forceinline__ int cached_len(const CachedPart &p, int cache)
{
    return p.len ? min(max(p.len[cache], 0), p.T) : p.T;
}
__device__ __forceinline__ int cached_end(const CachedArgs &c, bool own, int len, int t)
{
    if (!own || !c.a.causal) return len;
    return max(min(len, len - c.a.Tq + 1 + t), 0);
}

// A tile of codes on its way from memory to LDS.  A wave's lanes take its
// rows in rounds, 16 channels each.
template <typename T, int FMT, int DP, int KEYS>
struct CodeTile {
    using R = typename T::raw;
    static constexpr int UNITS = DP / 16, ROWS = 64 / UNITS, N = KEYS / ROWS;
    static constexpr int BYTES = code_bytes<FMT>(16), WORDS = BYTES / 4;
    uint32_t c[N][WORDS], s[N];

    static __device__ __forceinline__ int row(int lane) { return lane / UNITS; }
    static __device__ __forceinline__ int unit(int lane) { return lane % UNITS; }

    // The lane's place in a round, of strides under 2^24; `rows`: those of the
    // tile that are there (the others are read from the last, and set to zero
    // when they are placed).
    static __device__ __forceinline__ uint32_t offset(int lane, uint32_t stride, int D)
    {
        return row(lane) * stride + min(unit(lane), (D - 1) / 16) * BYTES;
    }
    static __device__ __forceinline__ uint32_t scale_offset(int lane, uint32_t stride, int D)
    {
        return row(lane) * stride + min(unit(lane), (D - 1) / 16) / 2;
    }
    // A tile at p, its scales at ps.
    __device__ __forceinline__ void load(const uint8_t *p, const uint8_t *ps, uint32_t stride,
                                         uint32_t sstride, uint32_t off, uint32_t soff, int rows,
                                         int lane)
    {
        if (__builtin_expect(rows >= KEYS, 1)) {
#pragma unroll
            for (int j = 0; j < N; ++j) {
                word(j, p + j * ROWS * stride + off);
                s[j] = (ps + j * ROWS * sstride)[soff];
            }
        } else {
            const int r = row(opaque(lane));
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const uint32_t at = min(j * ROWS + r, rows - 1) - r;       // (may be under 0: wraps)
                word(j, p + (uint32_t)(at * stride + off));
                s[j] = ps[(uint32_t)(at * sstride + soff)];
            }
        }
    }
    __device__ __forceinline__ void word(int j, const uint8_t *q)
    {
        if constexpr (WORDS == 4) {
            const u32x4 x = *(const u32x4 *)q;
            c[j][0] = x.x;
            c[j][1] = x.y;
            c[j][2] = x.z;
            c[j][3] = x.w;
        } else {
            const u32x2 x = *(const u32x2 *)q;
            c[j][0] = x.x;
            c[j][1] = x.y;
        }
    }
    // Any tile, from row k0 of base (up to row end - 1), 4 bytes or 1 at a time.
    __device__ __forceinline__ void load_any(const uint8_t *base, const uint8_t *sbase,
                                             int64_t stride, int64_t sstride, int k0, int end,
                                             int width, int D, int lane)
    {
        const int bytes = code_bytes<FMT>(D), u = min(unit(lane), (D - 1) / 16);
        const int left = bytes - u * BYTES;
        // (half of an odd row's last byte is no channel's: what it holds could be
        // past the type, and times the query's 0 there NaN)
        const int odd = FMT == kE2M1 && D & 1 ? D - u * 16 : 16;
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const int64_t r = min(k0 + j * ROWS + row(lane), end - 1);
            const uint8_t *q = base + r * stride + u * BYTES;
            s[j] = sbase[r * sstride + u / 2];
#pragma unroll
            for (int i = 0; i < WORDS; ++i) c[j][i] = 0u;
            if (width >= 4) {
#pragma unroll
                for (int i = 0; i < WORDS; ++i)
                    if (4 * i < left) c[j][i] = ((const uint32_t *)q)[i];
            } else {
#pragma unroll
                for (int i = 0; i < BYTES; ++i)
                    if (i < left) c[j][i / 4] |= (uint32_t)q[i] << (8 * (i % 4));
            }
            if constexpr (FMT == kE2M1) {
#pragma unroll
                for (int i = 0; i < WORDS; ++i)
                    if (odd / 8 == i) c[j][i] &= ~(15u << (4 * (odd % 8)));
            }
        }
    }
    // Into LDS, widened.  clear: rows from `end` on, and units past D, are
    // zero; drop: infinities and NaN too (true if there was one).
    __device__ __forceinline__ bool place(R *tile, int k0, int end, int D, bool clear, bool drop,
                                          int lane)
    {
        bool bad = false;
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const int r = j * ROWS + row(lane), u = unit(lane);
            if (__builtin_expect(clear, 0)) {
                const bool there = k0 + r < end && u * 16 < D;
                s[j] = there ? s[j] : 127u;
#pragma unroll
                for (int i = 0; i < WORDS; ++i) c[j][i] = there ? c[j][i] : 0u;
            }
            const float f = scale_of(s[j]);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                Frag<T> x;
                if constexpr (FMT == kE4M3) widen8<T, FMT>(c[j][2 * h], c[j][2 * h + 1], f, x.w);
                else widen8<T, FMT>(c[j][h], 0u, f, x.w);
                if (__builtin_expect(drop, 0)) bad |= drop_nonfinite<T>(x);
                u32x4 *q = (u32x4 *)(tile + tile_at<R, DP>(r, 2 * u + h));
#pragma unroll
                for (int i = 0; i < Frag<T>::NV; ++i) q[i] = x.w[i];
            }
        }
        return bad;
    }
};

// A tile of elements whose rows start anywhere, by way of registers: 8
// channels a lane, `width` bytes (8, 4, or an element) at a time.
template <typename T, int DP, int KEYS>
struct NarrowTile {
    using R = typename T::raw;
    static constexpr int UNITS = DP / 8, ROWS = 64 / UNITS, N = KEYS / ROWS;
    static constexpr int WORDS = 2 * sizeof(R), PER = 4 / sizeof(R);   // words of 8 channels,
                                                                       // channels of a word
    uint32_t c[N][WORDS];

    __device__ __forceinline__ void load_any(const R *base, const uint8_t *, int64_t stride, int64_t,
                                             int k0, int end, int width, int D, int lane)
    {
        const int d0 = min(lane % UNITS, (D - 1) / 8) * 8, left = D - d0;
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const int64_t r = min(k0 + j * ROWS + lane / UNITS, end - 1);
            const R *p = base + r * stride + d0;
#pragma unroll
            for (int i = 0; i < WORDS; ++i) c[j][i] = 0u;
            if (width >= 8) {
#pragma unroll
                for (int i = 0; i < WORDS; i += 2)
                    if (i * PER < left) {
                        const u32x2 x = ((const u32x2 *)p)[i / 2];
                        c[j][i] = x.x;
                        c[j][i + 1] = x.y;
                    }
            } else if (width == 4) {
#pragma unroll
                for (int i = 0; i < WORDS; ++i)
                    if (i * PER < left) c[j][i] = ((const uint32_t *)p)[i];
            } else if constexpr (PER == 2) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (i < left) c[j][i / 2] |= (uint32_t)p[i] << (16 * (i % 2));
            }
        }
    }
    __device__ __forceinline__ bool place(R *tile, int k0, int end, int D, bool, bool drop, int lane)
    {
        bool bad = false;
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const int r = j * ROWS + lane / UNITS, u = lane % UNITS;
            const bool there = k0 + r < end && u * 8 < D;
            Frag<T> x;
#pragma unroll
            for (int i = 0; i < Frag<T>::NV; ++i)
                x.w[i] = there ? u32x4{c[j][4 * i], c[j][4 * i + 1], c[j][4 * i + 2], c[j][4 * i + 3]}
                               : u32x4{0u, 0u, 0u, 0u};
            if (drop) bad |= drop_nonfinite<T>(x);
            u32x4 *q = (u32x4 *)(tile + tile_at<R, DP>(r, u));
#pragma unroll
            for (int i = 0; i < Frag<T>::NV; ++i) q[i] = x.w[i];
        }
        return bad;
    }
};

template <int N>
struct Half {
    static constexpr int value = N;
};

// The kernel's arguments, read no earlier than here.
__device__ __forceinline__ auto late_args()
{
    typedef const __attribute__((address_space(4))) CachedArgs args_t;
    const args_t *p = (const args_t *)__builtin_amdgcn_kernarg_segment_ptr();
    asm volatile("" : "+s"(p));
    return p;
}

// A workgroup's chunk: `id` of its part of the launch.  ANY: codes of any
// alignment and strides.
template <typename T, int FMT, int DP, int DU, bool GEN, bool ANY, int MB>
__device__ __forceinline__ void cached_chunk(const CachedArgs &c, bool own, uint32_t id,
                                             unsigned char *smem)
{
    using R = typename T::raw;
    using C = Cols<MB>;
    constexpr bool PLAIN = FMT == kPlain, DIRECT = PLAIN && !ANY;
    constexpr int KB = kCachedKeys, NW = kCachedWaves, SLOTS = cached_slots<FMT, MB>();
    constexpr int WR = MB == 16 ? 1 : NW, WK = NW / WR;    // waves that share the rows, the keys out
    constexpr int NC = DU / C::DEPTH, ND = DU / MB, NS = C::SCORES;
    // keys that a wave brings, and goes through, at a time
    constexpr int BRING = WR == 1 ? KB : 2 * KB / NW, TILES = WR == 1 ? 1 : 2;
    constexpr bool ALL = DU == DP;         // whole tiles with all their channels
    // The maximum m that weights are relative to is raised by a score past
    // m + kTop, to that score less kBelow.  float16 weights, which are lost as
    // operands of the second product under 2^-25, so are 2^12 to 2^15 for the
    // largest key, and others count from 2^-37 of it on.  (With it at 1: 2^20
    // keys of 2^-26 behind four of 1 were lost from out while l counted them,
    // 0.4 % of it.  4 x 128 drafts on 6272 keys, e2m1, cap: 69.1 us without, 69.8.)
    constexpr bool LOW = T::code == F16::code;
    constexpr float kTop = LOW ? 15.f : 8.f, kBelow = LOW ? 12.f : 0.f;
    const AttnArgs &a = c.a;
    const CachedPart &p = c.part[own];
    const int axes = GEN ? a.axes : 0;
    const int tid = threadIdx.x, wave = uniform(tid >> 6), lane = tid & 63, col = lane & (MB - 1),
              part4 = lane / MB * 4;
    int *const pos_lds = (int *)(smem + cached_tiles<T, FMT, DP, MB>());   // [NW][2][3][KB]
    float *const ml = (float *)pos_lds + NW * 2 * 3 * KB;              // [NW][MB][2]
    int *const flag = (int *)(ml + NW * 2 * MB);                       // something was dropped

    // Which cache, head, chunk and rows.  Blocks of rows that read the same
    // chunk go to the same XCD, one after another.
    int rb = 0;
    if (p.nrb > 1) {
        const uint32_t i = id >> 3, group = i / (uint32_t)p.nrb;
        rb = (int)(i - group * p.nrb);
        id = group * 8 + (id & 7);
        if (id >= (uint32_t)p.units) return;
    }
    const uint32_t rest_id = id / (uint32_t)a.Hk, sp_no = rest_id / (uint32_t)p.caches;
    const int hk = (int)(id - rest_id * a.Hk), cache = (int)(rest_id - sp_no * p.caches);
    const int rw = WR == 1 ? 0 : wave;

    // the rows: new token t and query head of a sequence
    const int per = a.Tq * a.G, row0 = rb * MB * WR, r = row0 + rw * MB + col;
    const int rc = min(r, p.rows - 1), seq = (uint32_t)rc / (uint32_t)per,
              in_seq = rc - seq * per, t = (uint32_t)in_seq / (uint32_t)a.G;
    const int b = cache * p.seqs + seq, h = hk * a.G + in_seq - t * a.G;
    const int len = cached_len(p, cache);
    const int end = cached_end(c, own, len, t);            // the row's keys
    // the workgroup's chunk, and the keys that all its rows see: the last row
    // of a block sees the most of an own cache, the first the least
    const int last = min(row0 + MB * WR, p.rows) - 1;
    const int most = cached_end(c, own, len, own ? last / a.G : 0);
    const int all = cached_end(c, own, len, own ? row0 / a.G : 0);
    const int c0 = (int)sp_no * p.chunk, c1 = (int)min((int64_t)c0 + p.chunk, (int64_t)most);
    // (the join does not read this chunk)
    if (c0 >= c1 && c.part[0].nsplit + c.part[1].nsplit > 1) return;
    if (tid == 0) *flag = 0;

    const auto *kp = (const R *)p.k, *vp = (const R *)p.v;             // plain
    const uint8_t *kq = (const uint8_t *)p.k, *vq = (const uint8_t *)p.v, *ksc = p.k_scale,
                  *vsc = p.v_scale;
    if constexpr (PLAIN) {
        kp += cache * p.ks[0] + hk * p.ks[2];
        vp += cache * p.vs[0] + hk * p.vs[2];
    } else {
        kq += cache * p.ks[0] + hk * p.ks[2];
        vq += cache * p.vs[0] + hk * p.vs[2];
        ksc += cache * p.kss[0] + hk * p.kss[2];
        vsc += cache * p.vss[0] + hk * p.vss[2];
    }
    typename C::acc o[ND];
#pragma unroll
    for (int d = 0; d < ND; ++d) o[d] = typename C::acc(0.f);
    float m = kNegInf, l = 0.f;
    bool dropped = false;
    __syncthreads();                       // (the flag)

    if (c0 < c1) {
        const int32_t *pos = p.pos + (int64_t)cache * p.T;
        const int64_t pos_axis = (int64_t)p.caches * p.T;
        // wr = 1: the wave's tiles of keys and values, one or two places.
        // wr = 4: the wave's part of two tiles of keys; those of values behind
        // them; the second half of LDS behind all that.
        constexpr int kHalf = 4 * KB * DP;
        R *const kt = (R *)smem + (WR == 1 ? wave * SLOTS * KB * DP : wave * BRING * DP);
        R *const vt = kt + (WR == 1 ? (SLOTS - 1) * KB * DP : 2 * KB * DP);
        // positions: [2][3][keys of a step]
        constexpr int kPos = WR == 1 ? KB : 2 * KB;
        int *const pk = pos_lds + (WR == 1 ? wave * 2 * 3 * KB : 0);

        // (a wave alone with its tile: its operations on LDS keep their order)
        auto in_order = [] { __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront"); };

        // the wave's queries: element by element by way of LDS, or (below, with
        // the first keys on their way) 16 bytes at a time
        const R *qp = (const R *)a.q + b * a.qs[0] + h * a.qs[2] + (int64_t)t * a.qs[1];
        Frag<T> qf[NC];
        if (__builtin_expect(!a.vec, 0)) {
            R *const x = (R *)smem + wave * MB * DP;
            for (int i = 0; i < MB; ++i) {
                const uint32_t lo = __builtin_amdgcn_readlane((uint32_t)(uintptr_t)qp, i),
                               hi = __builtin_amdgcn_readlane((uint32_t)((uintptr_t)qp >> 32), i);
                const R *row = (const R *)(((uintptr_t)hi << 32) | lo);
                for (int ch = lane; ch < DP; ch += 64)
                    x[tile_at<R, DP>(i, ch >> 3) + (ch & 7)] = ch < a.D ? row[ch] : R(0);
            }
            wait_all();
            in_order();
#pragma unroll
            for (int i = 0; i < NC; ++i)
                qf[i] = row_frag<T, DP>(x, col, i * C::DEPTH + part4 * 2);
            reads_done();
            __syncthreads();
        }

        // whole rows of elements: straight to LDS
        using Direct = TileDirect<T, DP, BRING, 64>;
        Direct kd, vd;
        bool whole = false;
        uint32_t lds_k = 0, lds_v = 0, lds_p = 0;
        if constexpr (DIRECT) {
            kd.init(lane, p.ks[1], a.D);
            vd.init(lane, p.vs[1], a.D);
            whole = !ALL || a.D == DP;
            lds_k = lds_address(kt);
            lds_v = lds_address(vt);
            lds_p = lds_address(pk);
            if (a.D < DP) {                // channels that no direct load writes
                for (int x = tid; x < NW * 2 * KB * DP * (int)sizeof(R) / 16; x += 64 * NW)
                    ((u32x4 *)smem)[x] = u32x4{0u, 0u, 0u, 0u};
                __syncthreads();
            }
        }
        auto direct = [&](const Direct &d, const R *x, int64_t stride, int k0, uint32_t lds) {
            if (whole && k0 + BRING <= c1) d.template load<ALL>(x + k0 * stride, lds);
            else d.load_edge(x, stride, k0, c0, c1, lds);
        };
        // three axes or none, so that what is in flight can be counted
        auto direct_pos = [&](int k0, int buf) {
            if (axes > 0 && lane < KB)
#pragma unroll
                for (int x = 0; x < 3; ++x)
                    direct4(pos + min(x, axes - 1) * pos_axis + k0,
                            (uint32_t)min(lane, p.T - 1 - k0) * 4, lds_p + (buf * 3 + x) * KB * 4);
        };

        // all others: by way of registers
        using Codes = CodeTile<T, PLAIN ? kE4M3 : FMT, DP, BRING>;
        std::conditional_t<PLAIN, NarrowTile<T, DP, BRING>, Codes> kc, vc;
        const uint32_t kst = (uint32_t)p.ks[1], vst = (uint32_t)p.vs[1], ksst = (uint32_t)p.kss[1],
                       vsst = (uint32_t)p.vss[1];
        const uint32_t koff = Codes::offset(lane, kst, a.D), voff = Codes::offset(lane, vst, a.D),
                       ksoff = Codes::scale_offset(lane, ksst, a.D),
                       vsoff = Codes::scale_offset(lane, vsst, a.D);
        int pr[3] = {0, 0, 0};
        auto fetch_pos = [&](int k0) {
#pragma unroll
            for (int x = 0; x < 3; ++x) {
                if (x >= axes) break;
                pr[x] = pos[x * pos_axis + min(k0 + (lane & (BRING - 1)), p.T - 1)];
            }
        };
        auto fetch_keys = [&](int k0) {
            if constexpr (PLAIN)
                kc.load_any(kp, nullptr, p.ks[1], 0, k0, c1, p.width, a.D, lane);
            else if constexpr (ANY)
                kc.load_any(kq, ksc, p.ks[1], p.kss[1], k0, c1, p.width, a.D, lane);
            else
                kc.load(kq + (int64_t)k0 * kst, ksc + (int64_t)k0 * ksst, kst, ksst, koff, ksoff,
                        c1 - k0, lane);
            fetch_pos(k0);
        };
        auto fetch_values = [&](int k0) {
            if constexpr (PLAIN)
                vc.load_any(vp, nullptr, p.vs[1], 0, k0, c1, p.width, a.D, lane);
            else if constexpr (ANY)
                vc.load_any(vq, vsc, p.vs[1], p.vss[1], k0, c1, p.width, a.D, lane);
            else
                vc.load(vq + (int64_t)k0 * vst, vsc + (int64_t)k0 * vsst, vst, vsst, voff, vsoff,
                        c1 - k0, lane);
        };
        // some of these keys are not there, or some rows do not see them
        auto partly = [&](int k0, int keys) { return k0 + keys > min(all, c1); };
        auto place_pos = [&](int buf) {
#pragma unroll
            for (int x = 0; x < 3; ++x) {
                if (x >= axes) break;
                if (lane < BRING)
                    pk[(buf * 3 + x) * kPos + (WR == 1 ? 0 : wave * BRING) + lane] = pr[x];
            }
        };
        auto place_keys = [&](int k0, int buf) {
            kc.place(kt + buf * kHalf, k0, c1, a.D, k0 + BRING > c1 || a.D < DP, false, lane);
            place_pos(buf);
        };
        auto place_values = [&](int k0, int buf) {
            dropped |= vc.place(vt + buf * kHalf, k0, c1, a.D, k0 + BRING > c1 || a.D < DP,
                                partly(k0, BRING), lane);
        };
        const int kbeg = c0 + wave * BRING;
        if (kbeg < c1) {
            if constexpr (DIRECT) {
                if (WR == 1) direct_pos(kbeg, 0);
                else fetch_pos(kbeg);
                direct(kd, kp, p.ks[1], kbeg, lds_k);
                direct(vd, vp, p.vs[1], kbeg, lds_v);
            } else {
                fetch_keys(kbeg);
                fetch_values(kbeg);
            }
        }

        if (a.vec) {
#pragma unroll
            for (int i = 0; i < NC; ++i) {
                const int d0 = i * C::DEPTH + part4 * 2;
                qf[i].zero();
                if (ALL || d0 < a.D)
#pragma unroll
                    for (int j = 0; j < Frag<T>::NV; ++j) qf[i].w[j] = ((const u32x4 *)(qp + min(d0, a.D - 8)))[j];
                if (ALL && d0 >= a.D) qf[i].zero();
            }
        }
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
        constexpr int kTile = Direct::LOADS;

        // The scores' factor, cap, bias and mask; keys from k0 on.
        auto finish = [&](typename C::scores (&s)[TILES], int k0, const int *px, bool part) {
            if (GEN) {
#pragma unroll
                for (int u = 0; u < TILES; ++u) multiply_scores(s[u], sc);
            }
            if (GEN && a.cap > 0.f) {
#pragma unroll
                for (int u = 0; u < TILES; ++u) cap_scores<T>(s[u], sc, part);
            }
#pragma unroll
            for (int x = 0; x < 3; ++x) {
                if (x >= axes) break;
                const int *q = px + x * kPos + part4;
#pragma unroll
                for (int u = 0; u < TILES; ++u)
#pragma unroll
                    for (int e = 0; e < NS; ++e) {
                        const int k = q[u * KB + C::group(e)];     // (up to 2^32 apart)
                        const uint32_t far = (uint32_t)max(k, pq[x]) - (uint32_t)min(k, pq[x]);
                        s[u][e] = fmaf(-sl[x], (float)far, s[u][e]);
                    }
            }
            if (part) {
                const int left = end - k0 - part4;
#pragma unroll
                for (int u = 0; u < TILES; ++u)
#pragma unroll
                    for (int e = 0; e < NS; ++e)
                        s[u][e] = u * KB + C::group(e) < left ? s[u][e] : kNegInf;
            }
        };
        // The maximum raised to these scores, and the sums so far with it.
        auto raise = [&](const typename C::scores (&s)[TILES]) {
            float mx = s[0][0];
#pragma unroll
            for (int u = 0; u < TILES; ++u)
#pragma unroll
                for (int e = 0; e < NS; ++e) mx = fmaxf(mx, s[u][e]);
            mx = C::over_parts_max(mx) * sc.mul;
            if (__any(mx > m + kTop)) {
                // (each query by itself: its sums do not depend on its neighbours')
                const float mn = mx > m + kTop ? mx - kBelow : m;
                const float al = __builtin_amdgcn_exp2f(m - (mn == kNegInf ? 0.f : mn));
                l *= al;
#pragma unroll
                for (int d = 0; d < ND; ++d)
#pragma unroll
                    for (int e = 0; e < C::PER; ++e) o[d][e] *= al;
                m = mn;
            }
        };
        auto weights = [&](typename C::scores &s) {
            const float ms = m == kNegInf ? 0.f : m;
#pragma unroll
            for (int e = 0; e < NS; ++e) {
                s[e] = __builtin_amdgcn_exp2f(fmaf(s[e], sc.mul, -ms));
                l += s[e];
            }
        };

        if constexpr (WR == 1) {
            typename C::scores s[1];
            auto products = [&] {
                Frag<T> kf[KB / MB][NC];
                typename C::acc x[KB / MB];
#pragma unroll
                for (int u = 0; u < KB / MB; ++u) {
                    x[u] = typename C::acc(0.f);
#pragma unroll
                    for (int d = 0; d < NC; ++d)
                        kf[u][d] = row_frag<T, DP>(kt, u * MB + col, d * C::DEPTH + part4 * 2);
                }
#pragma unroll
                for (int d = 0; d < NC; ++d)
#pragma unroll
                    for (int u = 0; u < KB / MB; ++u)
                        x[u] = mma_cols<T, MB>(kf[u][d], qf[d], x[u]);
#pragma unroll
                for (int u = 0; u < KB / MB; ++u)
#pragma unroll
                    for (int e = 0; e < C::PER; ++e) s[0][u * C::PER + e] = x[u][e];
            };
            int buf = 0;
            for (int k0 = kbeg; k0 < c1; k0 += NW * KB, buf ^= DIRECT) {
                const int next = k0 + NW * KB;
                const bool more = next < c1, part = partly(k0, KB);
                if constexpr (DIRECT) {
                    // keys: in flight after them are this tile's values
                    wait_loads<kTile>(true);
                    products();
                    reads_done();
                    if (more) {
                        direct_pos(next, buf ^ 1);
                        direct(kd, kp, p.ks[1], next, lds_k);
                    }
                    // values: in flight after them are the next tile's keys
                    if (axes > 0) wait_loads<kTile + 3>(more);
                    else wait_loads<kTile>(more);
                    if (part) {
                        dropped |= vd.scrub(vt, k0, c0, c1, true, nullptr, 0);
                        in_order();
                    }
                } else {
                    in_order();
                    place_keys(k0, 0);
                    if (more) fetch_keys(next);
                    in_order();
                    products();
                    in_order();
                    place_values(k0, 0);
                    if (more) fetch_values(next);
                    in_order();
                }
                Frag<T> vf[ND][NS / 8], w[NS / 8];
#pragma unroll
                for (int d = 0; d < ND; ++d)
#pragma unroll
                    for (int e = 0; e < NS / 8; ++e)
                        vf[d][e] = value_frag<T, DP, MB>(vt, e, d * MB, lane);
                if constexpr (DIRECT) {
                    reads_done();
                    if (more) direct(vd, vp, p.vs[1], next, lds_v);
                }
                finish(s, k0, pk + buf * 3 * KB, part);
                raise(s);
                weights(s[0]);
#pragma unroll
                for (int e = 0; e < NS / 8; ++e) w[e] = pack_scores<T>(s[0], e);
#pragma unroll
                for (int d = 0; d < ND; ++d)
#pragma unroll
                    for (int e = 0; e < NS / 8; ++e) o[d] = mma_cols<T, MB>(vf[d][e], w[e], o[d]);
            }
        } else {
            // this wave's part of two tiles, into the half `buf`
            auto place = [&](int k0, int buf) {
                if constexpr (DIRECT) {
                    wait_loads<0>(false);
                    if (k0 < c1) {
                        if (partly(k0, BRING))
                            dropped |= vd.scrub(vt + buf * kHalf, k0, c0, c1, true, nullptr, 0);
                        place_pos(buf);
                    }
                } else if (k0 < c1) {
                    place_keys(k0, buf);
                    place_values(k0, buf);
                }
                if (k0 >= c1 && k0 - wave * BRING < c1) {
                    // (behind the last key, in a step that has some)
                    for (int x = lane; x < BRING * DP * (int)sizeof(R) / 16; x += 64)
                        ((u32x4 *)(vt + buf * kHalf))[x] = u32x4{0u, 0u, 0u, 0u};
                }
                hand_over();
            };
            place(kbeg, 0);
            // blocks of channels whose values are read ahead of the weights
            constexpr int AHEAD = GEN ? 1 : ND / 2;
            auto step = [&](int first, auto half) {
                constexpr int buf = decltype(half)::value;
                const int next = first + 2 * KB + wave * BRING;
                const bool part = partly(first, 2 * KB);
                if (next < c1) {
                    if constexpr (DIRECT) {
                        constexpr uint32_t off = (buf ^ 1) * kHalf * (uint32_t)sizeof(R);
                        fetch_pos(next);
                        direct(kd, kp, p.ks[1], next, lds_k + off);
                        direct(vd, vp, p.vs[1], next, lds_v + off);
                    } else {
                        fetch_keys(next);
                        fetch_values(next);
                    }
                }
                const R *kb = (const R *)smem + buf * kHalf, *vb = kb + 2 * KB * DP;
                Frag<T> kf[NC][2], vf[ND][4], w[4];
                typename C::scores s[TILES] = {};
                auto read_values = [&](int d) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) vf[d][e] = col_frag<T, DP>(vb, e, d * 32, lane);
                };
#pragma unroll
                for (int d = 0; d < NC; ++d)
#pragma unroll
                    for (int u = 0; u < 2; ++u)
                        kf[d][u] = row_frag<T, DP>(kb, u * 32 + col, d * 16 + part4 * 2);
#pragma unroll
                for (int d = 0; d < NC; ++d)
#pragma unroll
                    for (int u = 0; u < 2; ++u) s[u] = mma<T>(kf[d][u], qf[d], s[u]);
#pragma unroll
                for (int d = 0; d < AHEAD; ++d) read_values(d);
                reads_ahead<T, NC>();
                products_and_reads<T, NC, 1>();
                products_and_reads<T, AHEAD * 4, 2>();
                products_and_reads<T, NC - AHEAD * 4, 0>();
                issued<T>();
                finish(s, first, pk + buf * 3 * kPos, part);
                raise(s);
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    weights(s[u]);
                    w[2 * u] = pack_scores<T>(s[u], 0);
                    w[2 * u + 1] = pack_scores<T>(s[u], 1);
                }
                // (a block's reads go out under the products of the AHEAD before)
#pragma unroll
                for (int x = 0; x < ND; x += AHEAD) {
#pragma unroll
                    for (int d = x + AHEAD; d < x + 2 * AHEAD && d < ND; ++d) read_values(d);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
#pragma unroll
                        for (int d = x; d < x + AHEAD && d < ND; ++d)
                            o[d] = mma<T>(vf[d][e], w[e], o[d]);
                }
                products_and_reads<T, (ND - AHEAD) * 4, 2>();
                products_and_reads<T, AHEAD * 4, 0>();
                issued<T>();
                if (first + 2 * KB < c1) place(next, buf ^ 1);
            };
            for (int first = c0; first < c1; first += 4 * KB) {
                step(first, Half<0>{});
                if (first + 2 * KB < c1) step(first + 2 * KB, Half<1>{});
            }
        }
        if (__any(dropped) && lane == 0) *flag = 1;
    }
    l = C::over_parts_sum(l);

    __syncthreads();

    if (WR > 1 && !*flag) {
        // every row is one wave's: straight from its registers
        const auto *late = late_args();
        const int64_t total = (int64_t)late->a.B * late->a.Hq * late->a.Tq;
        const int D = late->a.D, first_slot = late->part[0].nsplit,
                  slots = first_slot + late->part[1].nsplit,
                  slot = (int)sp_no + (own ? first_slot : 0);
        if (r >= late->part[own].rows) return;
        if (slots > 1) {
            const int64_t at = slot * total + ((int64_t)b * late->a.Hk + hk) * per + in_seq;
            float *out = late->a.part_o + at * cached_stride(D);
#pragma unroll
            for (int d = 0; d < ND; ++d)
#pragma unroll
                for (int e = 0; e < C::PER; e += 4) {
                    const int x = d * MB + C::group(e) + part4;
                    if (x < D) *(f32x4 *)(out + x) = f32x4{o[d][e], o[d][e + 1], o[d][e + 2], o[d][e + 3]};
                }
            if (part4 == 0) *(float2 *)(late->a.part_ml + 2 * at) = make_float2(m, l);
        } else {
            const int64_t at = ((int64_t)b * late->a.Tq + t) * late->a.Hq + h;
            if constexpr (MB == 32)
                store_cols<T, ND>((R *)late->a.out + at * D, o, l == 0.f ? 0.f : 1.f / l, D, part4 / 4);
            if (part4 == 0)
                late->a.lse[((int64_t)b * late->a.Hq + h) * late->a.Tq + t] =
                    l == 0.f ? kNegInf : (m + log2f(l)) * kLn2;
        }
        return;
    }

    // join the waves that have the same rows
    float *const jo = (float *)smem;                       // [NW][MB][DP + pad]
    constexpr int JW = DP + kCachedPad;
    if (part4 == 0) {
        ml[(wave * MB + col) * 2] = m;
        ml[(wave * MB + col) * 2 + 1] = l;
    }
#pragma unroll
    for (int d = 0; d < ND; ++d)
#pragma unroll
        for (int e = 0; e < C::PER; e += 4)
            *(f32x4 *)(jo + (wave * MB + col) * JW + d * MB + C::group(e) + part4) =
                f32x4{o[d][e], o[d][e + 1], o[d][e + 2], o[d][e + 3]};
    __syncthreads();
    // (the call's arguments are read again here: kept through the loops they
    // would fill the scalar registers)
    const auto *late = late_args();
    const int64_t total = (int64_t)late->a.B * late->a.Hq * late->a.Tq;
    const int D = late->a.D, G = late->a.G, rows = late->part[own].rows;
    const int first_slot = late->part[0].nsplit, slots = first_slot + late->part[1].nsplit;
    const int slot = (int)sp_no + (own ? first_slot : 0), stride = cached_stride(D);
    const bool some = *flag;               // an infinity or a NaN was dropped
    for (int x = tid; x < MB * WR * (DP / 4); x += 64 * NW) {
        const int rr = x / (DP / 4), d = (x - rr * (DP / 4)) * 4;
        if (row0 + rr >= rows) break;
        if (d >= D) continue;
        float mt = kNegInf;
#pragma unroll
        for (int w = 0; w < WK; ++w) mt = fmaxf(mt, ml[(w * MB + rr) * 2]);
        const float ms = mt == kNegInf ? 0.f : mt;
        float lt = 0.f;
        f32x4 ot = f32x4(0.f);
#pragma unroll
        for (int w = 0; w < WK; ++w) {
            const int at = w * MB + rr;
            const float f = __builtin_amdgcn_exp2f(ml[at * 2] - ms);
            lt = fmaf(f, ml[at * 2 + 1], lt);
            const f32x4 v = *(const f32x4 *)(jo + at * JW + d);
#pragma unroll
            for (int e = 0; e < 4; ++e) ot[e] = fmaf(f, v[e], ot[e]);
        }
        const int rg = row0 + rr, sq = rg / per, rest = rg - sq * per, tt = rest / G;
        if (some) {
            // the keys that some rows do not see again: what was dropped, to
            // the rows that do see it
            const int row_end = min(cached_end(c, own, len, tt), c1), whole = min(all, c1);
            for (int key = max(c0, whole - 2 * KB + 1); key < row_end; ++key) {
                if (key / BRING * BRING + BRING <= whole) continue;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if (d + e >= D) break;
                    float v;
                    if constexpr (PLAIN) v = T::widen(vp[(int64_t)key * p.vs[1] + d + e]);
                    else v = value_at<T, FMT>(vq + key * p.vs[1], vsc + key * p.vss[1], d + e);
                    if (!(fabsf(v) < __builtin_huge_valf())) ot[e] += v;
                }
            }
        }
        const int64_t bb = cache * (int64_t)late->part[own].seqs + sq;
        if (slots > 1) {
            const int64_t at = slot * total + (bb * late->a.Hk + hk) * per + rest;
            *(f32x4 *)(late->a.part_o + at * stride + d) = ot;
            if (d == 0) *(float2 *)(late->a.part_ml + 2 * at) = make_float2(mt, lt);
        } else {
            const int hh = hk * G + rest - tt * G;
            const int64_t at = (bb * late->a.Tq + tt) * late->a.Hq + hh;
            R *out = (R *)late->a.out + at * D + d;
            const float inv = lt == 0.f ? 0.f : 1.f / lt;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (d + e < D) out[e] = T::narrow(lt == 0.f ? 0.f : ot[e] * inv);
            if (d == 0)
                late->a.lse[(bb * late->a.Hq + hh) * late->a.Tq + tt] =
                    lt == 0.f ? kNegInf : (mt + log2f(lt)) * kLn2;
        }
    }
}

// MP, MO: columns of the prefix' and of the own caches' workgroups.
template <typename T, int FMT, int DP, int DU, bool GEN, bool ANY, int MP, int MO>
__global__ __launch_bounds__(64 * kCachedWaves,
                             (cached_occupancy(sizeof(typename T::raw), FMT, DP, GEN, MP)))
void attn_cached_kernel(CachedArgs c)
{
    extern __shared__ __align__(16) unsigned char smem[];
    const uint32_t first = (uint32_t)c.part[0].blocks;
    if constexpr (MP == MO) {
        const bool own = blockIdx.x >= first;
        cached_chunk<T, FMT, DP, DU, GEN, ANY, MP>(c, own, blockIdx.x - (own ? first : 0), smem);
    } else if (blockIdx.x < first) {
        cached_chunk<T, FMT, DP, DU, GEN, ANY, MP>(c, false, blockIdx.x, smem);
    } else {
        cached_chunk<T, FMT, DP, DU, GEN, ANY, MO>(c, true, blockIdx.x - first, smem);
    }
}

template <typename T, int FMT, int DP, int DU, bool GEN, bool ANY, int MP, int MO>
hipError_t run_cached(const CachedArgs &c, hipStream_t s)
{
    constexpr uint32_t p = cached_lds<T, FMT, DP, MP>(), o = cached_lds<T, FMT, DP, MO>();
    launch_kernel((attn_cached_kernel<T, FMT, DP, DU, GEN, ANY, MP, MO>),
                  dim3((uint32_t)(c.part[0].blocks + c.part[1].blocks)), dim3(64 * kCachedWaves),
                  p > o ? p : o, s, c);
    return hipGetLastError();
}

template <typename T, int FMT, int DP, int DU, bool GEN, bool ANY = false>
hipError_t run_cached_rows(const CachedArgs &c, hipStream_t s)
{
    // (a prefix has at least the rows of an own cache; a part without
    // workgroups takes the other's)
    if constexpr (T::code == F32::code || (FMT == kPlain && ANY)) {
        return run_cached<T, FMT, DP, DU, GEN, ANY, 16, 16>(c, s);
    } else {
        const int mo = c.part[1].blocks ? c.part[1].mb : c.part[0].mb;
        const int mp = c.part[0].blocks ? c.part[0].mb : mo;
        if (mp == 16) return run_cached<T, FMT, DP, DU, GEN, ANY, 16, 16>(c, s);
        if (mo == 16) return run_cached<T, FMT, DP, DU, GEN, ANY, 32, 16>(c, s);
        return run_cached<T, FMT, DP, DU, GEN, ANY, 32, 32>(c, s);
    }
}

template <typename T, int FMT, int DP, int DU>
hipError_t run_cached_scores(const CachedArgs &c, hipStream_t s)
{
    return attn_general(c.a) ? run_cached_rows<T, FMT, DP, DU, true>(c, s)
                             : run_cached_rows<T, FMT, DP, DU, false>(c, s);
}

template <typename T, int FMT>
hipError_t run_cached_width(const CachedArgs &c, hipStream_t s)
{
    if (c.any)
        return c.a.D <= 64 ? run_cached_rows<T, FMT, 64, 64, true, true>(c, s)
                           : run_cached_rows<T, FMT, 128, 128, true, true>(c, s);
    if (c.a.D <= 64) return run_cached_scores<T, FMT, 64, 64>(c, s);
    if (c.a.D <= 96) return run_cached_scores<T, FMT, 128, 96>(c, s);
    return run_cached_scores<T, FMT, 128, 128>(c, s);
}

// (in translation units by format and type)
template <typename T, int FMT>
hipError_t launch_cached(const CachedArgs &c, hipStream_t s);

}  // namespace mp3d
