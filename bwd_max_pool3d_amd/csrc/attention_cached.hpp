// attention_cached.hpp -- attention of new tokens over caches, plain or of 8
// or 4 bits, behind prefixes that sequences share: the kernel that walks
// them.
//
// One launch has two kinds of workgroups, over the shared prefixes and over
// the sequences' own caches; a chunk of keys of one cache and key head each.
// The rows of a block are the query heads that share the key head, of all
// new tokens, and over a prefix of all sequences that share it: so a prefix
// is read once for all of them (for each 32 wr rows, see below), not once a
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
// wr of a workgroup's four waves have rows of their own, 32 each, and share
// tiles; the other waves have other tiles.  wr = 1 (up to 32 rows): no wave
// waits for another.  wr = 2, 4: codes are read and widened once for 64 or 128
// rows, each wave a part of the tile, with two or four tiles of LDS in turn and
// a barrier a tile.
#pragma once

#include "attention.hpp"
#include "cache.hpp"

namespace mp3d {

constexpr int kCachedWaves = 4;
constexpr int kCachedKeys = 32;            // keys of a tile
constexpr int kCachedPad = 4;              // floats between the rows of the join

// floats between the rows of a chunk's sums, for loads of 4
__host__ __device__ inline int cached_stride(int D) { return (D + 3) & ~3; }

template <typename T, int DP>
constexpr uint32_t cached_tiles()
{
    const uint32_t tiles = kCachedWaves * 2 * kCachedKeys * DP * sizeof(typename T::raw);
    const uint32_t join = kCachedWaves * 32 * (DP + kCachedPad) * sizeof(float);
    return tiles > join ? tiles : join;
}
template <typename T, int DP>
constexpr uint32_t cached_lds()
{
    return cached_tiles<T, DP>() +
           (kCachedWaves * (2 * 3 * kCachedKeys + 64) + 4) * (uint32_t)sizeof(float);
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
// rows in rounds, 16 channels each; with wr waves to a tile each takes every
// wr-th round.
template <typename T, int FMT, int DP>
struct CodeTile {
    using R = typename T::raw;
    static constexpr int UNITS = DP / 16, ROWS = 64 / UNITS, N = kCachedKeys / ROWS;
    static constexpr int BYTES = code_bytes<FMT>(16), WORDS = BYTES / 4;
    uint32_t c[N][WORDS], s[N];

    static __device__ __forceinline__ int row(int lane) { return lane / UNITS; }
    static __device__ __forceinline__ int unit(int lane) { return lane % UNITS; }

    // Tile whose rows are all there, the first at p (scales at ps), of
    // strides under 2^24; `off`, `soff` the lane's places in a round.
    static __device__ __forceinline__ uint32_t offset(int lane, int64_t stride, int D)
    {
        return (uint32_t)(row(lane) * stride) + min(unit(lane), (D - 1) / 16) * BYTES;
    }
    static __device__ __forceinline__ uint32_t scale_offset(int lane, int64_t stride, int D)
    {
        return (uint32_t)(row(lane) * stride) + min(unit(lane), (D - 1) / 16) / 2;
    }
    __device__ __forceinline__ void load(const uint8_t *p, const uint8_t *ps, int64_t stride,
                                         int64_t sstride, uint32_t off, uint32_t soff, int rw,
                                         int wr)
    {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            if ((j & (wr - 1)) != rw) continue;
            const uint8_t *q = p + j * ROWS * stride + off;
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
            s[j] = (ps + j * ROWS * sstride)[soff];
        }
    }
    // Any tile, from row k0 of base; rows from `end` on are read from the last
    // before it, and set to zero when they are placed.
    __device__ __forceinline__ void load_any(const uint8_t *base, const uint8_t *sbase,
                                             int64_t stride, int64_t sstride, int k0, int end,
                                             int width, int D, int lane, int rw, int wr)
    {
        const int l = opaque(lane), bytes = code_bytes<FMT>(D);
        const int u = min(unit(l), (D - 1) / 16);
#pragma unroll
        for (int j = 0; j < N; ++j) {
            if ((j & (wr - 1)) != rw) continue;
            const int64_t r = min(k0 + j * ROWS + row(l), end - 1);
            const uint8_t *q = base + r * stride + u * BYTES;
            const int left = bytes - u * BYTES;
            s[j] = sbase[r * sstride + u / 2];
            if (width == BYTES) {
                const uint32_t *w = (const uint32_t *)__builtin_assume_aligned(q, BYTES);
#pragma unroll
                for (int i = 0; i < WORDS; ++i) c[j][i] = w[i];
            } else if (width == 4) {
#pragma unroll
                for (int i = 0; i < WORDS; ++i)
                    c[j][i] = 4 * i < left ? ((const uint32_t *)q)[i] : 0u;
            } else {
#pragma unroll
                for (int i = 0; i < WORDS; ++i) c[j][i] = 0u;
#pragma unroll
                for (int i = 0; i < BYTES; ++i)
                    if (i < left) c[j][i / 4] |= (uint32_t)q[i] << (8 * (i % 4));
            }
        }
    }
    // Into LDS, widened.  clear: rows from `end` on, and units past D, are
    // zero; drop: infinities and NaN too (true if there was one).
    __device__ __forceinline__ bool place(R *tile, int k0, int end, int D, bool clear, bool drop,
                                          int lane, int rw, int wr)
    {
        bool bad = false;
#pragma unroll
        for (int j = 0; j < N; ++j) {
            if ((j & (wr - 1)) != rw) continue;
            const int r = j * ROWS + row(lane), u = unit(lane);
            if (clear) {
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
                if (drop) bad |= drop_nonfinite<T>(x);
                u32x4 *q = (u32x4 *)(tile + tile_at<R, DP>(r, 2 * u + h));
#pragma unroll
                for (int i = 0; i < Frag<T>::NV; ++i) q[i] = x.w[i];
            }
        }
        return bad;
    }
};

template <typename T, int FMT, int DP, int DU, bool GEN>
__global__ __launch_bounds__(64 * kCachedWaves, (sizeof(typename T::raw) * DP > 256 ? 1 : 2))
void attn_cached_kernel(CachedArgs c)
{
    using R = typename T::raw;
    constexpr bool PLAIN = FMT == kPlain;
    constexpr int KB = kCachedKeys, NC = DU / 16, ND = DU / 32, NW = kCachedWaves;
    constexpr bool ALL = DU == DP;         // whole tiles with all their channels
    constexpr float kRaise = 8.f;
    extern __shared__ __align__(16) unsigned char smem[];
    const AttnArgs &a = c.a;
    const int axes = GEN ? a.axes : 0;
    const int tid = threadIdx.x, wave = uniform(tid >> 6), lane = tid & 63, col = lane & 31,
              half = lane >> 5;
    int *const pos_lds = (int *)(smem + cached_tiles<T, DP>());        // [NW][2][3][KB]
    float *const ml = (float *)pos_lds + NW * 2 * 3 * KB;              // [NW][32][2]
    int *const flag = (int *)(ml + NW * 64);                           // something was dropped

    // Which cache, head, chunk and rows.  Blocks of rows that read the same
    // chunk go to the same XCD, one after another.
    const bool own = blockIdx.x >= c.part[0].blocks;
    const CachedPart &p = c.part[own];
    int64_t id = blockIdx.x - (own ? c.part[0].blocks : 0);
    int rb = 0;
    if (p.nrb > 1) {
        const int64_t i = id >> 3;
        rb = (int)(i % p.nrb);
        id = (i / p.nrb) * 8 + (id & 7);
        if (id >= p.units) return;
    }
    const int hk = (int)(id % a.Hk);
    id /= a.Hk;
    const int cache = (int)(id % p.caches), sp_no = (int)(id / p.caches);
    const int wr = PLAIN ? 1 : p.wr, wk = NW / wr, rw = wave & (wr - 1), kw = wave / wr;

    // the rows: new token t and query head of a sequence
    const int per = a.Tq * a.G, row0 = rb * 32 * wr, r = row0 + rw * 32 + col;
    const int rc = min(r, p.rows - 1), seq = rc / per, t = (rc - seq * per) / a.G;
    const int b = cache * p.seqs + seq, h = hk * a.G + (rc - seq * per) % a.G;
    const int len = cached_len(p, cache);
    const int end = cached_end(c, own, len, t);            // the row's keys
    // the workgroup's chunk, and the keys that all its rows see: the last row
    // of a block sees the most of an own cache, the first the least
    const int last = min(row0 + 32 * wr, p.rows) - 1;
    const int most = cached_end(c, own, len, own ? last / a.G : 0);
    const int all = cached_end(c, own, len, own ? row0 / a.G : 0);
    const int c0 = sp_no * p.chunk, c1 = (int)min((int64_t)c0 + p.chunk, (int64_t)most);
    const int slots = c.part[0].nsplit + c.part[1].nsplit;
    if (c0 >= c1 && slots > 1) return;     // (the join does not read this chunk)
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
    f32x16 o[ND];
#pragma unroll
    for (int d = 0; d < ND; ++d) o[d] = f32x16(0.f);
    float m = kNegInf, l = 0.f;
    bool dropped = false;
    __syncthreads();                       // (the flag)

    if (c0 < c1) {
        R *const tiles = (R *)smem;
        int *const pk = pos_lds + wave * 2 * 3 * KB;
        const int32_t *pos = p.pos + (int64_t)cache * p.T;
        const int64_t pos_axis = (int64_t)p.caches * p.T;
        const int steps = ((c1 - c0 + KB - 1) / KB + wk - 1) / wk;

        // plain: straight to LDS
        TileDirect<T, DP, KB, 64> kd, vd;
        R *const kt = tiles + wave * 2 * KB * DP, *const vt = kt + KB * DP;
        bool usable = false, whole = false;
        uint32_t lds_k = 0, lds_v = 0, lds_p = 0;
        if constexpr (PLAIN) {
            kd.init(lane, p.ks[1], a.D);
            vd.init(lane, p.vs[1], a.D);
            usable = kd.usable(p.vec, p.ks[1], a.D) && vd.usable(p.vec, p.vs[1], a.D);
            whole = usable && (!ALL || a.D == DP);
            lds_k = lds_address(kt);
            lds_v = lds_address(vt);
            lds_p = lds_address(pk);
            if (a.D < DP) {                // channels that no direct load writes
                for (int x = lane; x < 2 * KB * DP * (int)sizeof(R) / 16; x += 64)
                    ((u32x4 *)kt)[x] = u32x4{0u, 0u, 0u, 0u};
                reads_done();              // (these writes are)
            }
        }
        auto direct = [&](const TileDirect<T, DP, KB, 64> &d, const R *x, int64_t stride, int k0,
                          uint32_t lds) {
            if (whole && k0 + KB <= c1) d.template load<ALL>(x + k0 * stride, lds);
            else if (usable) d.load_edge(x, stride, k0, c0, c1, lds);
        };
        auto by_registers = [&](const R *x, int64_t stride, int k0, R *tile) {
            TileRegs<T, DP, KB, 64> g;
            g.load(x, stride, k0, c0, c1, a.D, p.vec, lane);
            g.store(tile, lane);
            wait_all();
        };
        // three axes or none, so that what is in flight can be counted
        auto direct_pos = [&](int k0, int buf) {
            if (axes > 0 && lane < KB)
#pragma unroll
                for (int x = 0; x < 3; ++x)
                    direct4(pos + min(x, axes - 1) * pos_axis + k0,
                            (uint32_t)min(lane, p.T - 1 - k0) * 4, lds_p + (buf * 3 + x) * KB * 4);
        };

        // codes: by way of registers
        using Codes = CodeTile<T, PLAIN ? kE4M3 : FMT, DP>;
        Codes kc, vc;
        const bool fast = !PLAIN && p.width == Codes::BYTES &&
                          max(max(p.ks[1], p.vs[1]), max(p.kss[1], p.vss[1])) < (1 << 24);
        const uint32_t koff = Codes::offset(lane, p.ks[1], a.D),
                       voff = Codes::offset(lane, p.vs[1], a.D),
                       ksoff = Codes::scale_offset(lane, p.kss[1], a.D),
                       vsoff = Codes::scale_offset(lane, p.vss[1], a.D);
        int pr[3] = {0, 0, 0};
        auto fetch = [&](int k0) {
            if (fast && k0 + KB <= c1) {
                kc.load(kq + k0 * p.ks[1], ksc + k0 * p.kss[1], p.ks[1], p.kss[1], koff, ksoff, rw,
                        wr);
                vc.load(vq + k0 * p.vs[1], vsc + k0 * p.vss[1], p.vs[1], p.vss[1], voff, vsoff, rw,
                        wr);
            } else {
                kc.load_any(kq, ksc, p.ks[1], p.kss[1], k0, c1, p.width, a.D, lane, rw, wr);
                vc.load_any(vq, vsc, p.vs[1], p.vss[1], k0, c1, p.width, a.D, lane, rw, wr);
            }
#pragma unroll
            for (int x = 0; x < 3; ++x) {
                if (x >= axes) break;
                pr[x] = pos[x * pos_axis + min(k0 + col, p.T - 1)];
            }
        };

        const int kbeg = c0 + kw * KB;
        if constexpr (PLAIN) {
            if (kbeg < c1) {
                direct_pos(kbeg, 0);
                direct(kd, kp, p.ks[1], kbeg, lds_k);
                direct(vd, vp, p.vs[1], kbeg, lds_v);
            }
        } else {
            if (kbeg < c1) fetch(kbeg);
        }

        const R *qp = (const R *)a.q + b * a.qs[0] + h * a.qs[2] + (int64_t)t * a.qs[1];
        Frag<T> qf[NC];
#pragma unroll
        for (int i = 0; i < NC; ++i) qf[i] = load8<T>(qp, i * 16 + half * 8, a.D, a.vec);
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
        for (int i = 0; i < steps; ++i, buf ^= 1) {
            const int k0 = kbeg + i * wk * KB;
            const bool live = k0 < c1, more = k0 + wk * KB < c1, part = k0 + KB > min(all, c1);
            const R *kx = kt, *vx = vt;
            const int *px = pk + buf * 3 * KB;
            Frag<T> kf[NC], vf[ND][2];
            f32x16 s = f32x16(0.f);
            if constexpr (PLAIN) {
                if (!live) break;
                // keys: in flight after them are this tile's values.  (A wave's
                // LDS operations keep their order: no barrier)
                wait_loads<kTile>(usable);
                if (!usable) by_registers(kp, p.ks[1], k0, kt);
            } else {
                R *const slot = tiles + (kw * wr + (i & (wr - 1))) * 2 * KB * DP;
                kx = slot;
                vx = slot + KB * DP;
                px = pk;
                if (live) {
                    // (a wave alone with its tile: its reads of the last one
                    // come before these writes)
                    const bool edge = k0 + KB > c1 || a.D < DP;
                    kc.place(slot, k0, c1, a.D, edge, false, lane, rw, wr);
                    dropped |= vc.place(slot + KB * DP, k0, c1, a.D, edge, part, lane, rw, wr);
#pragma unroll
                    for (int x = 0; x < 3; ++x) {
                        if (x >= axes) break;
                        if (half == 0) pk[x * KB + col] = pr[x];
                    }
                }
                if (wr > 1) hand_over();
                else __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
                if (more) fetch(k0 + wk * KB);
                if (!live) continue;
            }
#pragma unroll
            for (int d = 0; d < NC; ++d) kf[d] = row_frag<T, DP>(kx, col, d * 16 + half * 8);
            if constexpr (PLAIN) {
                reads_done();
                if (more) {
                    direct_pos(k0 + wk * KB, buf ^ 1);
                    direct(kd, kp, p.ks[1], k0 + wk * KB, lds_k);
                }
            }
#pragma unroll
            for (int d = 0; d < NC; ++d) s = mma<T>(kf[d], qf[d], s);
            if constexpr (PLAIN) {
                // values: in flight after them are the next tile's keys
                if (axes > 0) wait_loads<kTile + 3>(more && usable);
                else wait_loads<kTile>(more && usable);
                if (!usable) by_registers(vp, p.vs[1], k0, vt);
                if (part) {
                    dropped |= vd.scrub(vt, k0, c0, c1, true, nullptr, 0);
                    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
                }
            }
#pragma unroll
            for (int d = 0; d < ND; ++d)
#pragma unroll
                for (int e = 0; e < 2; ++e) vf[d][e] = col_frag<T, DP>(vx, e, d * 32, lane);
            if constexpr (PLAIN) {
                reads_done();
                if (more) direct(vd, vp, p.vs[1], k0 + wk * KB, lds_v);
            }

            if (GEN) multiply_scores(s, sc);
            if (GEN && a.cap > 0.f) cap_scores<T>(s, sc, part);
#pragma unroll
            for (int x = 0; x < 3; ++x) {
                if (x >= axes) break;
                const int *q = px + x * KB + 4 * half;
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const int k = q[acc_row(e, 0)];        // (up to 2^32 apart)
                    s[e] = fmaf(-sl[x], (float)((uint32_t)max(k, pq[x]) - (uint32_t)min(k, pq[x])),
                                s[e]);
                }
            }
            if (part) {
                const int left = end - k0 - 4 * half;
#pragma unroll
                for (int e = 0; e < 16; ++e) s[e] = acc_row(e, 0) < left ? s[e] : kNegInf;
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
        if (__any(dropped) && lane == 0) *flag = 1;
    }
    l = halves_sum(l);

    __syncthreads();
    if (*flag) {
        // the wave's tiles again: infinities and NaN to the rows that see them
        for (int k0 = c0 + kw * KB; k0 < c1; k0 += wk * KB) {
            if (k0 + KB <= min(all, c1)) continue;
            for (int key = k0; key < min(k0 + KB, c1); ++key) {
                if (key >= end) continue;
#pragma unroll
                for (int d = 0; d < ND; ++d)
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const int x = d * 32 + acc_row(e, half);
                        float v = 0.f;
                        if (x < a.D) {
                            if constexpr (PLAIN) v = T::widen(vp[(int64_t)key * p.vs[1] + x]);
                            else
                                v = value_at<T, FMT>(vq + key * p.vs[1], vsc + key * p.vss[1], x);
                        }
                        if (!(fabsf(v) < __builtin_huge_valf())) o[d][e] += v;
                    }
            }
        }
    }

    // join the waves that have the same rows
    float *const jo = (float *)smem;                       // [NW][32][DP + pad]
    constexpr int JW = DP + kCachedPad;
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
    const int64_t total = (int64_t)a.B * a.Hq * a.Tq;
    const int slot = sp_no + (own ? c.part[0].nsplit : 0), stride = cached_stride(a.D);
    for (int x = tid; x < 32 * wr * (DP / 4); x += 64 * NW) {
        const int rr = x / (DP / 4), d = (x - rr * (DP / 4)) * 4;
        if (row0 + rr >= p.rows) break;
        if (d >= a.D) continue;
        const int first = (rr >> 5) * 32 + (rr & 31);      // row of the first such wave
        float mt = kNegInf;
        for (int w = 0; w < wk; ++w) mt = fmaxf(mt, ml[(w * wr * 32 + first) * 2]);
        const float ms = mt == kNegInf ? 0.f : mt;
        float lt = 0.f;
        f32x4 ot = f32x4(0.f);
        for (int w = 0; w < wk; ++w) {
            const int at = w * wr * 32 + first;
            const float f = __builtin_amdgcn_exp2f(ml[at * 2] - ms);
            lt = fmaf(f, ml[at * 2 + 1], lt);
            const f32x4 v = *(const f32x4 *)(jo + at * JW + d);
#pragma unroll
            for (int e = 0; e < 4; ++e) ot[e] = fmaf(f, v[e], ot[e]);
        }
        const int rg = row0 + rr, sq = rg / per, rest = rg - sq * per;
        const int64_t bb = cache * (int64_t)p.seqs + sq;
        if (slots > 1) {
            const int64_t at = slot * total + (bb * a.Hk + hk) * per + rest;
            *(f32x4 *)(a.part_o + at * stride + d) = ot;
            if (d == 0) *(float2 *)(a.part_ml + 2 * at) = make_float2(mt, lt);
        } else {
            const int tt = rest / a.G, hh = hk * a.G + rest - tt * a.G;
            R *out = (R *)a.out + ((bb * a.Tq + tt) * a.Hq + hh) * a.D + d;
            const float inv = lt == 0.f ? 0.f : 1.f / lt;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (d + e < a.D) out[e] = T::narrow(lt == 0.f ? 0.f : ot[e] * inv);
            if (d == 0)
                a.lse[(bb * a.Hq + hh) * a.Tq + tt] =
                    lt == 0.f ? kNegInf : (mt + log2f(lt)) * kLn2;
        }
    }
}

template <typename T, int FMT, int DP, int DU>
hipError_t run_cached(const CachedArgs &c, hipStream_t s)
{
    const dim3 grid((uint32_t)(c.part[0].blocks + c.part[1].blocks)), block(64 * kCachedWaves);
    if (attn_general(c.a))
        launch_kernel((attn_cached_kernel<T, FMT, DP, DU, true>), grid, block,
                      (cached_lds<T, DP>()), s, c);
    else
        launch_kernel((attn_cached_kernel<T, FMT, DP, DU, false>), grid, block,
                      (cached_lds<T, DP>()), s, c);
    return hipGetLastError();
}

template <typename T, int FMT>
hipError_t run_cached_width(const CachedArgs &c, hipStream_t s)
{
    if (c.a.D <= 64) return run_cached<T, FMT, 64, 64>(c, s);
    if (c.a.D <= 96) return run_cached<T, FMT, 128, 96>(c, s);
    return run_cached<T, FMT, 128, 128>(c, s);
}

// one translation unit a format
template <typename T>
hipError_t launch_cached_plain(const CachedArgs &c, hipStream_t s);
template <typename T>
hipError_t launch_cached_e4m3(const CachedArgs &c, hipStream_t s);
template <typename T>
hipError_t launch_cached_e2m1(const CachedArgs &c, hipStream_t s);

}  // namespace mp3d
