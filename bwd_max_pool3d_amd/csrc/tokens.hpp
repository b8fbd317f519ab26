// tokens.hpp -- launch plans and launchers of the token operators (rotary
// positions, attention, gated norm), shared by their C ABI layer
// (api_tokens.hip) and the kernel translation units.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "kernels.hpp"

namespace mp3d {

// --- rotary positions (rope.hip)
struct RopePlan {
    const void *src[2];        // q, k
    void *dst[2];
    int64_t ss[2][3], ds[2][3];  // strides in elements: batch, token, head
    int32_t heads[2];          // k: 0 when there is none
    const int32_t *pos;        // (3, B, T), or NULL: token t is cell t of the grid
    const float *freq;         // (P)
    int64_t B, T;
    int32_t D, P;
    int32_t e0, e1;            // pairs [0, e0) turn by the first axis, [e0, e1) by the second
    int32_t gh, gw;
    int32_t interleaved;
    float sign;                // +1 forward, -1 backward
    int32_t vec;               // elements per vector access (divides every offset): 8, 4, 2 or 1
    int32_t units;             // threads per token: pair vectors, then untouched channels
    int32_t rot_units;
    int32_t tpb;               // tokens per workgroup
    int32_t hpt;               // heads per thread
};
void plan_rope_heads(RopePlan *p);         // heads per thread
template <typename T>
hipError_t launch_rope(const RopePlan &p, hipStream_t s);

// --- gated norm (gated_norm.hip)
constexpr int kNormMaxC = 16384;
struct NormPlan {
    const void *x, *h, *gate, *post, *pre;
    void *y, *z;               // forward
    float *stats;              // (rows, 4): mean and 1/deviation of h, then of y
    const void *dy, *dz;       // backward
    void *dx, *dh;
    float *dgate, *dpost, *dpre;
    float *part;               // workspace: (nwg, 3, C) sums of dpost, dpre, dgate
    int64_t rows;
    int64_t gate_rows;         // 0: no gate
    int64_t rpg;               // rows per gate row
    int32_t C;
    float rs, eps;             // residual scale
    int32_t layer, has_post, has_pre;
    int32_t vec;               // 16-byte accesses possible
    int32_t threads;           // threads per row: 64 to 1024
    int32_t ept;               // elements per thread: 8 or 16
    // backward: workgroups walk groups of rows that share a gate row
    int64_t groups;            // gate rows (1 without a gate)
    int32_t wpg;               // workgroups per group
    int32_t nwg;
};
// threads, ept and vec from C, the element size and the pointers' alignment
void plan_norm(NormPlan *p, int es, bool aligned16);
// the backward's threads and ept, groups, wpg and nwg; returns the workspace bytes
size_t plan_norm_backward(NormPlan *p);
template <typename T>
hipError_t launch_norm_forward(const NormPlan &p, hipStream_t s);
template <typename T>
hipError_t launch_norm_backward(const NormPlan &p, hipStream_t s);
// zeros to dgate, dpost and dpre, where they are given
hipError_t launch_norm_no_rows(const NormPlan &p, hipStream_t s);

// --- attention (attention_*.hip)
constexpr int kAttnMaxD = 128;
constexpr int kAttnRows = 128;             // queries (keys, for dk and dv) of a workgroup
constexpr int kOrderMax = 512;             // blocks of a sequence that are ordered by length
struct AttnArgs {
    const void *q, *k, *v;
    void *out;                 // (B, Tq, Hq, D)
    float *lse;                // (B, Hq, Tq)
    const void *dout;          // backward
    void *dq, *dk, *dv;        // contiguous (B, T, H, D)
    int64_t qs[3], ks[3], vs[3], gs[3];  // strides of q, k, v, dout: batch, token, head
    int32_t B, Tq, Tk, Hq, Hk, G, D;     // G = Hq / Hk query heads share a key head
    float scale, cap;
    const float *slopes;       // (Hq, axes), with pos_q (axes, B, Tq), pos_k (axes, B, Tk)
    const int32_t *pos_q, *pos_k;
    int32_t axes;
    int32_t causal, ndocs;
    const int32_t *docs, *prefix, *kv_len;
    int32_t vec;               // every row of q, k, v (and dout) starts at a multiple of 16 bytes
    int32_t *order_q, *order_k;  // (B, blocks): blocks by falling length, or NULL
    // split form: rows of one key head (Tq * G) in blocks of 32, keys in chunks
    int32_t nrb, nsplit, chunk;
    float *part_o;             // (nsplit, B, Hk, Tq * G, D) sums, unnormalised
    float *part_ml;            // (nsplit, B, Hk, Tq * G, 2) maximum and sum
    // backward: a key head's query heads in gsplit parts
    int32_t gsplit;
    float *rowd;               // (B, Hq, Tq, 2): lse * log2 e, and -delta
    int32_t *spans;            // (B, Tq, 2): the keys [lo, hi) of each query
    int32_t *tiles;            // (B, ceil(Tq / 32), 4): over 32 queries, the union of
                               // their keys [lo, hi) and the keys all of them see
    uint32_t *parts_q, *parts_k;  // (axes, B, Tq, 2) and (axes, B, Tk, 2): positions in parts of
                                  // 8 bits
    int32_t *fars;             // (B, ceil(Tq / 32), 2): is a position 2^24 or more among these 32
                               // queries, among this share of the keys (with a bias)
    float *part_dk, *part_dv;  // (gsplit, B, Tk, Hk, D), when gsplit > 1
    // backward in float16 (attention_bwd.hip, range): |do|_1 of each query, the
    // largest of each 32, and the largest finite |v| of a workgroup's share of the
    // keys
    int32_t f16;
    float *norms;              // (B, Hq, Tq)
    float *norm_most, *v_most; // (B, Hq, ceil(Tq / 32)) each (of v a key head's first value_parts)
};
// Scores with a cap, a bias or a factor that is not positive: kernels of
// their own, whose registers the plain ones do not carry.
inline bool attn_general(const AttnArgs &a)
{
    return a.cap > 0.f || a.axes > 0 || !(a.scale > 1e-30f);
}
int64_t attn_order_bytes(const AttnArgs &a, bool keys);
void launch_attn_order(const AttnArgs &a, bool backward, hipStream_t s);
bool attn_split_wanted(const AttnArgs &a, bool f32);
// nrb, nsplit and chunk; returns the workspace bytes
size_t plan_attn_split(AttnArgs *a);
void place_attn_split(AttnArgs *a, void *workspace);
// gsplit; returns the workspace bytes
size_t plan_attn_backward(AttnArgs *a);
void place_attn_backward(AttnArgs *a, void *workspace);
template <typename T>
hipError_t launch_attn_backward(const AttnArgs &a, hipStream_t s);
template <typename T>
hipError_t launch_attn_forward(const AttnArgs &a, hipStream_t s);
template <typename T>
hipError_t launch_attn_split(const AttnArgs &a, hipStream_t s);

// --- caches in 8 or 4 bits (cache.hip), strides in bytes: sequence, token, head
struct CachePlan {
    const void *x[2];          // k, v (the read writes them, contiguous (B, T, H, D))
    int64_t xs[2][3];          // their strides in elements (write)
    uint8_t *codes[2], *scales[2];
    int64_t cs[2][3], ss[2][3];
    const int32_t *start, *count;  // (B) each, or NULL: 0 and T
    int64_t rows;              // of a sequence's cache
    int32_t B, T, H, D;
    int32_t format, vec;
    int32_t pieces, threads;   // threads of a row, of a workgroup
    int32_t per, tiles;        // tokens of a workgroup, workgroups of a sequence
};
constexpr int kCacheMaxD = 1024;
void plan_cache(CachePlan *p, int elem_bytes, bool read);
template <typename T>
hipError_t launch_cache(const CachePlan &p, bool read, hipStream_t s);

// --- attention over caches (attention_cached.hip): a prefix for every S
// sequences, and a cache of each sequence's own
struct CachedPart {
    const void *k, *v;         // elements, or codes
    const uint8_t *k_scale, *v_scale;
    int64_t ks[3], vs[3];      // strides in elements (bytes of codes): cache, token, head
    int64_t kss[3], vss[3];    // and of the scales, in bytes
    const int32_t *len;        // tokens in use of each cache, or NULL: T
    const int32_t *pos;        // (axes, caches, T)
    int32_t T, caches;
    int32_t seqs;              // sequences of a cache
    int32_t width;             // bytes that a load may take: 16, 8, 4, 2 or 1
    int32_t rows;              // seqs * Tq * G, of a key head
    int32_t mb;                // rows of a wave: 16 or 32
    int32_t wr;                // waves with rows of their own (4 / wr share the keys out)
    int32_t nrb, nsplit, chunk;  // blocks of mb wr rows, chunks of keys
    int64_t units, blocks;     // (cache, key head, chunk)s, workgroups
};
struct CachedArgs {
    AttnArgs a;                // q, the scores, out and lse, the parts
    CachedPart part[2];        // the prefix, the own caches
    int32_t format, f32;
    int32_t any;               // rows of any alignment and strides: kernels of their own
    int32_t any_strides;       // the same, whatever the rows' addresses
};
size_t plan_attn_cached(CachedArgs *c, int cus);
void place_attn_cached(CachedArgs *c, void *workspace);
template <typename T>
hipError_t launch_attn_cached(const CachedArgs &c, hipStream_t s);

}  // namespace mp3d
