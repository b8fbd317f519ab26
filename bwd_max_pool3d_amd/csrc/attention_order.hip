// attention_order.hip -- packed documents make blocks of queries (and of
// keys) of very different length: the longest first, or the last of them
// would run on an almost idle card.  One small workgroup per sequence ranks
// the blocks by the keys (queries) they walk; the attention kernels look
// their block up.  On 8192 tokens in 9 documents of 178 to 1605, 16 heads of
// 64 with a distance bias, the three kernels take 125, 137 and 208 us with it
// and 168, 184 and 266 without; the ranking takes 4.5 us forward, 13
// backward.  Up to kOrderMax blocks (one thread each); beyond that there are
// so many that the last ones no longer count.
#include "attention.hpp"

namespace mp3d {

namespace {

// Position of entry t of n works in descending order (ties by number).
__device__ __forceinline__ int rank_of(const int *work, int n, int t)
{
    const int w = work[t];
    int r = 0;
    for (int i = 0; i < n; ++i) r += work[i] > w || (work[i] == w && i < t);
    return r;
}

__global__ __launch_bounds__(kOrderMax) void attn_order_kernel(AttnArgs a, int backward)
{
    __shared__ int work[kOrderMax];
    const int b = blockIdx.x, t = threadIdx.x;
    const int nq = (a.Tq + kAttnRows - 1) / kAttnRows, nk = (a.Tk + kAttnRows - 1) / kAttnRows;
    if (a.order_q) {
        if (t < nq) {
            const Span x = row_span(a, b, t * kAttnRows);
            const Span y = row_span(a, b, min((t + 1) * kAttnRows, a.Tq) - 1);
            const int lo = x.hi > x.lo ? x.lo : y.lo, hi = max(x.hi, y.hi);
            work[t] = hi - lo;
        }
        __syncthreads();
        if (t < nq) a.order_q[(int64_t)b * nq + rank_of(work, nq, t)] = t;
    }
    if (backward && a.order_k) {
        __syncthreads();
        if (t < nk) {
            // the first query whose keys end past the block's start, and the
            // first whose keys start past its end (both grow with the query)
            const int k0 = t * kAttnRows;
            const int64_t row = (int64_t)b * a.Tq;
            int i = 0, j = a.Tq;
            while (i < j) {
                const int m = (i + j) >> 1;
                if (a.spans[2 * (row + m) + 1] > k0) j = m;
                else i = m + 1;
            }
            int p = i, e = a.Tq;
            while (p < e) {
                const int m = (p + e) >> 1;
                if (a.spans[2 * (row + m)] >= k0 + kAttnRows) e = m;
                else p = m + 1;
            }
            work[t] = p - i;
        }
        __syncthreads();
        if (t < nk) a.order_k[(int64_t)b * nk + rank_of(work, nk, t)] = t;
    }
}

}  // namespace

// Bytes of the order of the queries' blocks (and the keys', backward); 0
// where blocks are alike, too many to need one, or walk nothing: without
// queries nothing ranks the keys' blocks, and they go by number.
int64_t attn_order_bytes(const AttnArgs &a, bool keys)
{
    const int64_t n = ((keys ? a.Tk : a.Tq) + kAttnRows - 1) / kAttnRows;
    return a.docs && a.Tq > 0 && n > 1 && n <= kOrderMax ? (n * a.B * 4 + 15) / 16 * 16 : 0;
}

void launch_attn_order(const AttnArgs &a, bool backward, hipStream_t s)
{
    if (a.order_q || (backward && a.order_k))
        launch_kernel(attn_order_kernel, dim3((uint32_t)a.B), dim3(kOrderMax), 0, s, a,
                      (int)backward);
}

}  // namespace mp3d
