// What the kernels that walk the sequences of a paged cache share: a length as
// the table has room for it, and an even share of units (blocks, records) of all
// sequences and heads.  Internal to libw4.
#pragma once

#include "w4_kv.cuh"

#ifdef __CUDACC__
namespace w4 {

// Tokens of sequence b, `room` at most.
__device__ __forceinline__ int cached_len(const KvPool &pool, const int32_t *lens, int b,
                                          int room) {
    const int len = max(lens[b], 0);
    if (len <= room) return len;
    if (pool.error) atomicOr(pool.error, W4_KV_ERR_LENGTH);
    return room;
}

// The first record of a page of head h; NULL (and a bit of the error word) for a
// page that is not in the pool.
__device__ __forceinline__ char *page_records(const KvPool &pool, int page, int h,
                                              int record_bytes) {
    if (page < 0 || page >= pool.pages) {
        if (pool.error) atomicOr(pool.error, W4_KV_ERR_PAGE);
        return nullptr;
    }
    return pool.records +
           ((long long)page * pool.kv_heads + h) * pool.page_records * record_bytes;
}

// Worker w of W takes units start .. of the list (sequence, head, unit), `left`
// of them, one after another.  Sequence b has units(b) a head; the host refuses
// lists of 2^31.  A warp finds its start together: lane i adds up a 32nd of the
// sequences.
struct Share {
    int b, h, u, n;     // unit u of n
    int left;

    Share() = default;
    template <class Units>
    __device__ __forceinline__ Share(const Units &units, int seqs, int heads, int w, int W) {
        const int lane = threadIdx.x & 31, each = (seqs + 31) >> 5;
        const int b0 = min(lane * each, seqs), b1 = min(b0 + each, seqs);
        int mine = 0;
#pragma unroll 4
        for (int x = b0; x < b1; ++x) mine += units(x);
        int upto = mine;
#pragma unroll
        for (int x = 1; x < 32; x <<= 1) {
            const int v = __shfl_up_sync(0xFFFFFFFFu, upto, x);
            if (lane >= x) upto += v;
        }
        const int all = __shfl_sync(0xFFFFFFFFu, upto, 31) * heads;
        const int start = (int)((long long)all * w / W);
        left = (int)((long long)all * (w + 1) / W) - start;
        int in = start - (upto - mine) * heads;
        const bool here = in >= 0 && in < mine * heads;
        b = b0, n = 1;
        if (here)
            for (;; ++b) {
                n = units(b);
                if (in < n * heads) break;
                in -= n * heads;
            }
        const unsigned found = __ballot_sync(0xFFFFFFFFu, here);
        const int src = found ? __ffs(found) - 1 : 0;
        b = __shfl_sync(0xFFFFFFFFu, b, src);
        n = __shfl_sync(0xFFFFFFFFu, n, src);
        in = __shfl_sync(0xFFFFFFFFu, in, src);
        if (!found) left = 0;                                 // there is no unit at all
        h = in / n, u = in - h * n;
    }

    // Unit `w` of a list in which every sequence has `most` units a head, if it is
    // there: for grids that have a worker for each.
    template <class Units>
    __device__ __forceinline__ static Share one(const Units &units, int seqs, int heads, int most,
                                                int w) {
        Share s;
        const int row = w / most;
        s.u = w - row * most, s.b = row / heads, s.h = row - s.b * heads, s.n = most;
        s.left = s.b < seqs && s.u < units(s.b) ? 1 : 0;
        return s;
    }

    // `k` units on.
    template <class Units>
    __device__ __forceinline__ void next(const Units &units, int heads, int k = 1) {
        left -= k, u += k;
        while (u >= n && left > 0) {
            u -= n;
            if (++h < heads) continue;
            h = 0;
            do n = units(++b);                                // left > 0: there is one
            while (n == 0);
        }
    }
};

}  // namespace w4
#endif
