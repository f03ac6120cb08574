// Blocks of the paged cache: bounds of their keys (w4_key_bounds) and what q . k
// can be in them (w4_block_scores).
//
// With hi_d >= k_d >= lo_d for every key of a block, q_d k_d <= q_d hi_d where q_d >= 0
// and <= q_d lo_d elsewhere, so the sum of those bounds q . k whatever the key is.
// That is one product of 2 D values, (q+, q-) . (hi, lo), and goes to the tensor cores
// with 16 blocks as its rows and 8 rows of queries as its columns.
//
// Roundings.  Bounds are bfloat16, half the bytes of fp32 for a score that only ranks
// blocks: exact for a bf16 cache; of a quantised key, (q - z) s rounded to nearest as it
// is read back, so a product with the unrounded key may pass the bound by 2^-9 of its
// terms.  A score's products are exact and its sum is fp32.
//
// Both kernels move little and are a chain of trips to memory (length, page, bounds or
// keys).  What counts is how few trips there are and how many warps make them at a
// time: while there are few units, each has a worker of its own that needs no sum over
// the lengths.  Measured, captured calls: bounds of one step of 64 sequences 3.5 us
// (each worker summing the lengths first, a warp a block of 64 tokens: 4.9), of 16384
// tokens in 8 bits 4.8 us (8.2; a copy's rate is 1.4), of 16 such prompts in bf16 63 us
// (a copy's rate 41), in 8 and 4 bits, where the conversion of the codes sets the time,
// 60 and 67 (22 and 12); scores of 64 ragged sequences of up to 512 blocks 9.5 us (11.5;
// a copy's rate 5.1: two rounds of 16 warps an SM), of 8 x 8192 blocks 24.7 us = 82 % of a
// copy's rate.  With hi and lo one after the other in 64 registers, and twice as many
// warps, these two took 9.4 and 26.7 us (9.8 and 25.0 then), 8 new tokens 18.6 (17.1): not
// kept.
#include "w4_device.cuh"
#include "w4_kv_work.cuh"

namespace w4 {
namespace {

constexpr int kBlockWarps = 4;
constexpr int kDirectBlocks = 32;      // blocks an SM up to which units have one worker each

// Blocks of a sequence that hold its last tokens, and the first of them.
struct Touched {
    KvPool pool;
    const int32_t *lens;
    int tokens;

    __device__ __forceinline__ int len(int b) const {
        return cached_len(pool, lens, b, pool.width * pool.page_tokens);
    }
    __device__ __forceinline__ int first(int n) const {
        return max(n - tokens, 0) / pool.page_tokens;
    }
    __device__ __forceinline__ int operator()(int b) const {
        const int n = len(b);
        return n ? (n - 1) / pool.page_tokens - first(n) + 1 : 0;
    }
};

__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// 16 neighbouring values of one key as they are stored.
template <int FMT>
struct Raw {
    uint32_t w[FMT == W4_KV_BF16 ? 8 : FMT == W4_KV_INT8 ? 4 : 2];
    uint32_t meta;
};

// PARTS warps take a block of a head, every PARTS-th record each, and a key's
// values D / 16 lanes, 16 each, so that every load is 16 bytes (8 in 4 bits) of whole
// rows.
template <int FMT, int D, int PARTS>
__global__ void __launch_bounds__(32 * kBlockWarps)
bounds_kernel(const Touched touched, uint32_t *bounds, int most) {
    using L = KvLayout<FMT, D>;
    constexpr int LANES = D / 16, ROWS = 32 / LANES, LOADS = kRecTokens / ROWS;
    constexpr int UNITS = kBlockWarps / PARTS;
    __shared__ uint4 joined[UNITS][PARTS][4][LANES];
    begin_after_previous();
    const KvPool &pool = touched.pool;
    const int lane = threadIdx.x & 31, part = lane % LANES, row0 = lane / LANES;
    const int warp = threadIdx.x >> 5, mine = warp % PARTS, unit = warp / PARTS;
    Share s = most ? Share::one(touched, pool.seqs, pool.kv_heads, most,
                                blockIdx.x * UNITS + unit)
                   : Share(touched, pool.seqs, pool.kv_heads, blockIdx.x * UNITS + unit,
                           gridDim.x * UNITS);
    for (; s.left > 0; s.next(touched, pool.kv_heads)) {
        const int len = touched.len(s.b), block = touched.first(len) + s.u;
        const int page = pool.table[s.b * pool.stride + block];
        const char *rec = page_records(pool, page, s.h, L::kBytes);
        if (!rec) continue;
        const int there = min(len - block * pool.page_tokens, pool.page_tokens);
        uint32_t hi[8], lo[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) hi[i] = 0xFF80FF80u, lo[i] = 0x7F807F80u;
        rec += mine * L::kBytes;
        for (int r0 = mine * kRecTokens; r0 < there;
             r0 += PARTS * kRecTokens, rec += PARTS * L::kBytes) {
            Raw<FMT> raw[LOADS];
#pragma unroll
            for (int x = 0; x < LOADS; ++x) {
                const int r = row0 + x * ROWS;
                if constexpr (FMT == W4_KV_BF16) {
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const uint4 v = *reinterpret_cast<const uint4 *>(
                            rec + L::key(r, 16 * part + 8 * y));
                        raw[x].w[4 * y] = v.x, raw[x].w[4 * y + 1] = v.y;
                        raw[x].w[4 * y + 2] = v.z, raw[x].w[4 * y + 3] = v.w;
                    }
                } else {
                    if constexpr (FMT == W4_KV_INT8) {
                        const uint4 v =
                            *reinterpret_cast<const uint4 *>(rec + L::key(r, 16 * part));
                        raw[x].w[0] = v.x, raw[x].w[1] = v.y, raw[x].w[2] = v.z, raw[x].w[3] = v.w;
                    } else {
                        const uint2 v =
                            *reinterpret_cast<const uint2 *>(rec + L::key(r, 16 * part));
                        raw[x].w[0] = v.x, raw[x].w[1] = v.y;
                    }
                    raw[x].meta = *reinterpret_cast<const uint32_t *>(rec + L::kMeta + 4 * r);
                }
            }
#pragma unroll
            for (int x = 0; x < LOADS; ++x) {
                if (r0 + row0 + x * ROWS >= there) continue;
                uint32_t v[8];
                if constexpr (FMT == W4_KV_BF16) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[i] = raw[x].w[i];
                } else {
                    // (q - z) s is exact in fp32, and so is the difference below
                    const float sc = __half2float(
                        __ushort_as_half((unsigned short)(raw[x].meta & 0xFFFFu)));
                    const float off = -(float)(raw[x].meta >> 16) * sc;
                    const auto value = [&](int i) {
                        const uint32_t q =
                            FMT == W4_KV_INT8 ? raw[x].w[i >> 2] >> (8 * (i & 3)) & 255u
                                              : raw[x].w[i >> 3] >> (4 * (i & 7)) & 15u;
                        return fmaf((float)q, sc, off);
                    };
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[i] = bf16_pair(value(2 * i), value(2 * i + 1));
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) hi[i] = max2(hi[i], v[i]), lo[i] = min2(lo[i], v[i]);
            }
        }
#pragma unroll
        for (int x = LANES; x < 32; x <<= 1)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                hi[i] = max2(hi[i], __shfl_xor_sync(0xFFFFFFFFu, hi[i], x));
                lo[i] = min2(lo[i], __shfl_xor_sync(0xFFFFFFFFu, lo[i], x));
            }
        // the largest from the first lanes, the smallest from the next ones
        if constexpr (PARTS > 1) {
            const auto sync = [&]() {                         // of the block's warps
                asm volatile("bar.sync %0, %1;" ::"r"(1 + unit), "n"(32 * PARTS) : "memory");
            };
            if (row0 == 0) {
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    joined[unit][mine][y][part] =
                        make_uint4(hi[4 * y], hi[4 * y + 1], hi[4 * y + 2], hi[4 * y + 3]);
                    joined[unit][mine][2 + y][part] =
                        make_uint4(lo[4 * y], lo[4 * y + 1], lo[4 * y + 2], lo[4 * y + 3]);
                }
            }
            sync();
            if (mine == 0 && row0 < 2) {
#pragma unroll
                for (int x = 1; x < PARTS; ++x)
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const uint4 a = joined[unit][x][y][part], b = joined[unit][x][2 + y][part];
                        hi[4 * y] = max2(hi[4 * y], a.x), hi[4 * y + 1] = max2(hi[4 * y + 1], a.y);
                        hi[4 * y + 2] = max2(hi[4 * y + 2], a.z);
                        hi[4 * y + 3] = max2(hi[4 * y + 3], a.w);
                        lo[4 * y] = min2(lo[4 * y], b.x), lo[4 * y + 1] = min2(lo[4 * y + 1], b.y);
                        lo[4 * y + 2] = min2(lo[4 * y + 2], b.z);
                        lo[4 * y + 3] = min2(lo[4 * y + 3], b.w);
                    }
            }
            sync();                                           // joined is free again
        }
        if (mine == 0 && row0 < 2) {
            uint4 *out = reinterpret_cast<uint4 *>(
                bounds + ((long long)page * pool.kv_heads + s.h) * D + row0 * (D / 2) + 8 * part);
#pragma unroll
            for (int y = 0; y < 2; ++y)
                out[y] = row0 ? make_uint4(lo[4 * y], lo[4 * y + 1], lo[4 * y + 2], lo[4 * y + 3])
                              : make_uint4(hi[4 * y], hi[4 * y + 1], hi[4 * y + 2], hi[4 * y + 3]);
        }
    }
}

// Tiles of 16 blocks of a sequence.
struct Tiles {
    KvPool pool;
    const int32_t *lens;

    __device__ __forceinline__ int len(int b) const {
        return cached_len(pool, lens, b, pool.width * pool.page_tokens);
    }
    __device__ __forceinline__ int blocks(int len) const {
        return (len + pool.page_tokens - 1) / pool.page_tokens;
    }
    __device__ __forceinline__ int operator()(int b) const { return (blocks(len(b)) + 15) / 16; }
};

// q+ . hi + q- . lo on the tensor cores: 16 blocks are the rows of a tile, 8 rows
// of queries its columns, and the sum runs over 2 D values.  Which of them a
// lane holds in which register does not matter as long as both sides agree, so
// lane t takes the 16-byte pieces t, t + 4, ... of a row as they lie in memory.
template <int D>
__global__ void __launch_bounds__(32 * kBlockWarps)
scores_kernel(const Tiles tiles, const uint4 *bounds, const Heads q, int group,
              unsigned group_magic, int tokens, float *scores, int columns, int most) {
    constexpr int PIECES = D / 32;
    begin_after_previous();
    const KvPool &pool = tiles.pool;
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int rows = tokens * group;
    const int w = blockIdx.x * kBlockWarps + (threadIdx.x >> 5);
    Share s = most ? Share::one(tiles, pool.seqs, pool.kv_heads, most, w)
                   : Share(tiles, pool.seqs, pool.kv_heads, w, gridDim.x * kBlockWarps);
    for (; s.left > 0; s.next(tiles, pool.kv_heads)) {
        const int len = tiles.len(s.b), blocks = tiles.blocks(len);
        uint4 a[2][2][PIECES];                                // hi, lo of blocks g, g + 8
        bool there[2], valid[2];
        int page[2];
#pragma unroll
        for (int y = 0; y < 2; ++y) {
            const int block = 16 * s.u + g + 8 * y;
            there[y] = block < blocks;
            page[y] = there[y] ? pool.table[s.b * pool.stride + block] : -1;
        }
        // (ordinary loads: what they read may still be written when this kernel starts)
#pragma unroll
        for (int y = 0; y < 2; ++y) {
            valid[y] = page[y] >= 0 && page[y] < pool.pages;
            const uint4 *row =
                bounds + ((long long)(valid[y] ? page[y] : 0) * pool.kv_heads + s.h) * (D / 4) + t;
#pragma unroll
            for (int z = 0; z < 2; ++z)
#pragma unroll
                for (int j = 0; j < PIECES; ++j)
                    a[z][y][j] = valid[y] ? row[z * (D / 8) + 4 * j] : make_uint4(0u, 0u, 0u, 0u);
        }
        if (pool.error && ((there[0] && !valid[0]) || (there[1] && !valid[1])))
            atomicOr(pool.error, W4_KV_ERR_PAGE);
        float best[2] = {-INFINITY, -INFINITY};
        // (two rounds together: 8 new tokens 16.9 us, 18.2 one by one)
#pragma unroll 2
        for (int r0 = 0; r0 < rows; r0 += 8) {
            const int r = min(r0 + g, rows - 1);
            const int i = group == 1 ? r : (int)__umulhi((unsigned)r, group_magic);
            const uint4 *row = reinterpret_cast<const uint4 *>(
                reinterpret_cast<const __nv_bfloat16 *>(q.data) +
                (long long)(s.b * tokens + i) * q.token_stride +
                (long long)(s.h * group + r - i * group) * q.head_stride) + t;
            uint4 piece[PIECES];                              // all under way together
#pragma unroll
            for (int j = 0; j < PIECES; ++j) piece[j] = row[4 * j];
            // (two sums: half as many products wait for one another, and each rounds less)
            float d[4] = {0.f, 0.f, 0.f, 0.f}, e[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int j = 0; j < PIECES; ++j) {
                const uint4 v = piece[j];
                const uint4 up = make_uint4(max2(v.x, 0u), max2(v.y, 0u), max2(v.z, 0u),
                                            max2(v.w, 0u));
                const uint4 down = make_uint4(min2(v.x, 0u), min2(v.y, 0u), min2(v.z, 0u),
                                              min2(v.w, 0u));
#pragma unroll
                for (int z = 0; z < 2; ++z) {
                    const uint4 &k0 = a[z][0][j], &k1 = a[z][1][j], &b = z ? down : up;
                    mma_bf16_16816(d, k0.x, k1.x, k0.y, k1.y, b.x, b.y);
                    mma_bf16_16816(e, k0.z, k1.z, k0.w, k1.w, b.z, b.w);
                }
            }
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                // (columns past the last row repeat it)
                const int rc = min(r0 + 2 * t + (c & 1), rows - 1);
                const int ic = group == 1 ? rc : (int)__umulhi((unsigned)rc, group_magic);
                const float sum = d[c] + e[c], v = fabsf(sum) < INFINITY ? sum : INFINITY;
                if (len - tokens + ic >= 0) best[c >> 1] = fmaxf(best[c >> 1], v);
            }
        }
#pragma unroll
        for (int y = 0; y < 2; ++y) {
            best[y] = fmaxf(best[y], __shfl_xor_sync(0xFFFFFFFFu, best[y], 1));
            best[y] = fmaxf(best[y], __shfl_xor_sync(0xFFFFFFFFu, best[y], 2));
            const int block = 16 * s.u + g + 8 * y;
            if (t == 0 && block < blocks)
                scores[((long long)s.b * pool.kv_heads + s.h) * columns + block] =
                    valid[y] ? best[y] : -INFINITY;
        }
    }
}

// The blocks of a launch for at most `most` units a head, `each` of them a block.  A
// worker for every unit that there could be while they are few: it finds its own
// without adding up all sequences' lengths, and those without one end at once.  With
// more, as where tables are much wider than the sequences, as many as the device
// holds share the units that there are (*most = 0).
int grid_of(const KvPool &pool, int *most, int each, int num_sms) {
    const long long units = (long long)*most * pool.seqs * pool.kv_heads;
    const long long blocks = (units + each - 1) / each;
    if (blocks <= (long long)kDirectBlocks * num_sms) return (int)blocks;
    *most = 0;
    return 4 * num_sms;
}

template <int FMT, int D, int PARTS>
cudaError_t launch_bounds(const Touched &touched, void *bounds, int most, int num_sms,
                          cudaStream_t stream) {
    const int grid = grid_of(touched.pool, &most, kBlockWarps / PARTS, num_sms);
    return launch_overlapped(bounds_kernel<FMT, D, PARTS>, dim3(grid), dim3(32 * kBlockWarps), 0,
                             stream, touched, static_cast<uint32_t *>(bounds), most);
}

template <int FMT, int D>
cudaError_t launch_parts(const Touched &touched, void *bounds, int most, int num_sms,
                         cudaStream_t stream) {
    const int records = touched.pool.page_records;
    return records >= 4   ? launch_bounds<FMT, D, 4>(touched, bounds, most, num_sms, stream)
           : records >= 2 ? launch_bounds<FMT, D, 2>(touched, bounds, most, num_sms, stream)
                          : launch_bounds<FMT, D, 1>(touched, bounds, most, num_sms, stream);
}

}  // namespace

cudaError_t launch_key_bounds(const KvPool &pool, int format, int head_dim, void *bounds,
                              int tokens, const int32_t *lens, int num_sms,
                              cudaStream_t stream) {
    const Touched touched = {pool, lens, tokens};
    const long long reach = ((long long)tokens + pool.page_tokens - 2) / pool.page_tokens + 1;
    const int most = (int)(reach < pool.width ? reach : pool.width);
    const auto run = [&](auto f) { return f(touched, bounds, most, num_sms, stream); };
    if (head_dim == 128)
        return format == W4_KV_BF16   ? run(launch_parts<W4_KV_BF16, 128>)
               : format == W4_KV_INT8 ? run(launch_parts<W4_KV_INT8, 128>)
                                      : run(launch_parts<W4_KV_INT4, 128>);
    return format == W4_KV_BF16   ? run(launch_parts<W4_KV_BF16, 64>)
           : format == W4_KV_INT8 ? run(launch_parts<W4_KV_INT8, 64>)
                                  : run(launch_parts<W4_KV_INT4, 64>);
}

cudaError_t launch_block_scores(const KvPool &pool, int head_dim, const void *bounds,
                                const Heads &q, int group, unsigned group_magic, int tokens,
                                const int32_t *lens, float *scores, int columns, int num_sms,
                                cudaStream_t stream) {
    const Tiles tiles = {pool, lens};
    int most = (pool.width + 15) / 16;
    const int grid = grid_of(pool, &most, kBlockWarps, num_sms);
    const auto run = [&](auto kernel) {
        return launch_overlapped(kernel, dim3(grid), dim3(32 * kBlockWarps), 0, stream, tiles,
                                 static_cast<const uint4 *>(bounds), q, group, group_magic,
                                 tokens, scores, columns, most);
    };
    return head_dim == 128 ? run(scores_kernel<128>) : run(scores_kernel<64>);
}

}  // namespace w4
