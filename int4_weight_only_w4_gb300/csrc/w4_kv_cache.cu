// The paged key-value cache: writing tokens (w4_kv_append: rotation of q and
// k, quantisation, the record layout) and reading them back (w4_kv_read).
//
// Mathematics of a (token, head) group: w4_quantize's asymmetric rule with
// Q = 255 or 15 levels (include/w4.h), every operation rounded to nearest in
// fp32, so the codes are those of any other evaluation of the rule bit for bit.
//
// A block takes a tile of up to 16 listed tokens and one key/value head, cut so
// that the tokens of a sequence in order fall into whole records.  Such a
// record is put together (or taken apart) in shared memory and moved with
// 16-byte accesses; the values' layout scatters a token over 64 sectors, so
// moving it byte by byte would cost up to 16 times the traffic.  Tiles that are
// no whole record (decode steps, the ends of a prompt, tokens in another
// order) go byte by byte, straight to the cache.
#include "w4_kv.cuh"

namespace w4 {
namespace {

constexpr int kKvThreads = 128, kKvWarps = kKvThreads / 32;

// The tile's tokens: list indexes i0 .. i0 + 15 of which [lo, hi) are there.
struct Tile16 {
    long long page_record[kRecTokens];
    int in_page[kRecTokens];
    int position[kRecTokens];
    int valid[kRecTokens];
};

// Fills the tile of this block; returns the list index of its token 0, or a
// negative number's worth of nothing: `count` is 0 when no token is there.
// whole: the tokens are one record.  All threads call.
__device__ __forceinline__ int load_tile(const KvPool &pool, const TokenList &list, int tile_no,
                                         int tiles, int rotation_rows, Tile16 *tile, int *first, int *count,
                                         bool *whole) {
    const int b = tile_no / tiles, j = tile_no - b * tiles;
    const int base = b * list.run;
    const int shift = list.positions[base] & (kRecTokens - 1);
    const int i0 = j * kRecTokens - shift;
    *first = max(0, -i0);
    *count = min(kRecTokens, list.run - i0) - *first;
    if (*count <= 0) return 0;
    const int r = threadIdx.x;
    if (r < kRecTokens) {
        TokenPlace at = {};
        const bool there = r >= *first && r < *first + *count;
        // (one block of a tile's heads records what is out of range)
        const bool ok = there && kv_place(pool, list, base + i0 + r, rotation_rows, &at);
        tile->valid[r] = ok;
        tile->in_page[r] = at.in_page;
        tile->position[r] = at.position;
        tile->page_record[r] = at.page_record;
    }
    __syncthreads();
    bool same = true;
    if (r < kRecTokens)
        same = tile->valid[r] && tile->page_record[r] == tile->page_record[0] &&
               tile->in_page[r] == tile->in_page[0] + r && tile->in_page[0] % kRecTokens == 0;
    *whole = __syncthreads_and(same);
    return base + i0;
}

__device__ __forceinline__ float clampf(float v, float a, float b) {
    return fminf(fmaxf(v, a), b);
}

// rint(w / s) for the correctly rounded quotient (NaN: 0), with r = rcp_rn(s)
// and tol = T * 2^-21, T >= |w r|: w r is within 2^-22.4 of the quotient's
// magnitude, so the two round alike unless w r lies that close to a half; there
// the division decides.
__device__ __forceinline__ float rint_quotient(float w, float s, float r, float tol) {
    const float t = __fmul_rn(w, r), n = rintf(t);
    if (0.5f - fabsf(__fsub_rn(t, n)) > tol) return n;
    const float q = rintf(__fdiv_rn(w, s));
    return q == q ? q : 0.f;
}

// The queries of a launch of append_kernel, turned as by w4_rope in blocks of
// their own (in the rows' loop below every lane would turn its partner too:
// 16 k tokens of 28 query heads 146 us against 84).
struct Queries {
    Heads q, out;
    int heads;
    unsigned groups, units;    // see turn_unit
    unsigned all;              // tokens * groups * units
    unsigned first_block;      // blocks from here on turn queries
};

// Keys and values: D / 8 lanes take a row (a head of a token), 8 values a lane;
// a warp takes the key and value of 128 / D tokens at a time.
template <int FMT, int D, int HEADS>
__global__ void __launch_bounds__(kKvThreads)
append_kernel(KvPool pool, Heads k, Heads v, Queries q, TokenList list, Rotation rot, int tiles) {
    using L = KvLayout<FMT, D>;
    constexpr int LANES = D / 8, TOKENS = 16 / LANES;
    __shared__ Tile16 tile;
    __shared__ __align__(16) unsigned char staged[L::kBytes];
    begin_after_previous();
    if (blockIdx.x >= q.first_block) {
        const unsigned e = (blockIdx.x - q.first_block) * kKvThreads + threadIdx.x;
        if (e >= q.all) return;
        const unsigned tg = e / q.units, u = e - tg * q.units, t = tg / q.groups;
        TokenPlace at;
        if (!kv_place(pool, list, t, rot.rows, &at)) return;
        if (rot.layout == W4_ROPE_HALF)
            turn_unit<W4_ROPE_HALF, HEADS>(q.q, q.out, t, u, tg - t * q.groups, q.groups, q.heads,
                                           rot, at.position, false);
        else
            turn_unit<W4_ROPE_INTERLEAVED, HEADS>(q.q, q.out, t, u, tg - t * q.groups, q.groups,
                                                  q.heads, rot, at.position, false);
        return;
    }
    const int tile_no = blockIdx.x / pool.kv_heads, h = blockIdx.x - tile_no * pool.kv_heads;
    int first, count;
    bool whole;
    const int i0 = load_tile(pool, list, tile_no, tiles, rot.table ? rot.rows : 0x7FFFFFFF, &tile, &first,
                             &count, &whole);
    if (count <= 0) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c = lane % LANES;
    for (int n0 = warp * TOKENS; n0 < count; n0 += kKvWarps * TOKENS) {
        const int r = min(first + n0 + lane / (2 * LANES), kRecTokens - 1);
        const bool valid = n0 + lane / (2 * LANES) < count && tile.valid[r];
        const int t = i0 + r, pos = tile.position[r];
        const bool is_v = lane / LANES & 1;
        const Heads &src = is_v ? v : k;
        uint4 raw = make_uint4(0u, 0u, 0u, 0u);
        if (valid)
            raw = *reinterpret_cast<const uint4 *>(
                reinterpret_cast<const __nv_bfloat16 *>(src.data) + t * src.token_stride +
                h * src.head_stride + 8 * c);
        float x[8];
        const uint32_t *w = &raw.x;
#pragma unroll
        for (int i = 0; i < 4; ++i) x[2 * i] = bf16_low(w[i]), x[2 * i + 1] = bf16_high(w[i]);
        if (rot.table) {
            const bool turns = valid && !is_v && 8 * c < 2 * rot.pairs;
            const float *row_of = rot.table + 2LL * (valid ? pos : 0) * rot.pairs;
            if (rot.layout == W4_ROPE_INTERLEAVED) {
                if (turns) {
                    const float4 *tab = reinterpret_cast<const float4 *>(row_of + 8 * c);
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float4 cs = tab[i];
                        const float2 y0 = turn_pair(x[4 * i], x[4 * i + 1], make_float2(cs.x, cs.y));
                        const float2 y1 =
                            turn_pair(x[4 * i + 2], x[4 * i + 3], make_float2(cs.z, cs.w));
                        x[4 * i] = y0.x, x[4 * i + 1] = y0.y;
                        x[4 * i + 2] = y1.x, x[4 * i + 3] = y1.y;
                    }
                }
            } else {
                // the partners are another lane's values
                const int half = rot.pairs / 8;
                const bool upper = c >= half;
                const int from = lane - c + (upper ? c - half : c + half);
                uint32_t p[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) p[i] = __shfl_sync(0xFFFFFFFFu, w[i], from & 31);
                if (turns) {
                    const float4 *tab = reinterpret_cast<const float4 *>(
                        row_of + 16 * (upper ? c - half : c));
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float4 cs = tab[i];
                        const float p0 = bf16_low(p[i]), p1 = bf16_high(p[i]);
                        const float2 y0 = upper ? turn_pair(p0, x[2 * i], make_float2(cs.x, cs.y))
                                                : turn_pair(x[2 * i], p0, make_float2(cs.x, cs.y));
                        const float2 y1 =
                            upper ? turn_pair(p1, x[2 * i + 1], make_float2(cs.z, cs.w))
                                  : turn_pair(x[2 * i + 1], p1, make_float2(cs.z, cs.w));
                        x[2 * i] = upper ? y0.y : y0.x;
                        x[2 * i + 1] = upper ? y1.y : y1.x;
                    }
                }
            }
        }
        const uint4 packed = make_uint4(bf16_pair(x[0], x[1]), bf16_pair(x[2], x[3]),
                                        bf16_pair(x[4], x[5]), bf16_pair(x[6], x[7]));
        const int in = tile.in_page[r], rr = in % kRecTokens;
        unsigned char *rec =
            whole ? staged
                  : reinterpret_cast<unsigned char *>(pool.records) +
                        (tile.page_record[r] + (long long)h * pool.page_records +
                         in / kRecTokens) * L::kBytes;
        if constexpr (FMT == W4_KV_BF16) {
            if (valid)
                *reinterpret_cast<uint4 *>(rec + (is_v ? L::value(rr, 8 * c) : L::key(rr, 8 * c))) =
                    packed;
        } else {
            float lo = 0.f, hi = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) lo = fminf(lo, x[i]), hi = fmaxf(hi, x[i]);
#pragma unroll
            for (int o = LANES / 2; o > 0; o >>= 1) {
                lo = fminf(lo, __shfl_xor_sync(0xFFFFFFFFu, lo, o));
                hi = fmaxf(hi, __shfl_xor_sync(0xFFFFFFFFu, hi, o));
            }
            constexpr float top = (float)L::kLevels;
            const __half sh =
                __float2half_rn(fminf(__fdiv_rn(__fsub_rn(hi, lo), top), 65504.f));
            const float s = __half2float(sh);
            const float z = s == 0.f ? 0.f : clampf(rintf(__fdiv_rn(-lo, s)), 0.f, top);
            const float rcp = s == 0.f ? 0.f : __frcp_rn(s);
            const float tol = __fmul_rn(__fmul_rn(fmaxf(-lo, hi), rcp), 0x1p-21f);
            uint32_t code[2] = {0u, 0u};                      // 8 codes, a byte each
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float f =
                    s == 0.f ? 0.f : clampf(rint_quotient(x[i], s, rcp, tol) + z, 0.f, top);
                code[i / 4] |= (uint32_t)f << (8 * (i % 4));
            }
            if constexpr (FMT == W4_KV_INT8) {
                if (valid && !is_v)
                    *reinterpret_cast<uint2 *>(rec + L::key(rr, 8 * c)) =
                        make_uint2(code[0], code[1]);
                if (valid && is_v) {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        rec[L::value(rr, 8 * c + i)] = (unsigned char)(code[i / 4] >> 8 * (i % 4));
                }
            } else {
                // the other nibble of a value's byte is 8 values on: the next
                // lane's (each of the two writes half of the bytes)
                const uint32_t other0 = __shfl_xor_sync(0xFFFFFFFFu, code[0], 1);
                const uint32_t other1 = __shfl_xor_sync(0xFFFFFFFFu, code[1], 1);
                if (valid && !is_v) {
                    uint32_t bytes = 0u;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t two = code[i / 2] >> (16 * (i % 2));
                        bytes |= ((two & 15u) | (two >> 4 & 0xF0u)) << (8 * i);
                    }
                    *reinterpret_cast<uint32_t *>(rec + L::key(rr, 8 * c)) = bytes;
                }
                if (valid && is_v) {
                    const bool odd = c & 1;
                    const uint32_t both = odd ? other1 | code[1] << 4 : code[0] | other0 << 4;
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        rec[L::value(rr, 8 * (c & ~1) + (odd ? 4 : 0) + i)] =
                            (unsigned char)(both >> 8 * i);
                }
            }
            if (valid && c == 0)
                *reinterpret_cast<uint32_t *>(rec + (is_v ? L::kMetaV : L::kMeta) + 4 * rr) =
                    (uint32_t)__half_as_ushort(sh) | (uint32_t)z << 16;
        }
    }
    if (!whole) return;
    __syncthreads();
    uint4 *out = reinterpret_cast<uint4 *>(
        pool.records + (tile.page_record[0] + (long long)h * pool.page_records +
                        tile.in_page[0] / kRecTokens) * L::kBytes);
    for (int i = threadIdx.x; i < L::kBytes / 16; i += kKvThreads)
        out[i] = reinterpret_cast<const uint4 *>(staged)[i];
}

template <int FMT, int D>
__global__ void __launch_bounds__(kKvThreads)
read_kernel(KvPool pool, Heads k, Heads v, TokenList list, int tiles) {
    using L = KvLayout<FMT, D>;
    constexpr int LANES = D / 8, TOKENS = 16 / LANES;         // tokens a warp takes at a time
    __shared__ Tile16 tile;
    __shared__ __align__(16) unsigned char staged[L::kBytes];
    begin_after_previous();
    int first, count;
    bool whole;
    const int i0 = load_tile(pool, list, blockIdx.x, tiles, 0x7FFFFFFF, &tile, &first, &count, &whole);
    if (count <= 0) return;
    const int h = blockIdx.y;
    if (whole) {
        const uint4 *in = reinterpret_cast<const uint4 *>(
            pool.records + (tile.page_record[0] + (long long)h * pool.page_records +
                            tile.in_page[0] / kRecTokens) * L::kBytes);
#pragma unroll
        for (int i = 0; i < (L::kBytes / 16 + kKvThreads - 1) / kKvThreads; ++i) {
            const int at = i * kKvThreads + threadIdx.x;
            if (at < L::kBytes / 16) reinterpret_cast<uint4 *>(staged)[at] = in[at];
        }
        __syncthreads();
    }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c = lane % LANES;
    // 2 LANES lanes take a token: its key, then its value
    for (int n = warp * TOKENS + lane / (2 * LANES); n < count; n += kKvWarps * TOKENS) {
        const int r = first + n;
        const bool is_v = lane / LANES & 1;
        const Heads &dst = is_v ? v : k;
        if (!tile.valid[r] || !dst.data) continue;
        const int in = tile.in_page[r], rr = in % kRecTokens;
        const unsigned char *rec =
            whole ? staged
                  : reinterpret_cast<const unsigned char *>(pool.records) +
                        (tile.page_record[r] + (long long)h * pool.page_records +
                         in / kRecTokens) * L::kBytes;
        uint4 packed;
        if constexpr (FMT == W4_KV_BF16) {
            packed = *reinterpret_cast<const uint4 *>(
                rec + (is_v ? L::value(rr, 8 * c) : L::key(rr, 8 * c)));
        } else {
            const uint32_t m = *reinterpret_cast<const uint32_t *>(
                rec + (is_v ? L::kMetaV : L::kMeta) + 4 * rr);
            const float s = __half2float(__ushort_as_half((unsigned short)(m & 0xFFFFu)));
            const int z = (int)(m >> 16);
            uint32_t code[2] = {0u, 0u};
            if constexpr (FMT == W4_KV_INT8) {
                if (!is_v) {
                    const uint2 w = *reinterpret_cast<const uint2 *>(rec + L::key(rr, 8 * c));
                    code[0] = w.x, code[1] = w.y;
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        code[i / 4] |= (uint32_t)rec[L::value(rr, 8 * c + i)] << (8 * (i % 4));
                }
            } else if (!is_v) {
                const uint32_t w = *reinterpret_cast<const uint32_t *>(rec + L::key(rr, 8 * c));
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    code[i / 4] |= (w >> (4 * i) & 15u) << (8 * (i % 4));
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    code[i / 4] |= ((uint32_t)rec[L::value(rr, 8 * c + i)] >> (4 * (c & 1)) & 15u)
                                   << (8 * (i % 4));
            }
            float x[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                x[i] = __fmul_rn((float)((int)(code[i / 4] >> (8 * (i % 4)) & 255u) - z), s);
            packed = make_uint4(bf16_pair(x[0], x[1]), bf16_pair(x[2], x[3]),
                                bf16_pair(x[4], x[5]), bf16_pair(x[6], x[7]));
        }
        *reinterpret_cast<uint4 *>(reinterpret_cast<__nv_bfloat16 *>(dst.data) +
                                   (i0 + r) * dst.token_stride + h * dst.head_stride + 8 * c) =
            packed;
    }
}

// Tiles that a run of `run` tokens can touch, wherever in a record it starts.
int tiles_of(int run) { return (run + 2 * (kRecTokens - 1)) / kRecTokens; }

template <int D, int HEADS>
cudaError_t append_dim(const KvPool &pool, int format, const Heads &k, const Heads &v, Queries q,
                       const TokenList &list, const Rotation &rot, cudaStream_t stream) {
    const int tiles = tiles_of(list.run);
    q.first_block = (unsigned)(list.tokens / list.run * tiles) * pool.kv_heads;
    const dim3 grid(q.first_block + (q.all + kKvThreads - 1) / kKvThreads);
    const auto kernel = format == W4_KV_BF16   ? append_kernel<W4_KV_BF16, D, HEADS>
                        : format == W4_KV_INT8 ? append_kernel<W4_KV_INT8, D, HEADS>
                                               : append_kernel<W4_KV_INT4, D, HEADS>;
    return launch_overlapped(kernel, grid, dim3(kKvThreads), 0, stream, pool, k, v, q, list, rot,
                             tiles);
}

template <int D>
cudaError_t read_dim(const KvPool &pool, int format, const Heads &k, const Heads &v,
                     const TokenList &list, cudaStream_t stream) {
    const int tiles = tiles_of(list.run);
    const dim3 grid((unsigned)(list.tokens / list.run * tiles), (unsigned)pool.kv_heads);
    const auto kernel = format == W4_KV_BF16   ? read_kernel<W4_KV_BF16, D>
                        : format == W4_KV_INT8 ? read_kernel<W4_KV_INT8, D>
                                               : read_kernel<W4_KV_INT4, D>;
    return launch_overlapped(kernel, grid, dim3(kKvThreads), 0, stream, pool, k, v, list, tiles);
}

}  // namespace

cudaError_t launch_kv_append(const KvPool &pool, int format, int head_dim, const Heads &k,
                             const Heads &v, const Heads &q, const Heads &q_out, int q_heads,
                             const TokenList &list, const Rotation &rot, int num_sms,
                             cudaStream_t stream) {
    Queries qs = {q, q_out, q_heads, 1, 1, 0, 0};
    bool four = false;
    if (q_heads > 0) {
        // four heads a thread once that still gives every SM two blocks
        qs.units = turn_units(q, q_out, head_dim, rot);
        const long long by_four = (long long)list.tokens * ((q_heads + 3) / 4) * qs.units;
        four = by_four >= 2LL * num_sms * kKvThreads;
        qs.groups = four ? (q_heads + 3) / 4 : q_heads;
        qs.all = (unsigned)((long long)list.tokens * qs.groups * qs.units);
    }
    if (head_dim == 64)
        return four ? append_dim<64, 4>(pool, format, k, v, qs, list, rot, stream)
                    : append_dim<64, 1>(pool, format, k, v, qs, list, rot, stream);
    return four ? append_dim<128, 4>(pool, format, k, v, qs, list, rot, stream)
                : append_dim<128, 1>(pool, format, k, v, qs, list, rot, stream);
}

cudaError_t launch_kv_read(const KvPool &pool, int format, int head_dim, const Heads &k,
                           const Heads &v, const TokenList &list, cudaStream_t stream) {
    return head_dim == 64 ? read_dim<64>(pool, format, k, v, list, stream)
                          : read_dim<128>(pool, format, k, v, list, stream);
}

}  // namespace w4
