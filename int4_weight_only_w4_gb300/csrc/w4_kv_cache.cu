// The paged key-value cache: writing tokens (w4_kv_append: rotation of q and
// k, quantisation, the record layout) and reading them back (w4_kv_read).
//
// Mathematics of a (token, head) group: the rule of include/w4.h, w4_quantize's
// asymmetric one with Q = 255 or 15 levels but for the scale, which is a
// product with 1 / Q instead of a quotient; every operation rounded to nearest
// in fp32, so the codes are those of any other evaluation of the rule bit for
// bit.
//
// A tile is up to 16 listed tokens, cut so that the tokens of a sequence in
// order fall into whole records.  A warp (or four) takes the keys, or the
// values, of a tile and head; all its loads are under way together.  The layout
// of quantised values scatters a token over 64 sectors, so those of a whole
// record are turned, by ldmatrix (by stmatrix on the way back), and moved with
// 16-byte accesses: byte by byte 16384 tokens of 28 + 4 heads of 128 in 4 bits
// took 95 us to write and read back, turned they take 62 (5.28 TB/s: 78 % of a
// copy's rate).  Tiles that are no whole record (decode steps, the ends of a
// prompt, tokens in another order) go byte by byte.
//
// What bounds it (captured calls, written and read back; each by itself): one
// token of each of 64 sequences 6.0 us (3.2, 2.8), two launches and a chain of
// four dependent trips to memory (position, page, row, record); 4096 tokens in 8
// bits 23.6 us (18.3, 4.5; the bytes take 10.8 and 1.9): writing issues in 57 % of
// its cycles and waits for rows and table, reading is one wave of blocks that wait
// at their tile's barriers; 16 k tokens in 4 bits 61.9 us (51.8, 10.1; bytes 42.1
// and 6.3), the traffic of the queries, which pass through (writing: 62 % of the
// issue slots, 57 % of the DRAM's).  Read back at once the records come from L2.
#include "w4_kv.cuh"

namespace w4 {
namespace {

constexpr int kKvThreads = 128, kKvWarps = kKvThreads / 32;

// The tile's tokens: list indexes i0 .. i0 + 15 of which [lo, hi) are there.
struct Tile16 {
    unsigned char *record[kRecTokens];    // of head 0; NULL: the token is left out
    int in_record[kRecTokens];
    int position[kRecTokens];
};

// Fills the tile of this block; returns the list index of its token 0; tokens
// first .. first + count - 1 are there (count <= 0: none).  whole (if ASK): the
// tokens are one record.  All threads call.
template <bool ASK>
__device__ __forceinline__ int load_tile(const KvPool &pool, const TokenList &list, int tile_no,
                                         int tiles, int rotation_rows, int record_bytes,
                                         Tile16 *tile, int *first, int *count, bool *whole) {
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
        tile->record[r] = ok ? reinterpret_cast<unsigned char *>(pool.records) +
                                   (at.page_record + at.in_page / kRecTokens) * record_bytes
                             : nullptr;
        tile->in_record[r] = at.in_page % kRecTokens;
        tile->position[r] = at.position;
    }
    __syncthreads();
    *whole = false;
    if (!ASK) return base + i0;
    bool same = true;
    if (r < kRecTokens)
        same = tile->record[r] && tile->record[r] == tile->record[0] && tile->in_record[r] == r;
    *whole = __syncthreads_and(same);
    return base + i0;
}

// Two fp32 operations in one instruction, each rounded to nearest.
union Two {
    unsigned long long both;
    float2 f;
    int2 i;
};
__device__ __forceinline__ Two mul2(Two a, Two b) {
    Two r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.both) : "l"(a.both), "l"(b.both));
    return r;
}
__device__ __forceinline__ Two add2(Two a, Two b) {
    Two r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.both) : "l"(a.both), "l"(b.both));
    return r;
}
__device__ __forceinline__ Two twice(float v) {
    Two r;
    r.f = make_float2(v, v);
    return r;
}

// The largest of three; NaN if any is (fmaxf would drop it).
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
    float r;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ int rint_quotient(float w, float s) {
    const float q = rintf(__fdiv_rn(w, s));
    return q == q ? (int)fminf(fmaxf(q, -512.f), 512.f) : 0;
}

// Zero point and codes of 8 of a row's values, of range [lo, hi]; s > 0.  The
// rule wants rint(w / s), w / s the correctly rounded quotient.  With r within an
// ulp of 1 / s, t = w r is within 2^-22.4 of the quotient's magnitude; adding and
// subtracting 1.5 * 2^23 rounds t to the nearest integer (ties to even), and
// where t is further than T * 2^-21 (T >= every |t| of the row) from a half,
// that integer is the rule's.  In the rare other case, and where a value is NaN
// (its distance is, too), the division decides; NaN gets the code of 0.
template <int BITS>
__device__ __forceinline__ void codes_of(const float (&w)[8], float lo, float hi, float s,
                                         int *zero, int (&n)[8]) {
    constexpr float kMagic = 12582912.f;                      // 1.5 * 2^23
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
    const float tol = __fmul_rn(__fmul_rn(fmaxf(-lo, hi), r), 0x1p-21f);
    const float tz = __fmul_rn(-lo, r), yz = __fadd_rn(tz, kMagic);
    float far = fabsf(__fsub_rn(tz, __fsub_rn(yz, kMagic)));   // from an integer
    int z = __float_as_int(yz) - __float_as_int(kMagic);
    z = min(max(z, 0), (1 << BITS) - 1);
    const int shift = z - __float_as_int(kMagic);
    const Two up = twice(kMagic), down = twice(-kMagic), rr = twice(r), minus = twice(-1.f);
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        Two x;
        x.f = make_float2(w[i], w[i + 1]);
        const Two q = mul2(x, rr), y = add2(q, up);
        const Two d = add2(mul2(add2(y, down), minus), q);    // exact
        far = max3_nan(far, fabsf(d.f.x), fabsf(d.f.y));
        n[i] = y.i.x + shift, n[i + 1] = y.i.y + shift;
    }
    if (!(0.5f - far > tol)) {
        z = min(max(rint_quotient(-lo, s), 0), (1 << BITS) - 1);
#pragma unroll
        for (int i = 0; i < 8; ++i) n[i] = rint_quotient(w[i], s) + z;
    }
    *zero = z;
}

// Four codes clamped (by saturation) to bytes; eight to nibbles.
__device__ __forceinline__ uint32_t to_bytes(int n0, int n1, int n2, int n3) {
    uint32_t w;
    asm("cvt.pack.sat.u8.s32.b32 %0, %1, %2, 0;" : "=r"(w) : "r"(n3), "r"(n2));
    asm("cvt.pack.sat.u8.s32.b32 %0, %1, %2, %3;" : "=r"(w) : "r"(n1), "r"(n0), "r"(w));
    return w;
}
__device__ __forceinline__ uint32_t to_nibbles(const int (&n)[8]) {
    uint32_t w = 0u;
#pragma unroll
    for (int i = 6; i >= 0; i -= 2)
        asm("cvt.pack.sat.u4.s32.b32 %0, %1, %2, %3;"
            : "=r"(w)
            : "r"(n[i + 1]), "r"(n[i]), "r"(w));
    return w;
}

// The queries of a launch of append_kernel, turned (without a rotation: copied)
// as by w4_rope in blocks of their own (in the rows' loop below every lane would turn its partner too:
// 16 k tokens of 28 query heads, written and read back, 148 us against 95).
struct Queries {
    Heads q, out;
    int heads;
    unsigned groups, units;    // see turn_unit
    unsigned all;              // tokens * groups * units
    unsigned rows_blocks;      // blocks that take keys and values: every period-th,
    unsigned period;           // from the first on, so that their arithmetic
};                             // and the others' traffic overlap

// Keys and values: D / 8 lanes take a row (a head of a token), 8 values a lane.
// WHOLE: some tiles may be whole records; without that code, which short runs
// do not need, one token of 64 sequences is written 1.3 us faster.  Eight blocks
// an SM (64 registers) where queries go by four heads of 128: 16384 tokens in 4
// bits, written and read back, 62.1 us instead of 63.8; with heads of 64 it costs
// (8192 tokens 14.4 instead of 13.8).  0: no such bound; with 1 the compiler
// takes 61 registers instead of 48 for short runs, and they 7.1 us instead of 6.0.
template <int FMT, int D, int HEADS, bool WHOLE>
__global__ void
__launch_bounds__(kKvThreads, FMT != W4_KV_BF16 && D == 128 && HEADS == 4 ? 8 : 0)
append_kernel(KvPool pool, Heads k, Heads v, Queries q, TokenList list, Rotation rot, int tiles,
              int split) {
    using L = KvLayout<FMT, D>;
    constexpr int LANES = D / 8, TOKENS = 32 / LANES;
    __shared__ Tile16 tile;
    __shared__ uint4 rows[kKvWarps][kRecTokens * LANES];
    begin_after_previous();
    const unsigned turn = blockIdx.x / q.period;
    if (blockIdx.x != turn * q.period || turn >= q.rows_blocks) {
        const unsigned e =
            (blockIdx.x - min(turn + 1, q.rows_blocks)) * kKvThreads + threadIdx.x;
        if (e >= q.all) return;
        const unsigned tg = e / q.units, u = e - tg * q.units, t = tg / q.groups;
        TokenPlace at;
        if (!kv_place(pool, list, t, rot.table ? rot.rows : 0x7FFFFFFF, &at)) return;
        if (rot.layout == W4_ROPE_HALF)
            turn_unit<W4_ROPE_HALF, HEADS>(q.q, q.out, t, u, tg - t * q.groups, q.groups, q.heads,
                                           rot, at.position, false);
        else
            turn_unit<W4_ROPE_INTERLEAVED, HEADS>(q.q, q.out, t, u, tg - t * q.groups, q.groups,
                                                  q.heads, rot, at.position, false);
        return;
    }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c = lane % LANES;
    const int parts = (2 * pool.kv_heads * split + kKvWarps - 1) / kKvWarps;    // blocks of a tile
    const int tile_no = turn / parts;
    int task = (turn - tile_no * parts) * kKvWarps + warp;
    const int part = task % split;
    task /= split;
    int first, count;
    bool whole;
    const int i0 = load_tile<WHOLE>(pool, list, tile_no, tiles,
                                    rot.table ? rot.rows : 0x7FFFFFFF, L::kBytes, &tile, &first,
                                    &count, &whole);
    if (count <= 0 || task >= 2 * pool.kv_heads) return;
    const bool is_v = task & 1;
    const int h = task >> 1;
    const long long head_bytes = (long long)h * pool.page_records * L::kBytes;
    const __nv_bfloat16 *src = reinterpret_cast<const __nv_bfloat16 *>((is_v ? v : k).data) +
                               h * (is_v ? v : k).head_stride + 8 * c;
    const long long stride = (is_v ? v : k).token_stride;
    // all rows are asked for at once, into shared memory: held in registers
    // they would need an unrolled loop, which its instructions' fetching slows
    for (int x = part; x * TOKENS < count; x += split) {
        const int n = x * TOKENS + lane / LANES;
        if (n < count && tile.record[first + n])
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                             (uint32_t)__cvta_generic_to_shared(&rows[warp][32 * x + lane])),
                         "l"(src + (i0 + first + n) * stride)
                         : "memory");
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncwarp();
#pragma unroll 1
    for (int x0 = part; x0 * TOKENS < count; x0 += split) {
        const int n = x0 * TOKENS + lane / LANES, r = min(first + n, kRecTokens - 1);
        unsigned char *rec = n < count ? tile.record[r] : nullptr;
        const bool valid = rec != nullptr;
        rec += head_bytes;
        const int pos = tile.position[r];
        float x[8];
        const uint4 raw = valid ? rows[warp][32 * x0 + lane] : make_uint4(0u, 0u, 0u, 0u);
        const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) x[2 * i] = bf16_low(w[i]), x[2 * i + 1] = bf16_high(w[i]);
        if (rot.table && !is_v) {
            const bool turns = valid && 8 * c < 2 * rot.pairs;
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
                // the partners are another lane's values; a lane works out its
                // own half of each pair: x c + p s, with -s in the lower half
                const int half = rot.pairs / 8;
                const bool upper = c >= half;
                const int from = lane - c + (upper ? c - half : c + half);
                const uint32_t flip = upper ? 0u : 0x80000000u;
                uint32_t p[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) p[i] = __shfl_sync(0xFFFFFFFFu, w[i], from & 31);
                if (turns) {
                    const float4 *tab = reinterpret_cast<const float4 *>(
                        row_of + 16 * (upper ? c - half : c));
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float4 cs = tab[i];
                        const float s0 = __uint_as_float(__float_as_uint(cs.y) ^ flip);
                        const float s1 = __uint_as_float(__float_as_uint(cs.w) ^ flip);
                        x[2 * i] = __fadd_rn(__fmul_rn(x[2 * i], cs.x),
                                             __fmul_rn(bf16_low(p[i]), s0));
                        x[2 * i + 1] = __fadd_rn(__fmul_rn(x[2 * i + 1], cs.z),
                                                 __fmul_rn(bf16_high(p[i]), s1));
                    }
                }
            }
        }
        const int rr = tile.in_record[r];
        if constexpr (FMT == W4_KV_BF16) {
            if (valid)
                *reinterpret_cast<uint4 *>(rec + (is_v ? L::value(rr, 8 * c) : L::key(rr, 8 * c))) =
                    make_uint4(bf16_pair(x[0], x[1]), bf16_pair(x[2], x[3]), bf16_pair(x[4], x[5]),
                               bf16_pair(x[6], x[7]));
        } else {
            float lo = 0.f, hi = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) lo = fminf(lo, x[i]), hi = fmaxf(hi, x[i]);
#pragma unroll
            for (int o = LANES / 2; o > 0; o >>= 1) {
                lo = fminf(lo, __shfl_xor_sync(0xFFFFFFFFu, lo, o));
                hi = fmaxf(hi, __shfl_xor_sync(0xFFFFFFFFu, hi, o));
            }
            constexpr float level = 1.f / L::kLevels;
            const __half sh =
                __float2half_rn(fminf(__fmul_rn(__fsub_rn(hi, lo), level), 65504.f));
            const float s = __half2float(sh);
            int z = 0, n8[8] = {0, 0, 0, 0, 0, 0, 0, 0};
            if (s > 0.f) codes_of<L::kBits>(x, lo, hi, s, &z, n8);
            if (WHOLE && is_v && whole) {
                // in 16 bits each, in the place of the row's own values (its
                // pieces exchanged so that 8 rows lie in different banks)
                uint32_t u[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    asm("cvt.pack.sat.u16.s32 %0, %1, %2;"
                        : "=r"(u[i])
                        : "r"(n8[2 * i + 1]), "r"(n8[2 * i]));
                    u[i] = __vminu2(u[i], L::kLevels * 0x00010001u);
                }
                __syncwarp();
                rows[warp][32 * x0 + lane - c + (c ^ (n & 7))] = make_uint4(u[0], u[1], u[2], u[3]);
            } else if constexpr (FMT == W4_KV_INT8) {
                const uint32_t b0 = to_bytes(n8[0], n8[1], n8[2], n8[3]);
                const uint32_t b1 = to_bytes(n8[4], n8[5], n8[6], n8[7]);
                if (valid && !is_v)
                    *reinterpret_cast<uint2 *>(rec + L::key(rr, 8 * c)) = make_uint2(b0, b1);
                if (valid && is_v) {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        rec[L::value(rr, 8 * c + i)] =
                            (unsigned char)((i < 4 ? b0 : b1) >> 8 * (i & 3));
                }
            } else if (!is_v) {
                if (valid) *reinterpret_cast<uint32_t *>(rec + L::key(rr, 8 * c)) = to_nibbles(n8);
            } else {
                // the high nibble of a value's byte is 8 values on, in the next
                // lane: the even lane writes the first four bytes of the two,
                // the odd one the others (15 is the largest code: the bytes
                // are saturated at 4 bits first)
                uint32_t b[2];
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    b[i] = to_bytes(min(n8[4 * i], 15), min(n8[4 * i + 1], 15),
                                    min(n8[4 * i + 2], 15), min(n8[4 * i + 3], 15));
                const bool odd = c & 1;
                const uint32_t got = __shfl_xor_sync(0xFFFFFFFFu, odd ? b[0] : b[1], 1);
                const uint32_t bytes = odd ? got | b[1] << 4 : b[0] | got << 4;
                if (valid) {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        rec[L::value(rr, 8 * (c & ~1) + (odd ? 4 : 0) + i)] =
                            (unsigned char)(bytes >> 8 * i);
                }
            }
            if (valid && c == 0)
                *reinterpret_cast<uint32_t *>(rec + (is_v ? L::kMetaV : L::kMeta) + 4 * rr) =
                    (uint32_t)__half_as_ushort(sh) | (uint32_t)z << 16;
        }
    }
    // a whole record's values: the rows' codes, turned, give every lane those
    // of one d and tokens 2t, 2t + 1 (and 8 on), which are the bytes of its words
    if constexpr (WHOLE) {
        if (!whole || !is_v) return;
        if (split == 1)
            __syncwarp();
        else
            __syncthreads();                                  // the block has one task
        const int n = lane & 15;
        const uint32_t row = (uint32_t)__cvta_generic_to_shared(
            &rows[split == 1 ? warp : (n / TOKENS) % kKvWarps][n * LANES]);
        uint4 *out = reinterpret_cast<uint4 *>(tile.record[0] + head_bytes + L::kPart) + lane;
        constexpr int PIECES = L::kPart / 512;
#pragma unroll
        for (int i = 0; i < PIECES; ++i) {
            if (split != 1 && i % kKvWarps != part) continue;
            uint32_t w[4];
            const auto get = [&](int x, uint32_t *m) {        // d of 8 x .. 8 x + 15
                asm volatile(
                    "ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                    : "=r"(m[0]), "=r"(m[1]), "=r"(m[2]), "=r"(m[3])
                    : "r"(row + (((x + (lane >> 4)) ^ (n & 7)) << 4))
                    : "memory");
            };
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint32_t m[4];
                if constexpr (FMT == W4_KV_INT4) {
                    get(8 * i + 2 * j, m);
                    w[j] = (m[0] | m[1] << 8) | (m[2] | m[3] << 8) << 4;
                } else if (j % 2 == 0) {
                    get(4 * i + j, m);
                    w[j] = m[0] | m[1] << 8, w[j + 1] = m[2] | m[3] << 8;
                }
            }
            out[32 * i] = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
}

// Eight values of a row from their codes, (u - z) s each; zm: -(2^23 + z).
__device__ __forceinline__ uint4 row_values(uint32_t c0, uint32_t c1, Two zm, Two ss) {
    uint32_t out[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t w = i < 2 ? c0 : c1;
        Two y;
        y.i.x = __byte_perm(w, 0x4B000000u, 0x7540 + 2 * (i & 1));
        y.i.y = __byte_perm(w, 0x4B000000u, 0x7541 + 2 * (i & 1));
        y = mul2(add2(y, zm), ss);                            // the sum is exact
        out[i] = bf16_pair(y.f.x, y.f.y);
    }
    return make_uint4(out[0], out[1], out[2], out[3]);
}
__device__ __forceinline__ float less_of(uint32_t meta) { return -(float)(8388608 + (meta >> 16)); }
__device__ __forceinline__ float scale_of(uint32_t meta) {
    return __half2float(__ushort_as_half((unsigned short)(meta & 0xFFFFu)));
}
// The codes of 8 of a key's values: nibbles 0, 2, 4, 6 and 1, 3, 5, 7 to bytes,
// then in order.
__device__ __forceinline__ void key_codes(uint32_t w, uint32_t *code) {
    const uint32_t lo = w & 0x0F0F0F0Fu, hi = w >> 4 & 0x0F0F0F0Fu;
    code[0] = __byte_perm(lo, hi, 0x5140);
    code[1] = __byte_perm(lo, hi, 0x7362);
}

// A whole record's keys to 16 rows from `dst` on: every lane's loads at once.
template <int FMT, int D>
__device__ __forceinline__ void read_keys(const unsigned char *rec, __nv_bfloat16 *dst,
                                          long long stride) {
    using L = KvLayout<FMT, D>;
    constexpr int LANES = D / 8, TOKENS = 32 / LANES, STEPS = kRecTokens / TOKENS;
    const int lane = threadIdx.x & 31, c = lane % LANES, r0 = lane / LANES;
    uint32_t meta[STEPS];
    uint2 w[STEPS];
#pragma unroll
    for (int x = 0; x < STEPS; ++x) {
        const unsigned char *at = rec + L::key(x * TOKENS + r0, 8 * c);
        meta[x] = *reinterpret_cast<const uint32_t *>(rec + L::kMeta + 4 * (x * TOKENS + r0));
        if (FMT == W4_KV_INT8)
            w[x] = *reinterpret_cast<const uint2 *>(at);
        else
            w[x].x = *reinterpret_cast<const uint32_t *>(at);
    }
    dst += r0 * stride + 8 * c;
#pragma unroll
    for (int x = 0; x < STEPS; ++x) {
        uint32_t code[2];
        if (FMT == W4_KV_INT4)
            key_codes(w[x].x, code);
        else
            code[0] = w[x].x, code[1] = w[x].y;
        *reinterpret_cast<uint4 *>(dst + x * TOKENS * stride) =
            row_values(code[0], code[1], twice(less_of(meta[x])), twice(scale_of(meta[x])));
    }
}

// A whole record's values: a lane's 16 bytes are of two tokens (and two more,
// 8 on) and one d modulo 8, so the values come out as 8 x 8 matrices d x token,
// which stmatrix turns on their way to the rows in shared memory.  (Gathered
// byte by byte from there, reading 16 k tokens of 4 heads took 21 us.)
template <int FMT, int D>
__device__ __forceinline__ void read_values(const unsigned char *rec, unsigned char *rows,
                                            __nv_bfloat16 *dst, long long stride) {
    using L = KvLayout<FMT, D>;
    constexpr int LANES = D / 8, TOKENS = 32 / LANES, STEPS = kRecTokens / TOKENS;
    constexpr int ROW = 2 * D + 16, PIECES = L::kPart / 512;
    const int lane = threadIdx.x & 31, t = lane & 3;
    uint4 raw[PIECES];
#pragma unroll
    for (int i = 0; i < PIECES; ++i)
        raw[i] = *reinterpret_cast<const uint4 *>(rec + L::kPart + i * 512 + lane * 16);
    Two zm[2], ss[2];                                         // of tokens 2t, 2t + 1 (+ 8)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint2 m = *reinterpret_cast<const uint2 *>(rec + L::kMetaV + 4 * (2 * t + 8 * h));
        zm[h].f = make_float2(less_of(m.x), less_of(m.y));
        ss[h].f = make_float2(scale_of(m.x), scale_of(m.y));
    }
    const uint32_t at = (uint32_t)__cvta_generic_to_shared(rows) + (lane & 15) * ROW +
                        (lane >> 4) * 16;
    const auto pair = [&](uint32_t v, int h) {
        Two y;
        y.i.x = __byte_perm(v, 0x4B000000u, 0x7540 + h);
        y.i.y = __byte_perm(v, 0x4B000000u, 0x7542 + h);
        y = mul2(add2(y, zm[h]), ss[h]);                      // the sum is exact
        return bf16_pair(y.f.x, y.f.y);
    };
    const auto put = [&](int x, uint32_t v0, uint32_t v1) {   // d of 8 x .. 8 x + 15
        asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(
                         at + 16 * x),
                     "r"(pair(v0, 0)), "r"(pair(v0, 1)), "r"(pair(v1, 0)), "r"(pair(v1, 1))
                     : "memory");
    };
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
        const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
        if constexpr (FMT == W4_KV_INT8) {
            put(4 * i, w[0], w[1]);
            put(4 * i + 2, w[2], w[3]);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                put(8 * i + 2 * j, w[j] & 0x0F0F0F0Fu, w[j] >> 4 & 0x0F0F0F0Fu);
        }
    }
    __syncwarp();
    const int c = lane % LANES, r0 = lane / LANES;
    dst += r0 * stride + 8 * c;
#pragma unroll
    for (int x = 0; x < STEPS; ++x)
        *reinterpret_cast<uint4 *>(dst + x * TOKENS * stride) =
            *reinterpret_cast<const uint4 *>(rows + (x * TOKENS + r0) * ROW + 16 * c);
}

template <int FMT, int D>
__global__ void __launch_bounds__(kKvThreads)
read_kernel(KvPool pool, Heads k, Heads v, TokenList list, int tiles, int split) {
    using L = KvLayout<FMT, D>;
    constexpr int LANES = D / 8, TOKENS = 32 / LANES, STEPS = kRecTokens / TOKENS;
    __shared__ Tile16 tile;
    __shared__ __align__(16) unsigned char
        turned[kKvWarps][FMT == W4_KV_BF16 ? 16 : kRecTokens * (2 * D + 16)];
    begin_after_previous();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c = lane % LANES;
    const int parts = (2 * pool.kv_heads * split + kKvWarps - 1) / kKvWarps;    // of a tile
    const int tile_no = blockIdx.x / parts;
    int task = (blockIdx.x - tile_no * parts) * kKvWarps + warp;
    const int part = task % split;
    task /= split;
    int first, count;
    bool whole;
    const int i0 = load_tile<FMT != W4_KV_BF16>(pool, list, tile_no, tiles, 0x7FFFFFFF, L::kBytes,
                                                &tile, &first, &count, &whole);
    const bool is_v = task & 1;
    const int h = task >> 1;
    const long long head_bytes = (long long)h * pool.page_records * L::kBytes;
    if (count <= 0 || task >= 2 * pool.kv_heads || !(is_v ? v : k).data) return;
    __nv_bfloat16 *dst = reinterpret_cast<__nv_bfloat16 *>((is_v ? v : k).data) +
                         h * (is_v ? v : k).head_stride;
    const long long stride = (is_v ? v : k).token_stride;
    if constexpr (FMT != W4_KV_BF16) {
        if (whole && split == 1) {
            const unsigned char *rec = tile.record[0] + head_bytes;
            if (is_v)
                read_values<FMT, D>(rec, turned[warp], dst + i0 * stride, stride);
            else
                read_keys<FMT, D>(rec, dst + i0 * stride, stride);
            return;
        }
    }
    dst += 8 * c;
#pragma unroll 2
    for (int x0 = part; x0 < STEPS; x0 += split) {
        const int n = x0 * TOKENS + lane / LANES, r = min(first + n, kRecTokens - 1);
        if (n >= count || !tile.record[r]) continue;
        const int rr = tile.in_record[r];
        const unsigned char *rec = tile.record[r] + head_bytes;
        uint4 packed;
        if constexpr (FMT == W4_KV_BF16) {
            packed = *reinterpret_cast<const uint4 *>(
                rec + (is_v ? L::value(rr, 8 * c) : L::key(rr, 8 * c)));
        } else {
            const uint32_t m = *reinterpret_cast<const uint32_t *>(
                rec + (is_v ? L::kMetaV : L::kMeta) + 4 * rr);
            uint32_t code[2] = {0u, 0u};
            if (is_v) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    code[i / 4] |= (uint32_t)rec[L::value(rr, 8 * c + i)] << (8 * (i % 4));
                if (FMT == W4_KV_INT4) {
                    code[0] = code[0] >> (4 * (c & 1)) & 0x0F0F0F0Fu;
                    code[1] = code[1] >> (4 * (c & 1)) & 0x0F0F0F0Fu;
                }
            } else if constexpr (FMT == W4_KV_INT8) {
                const uint2 w = *reinterpret_cast<const uint2 *>(rec + L::key(rr, 8 * c));
                code[0] = w.x, code[1] = w.y;
            } else {
                key_codes(*reinterpret_cast<const uint32_t *>(rec + L::key(rr, 8 * c)), code);
            }
            packed = row_values(code[0], code[1], twice(less_of(m)), twice(scale_of(m)));
        }
        *reinterpret_cast<uint4 *>(dst + (i0 + r) * stride) = packed;
    }
}

// Tiles that a run of `run` tokens can touch, wherever in a record it starts.
int tiles_of(int run) { return (run + 2 * (kRecTokens - 1)) / kRecTokens; }

// Warps that share a tile's keys (values) of a head: four where the time is that
// of one block, and always in bf16 (whose 16 bytes a lane have no other work);
// one where the blocks fill the GPU.  Writing and reading back 4096 tokens of 4
// heads of 128 in 8 bits (2056 warps of tiles): 23.9 us with four, 24.8 with one;
// 16384 tokens in 4 bits: 81.8, 64.3; 8192 tokens of 2 heads of 64: 16.9, 13.9.
int split_of(const KvPool &pool, int format, int head_dim, const TokenList &list, int tiles,
             int num_sms) {
    if (list.run <= 256 / head_dim) return 1;
    const long long warps = (long long)(list.tokens / list.run) * tiles * 2 * pool.kv_heads;
    return format == W4_KV_BF16 || warps < (long long)(head_dim / 8) * num_sms ? 4 : 1;
}
unsigned blocks_of(const KvPool &pool, const TokenList &list, int tiles, int split) {
    return (unsigned)(list.tokens / list.run * tiles) *
           ((2 * (unsigned)pool.kv_heads * split + kKvWarps - 1) / kKvWarps);
}

template <int D, int HEADS>
cudaError_t append_dim(const KvPool &pool, int format, const Heads &k, const Heads &v, Queries q,
                       const TokenList &list, const Rotation &rot, int num_sms,
                       cudaStream_t stream) {
    const int tiles = tiles_of(list.run), split = split_of(pool, format, D, list, tiles, num_sms);
    q.rows_blocks = blocks_of(pool, list, tiles, split);
    const dim3 grid(q.rows_blocks + (q.all + kKvThreads - 1) / kKvThreads);
    q.period = grid.x / q.rows_blocks;
    const bool whole = list.run >= kRecTokens;
    const auto kernel =
        format == W4_KV_BF16 ? append_kernel<W4_KV_BF16, D, HEADS, false>
        : format == W4_KV_INT8
            ? whole ? append_kernel<W4_KV_INT8, D, HEADS, true>
                    : append_kernel<W4_KV_INT8, D, HEADS, false>
            : whole ? append_kernel<W4_KV_INT4, D, HEADS, true>
                    : append_kernel<W4_KV_INT4, D, HEADS, false>;
    return launch_overlapped(kernel, grid, dim3(kKvThreads), 0, stream, pool, k, v, q, list, rot,
                             tiles, split);
}

template <int D>
cudaError_t read_dim(const KvPool &pool, int format, const Heads &k, const Heads &v,
                     const TokenList &list, int num_sms, cudaStream_t stream) {
    const int tiles = tiles_of(list.run);
    // (one warp takes a whole record: 4096 tokens in 8 bits 26.4 us, 28.3 with four)
    const int split = format != W4_KV_BF16 && list.run >= kRecTokens
                          ? 1
                          : split_of(pool, format, D, list, tiles, num_sms);
    const auto kernel = format == W4_KV_BF16   ? read_kernel<W4_KV_BF16, D>
                        : format == W4_KV_INT8 ? read_kernel<W4_KV_INT8, D>
                                               : read_kernel<W4_KV_INT4, D>;
    return launch_overlapped(kernel, dim3(blocks_of(pool, list, tiles, split)), dim3(kKvThreads),
                             0, stream, pool, k, v, list, tiles, split);
}

}  // namespace

cudaError_t launch_kv_append(const KvPool &pool, int format, int head_dim, const Heads &k,
                             const Heads &v, const Heads &q, const Heads &q_out, int q_heads,
                             const TokenList &list, const Rotation &rot, int num_sms,
                             cudaStream_t stream) {
    Queries qs = {q, q_out, q_heads, 1, 1, 0, 0, 1};
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
        return four ? append_dim<64, 4>(pool, format, k, v, qs, list, rot, num_sms, stream)
                    : append_dim<64, 1>(pool, format, k, v, qs, list, rot, num_sms, stream);
    return four ? append_dim<128, 4>(pool, format, k, v, qs, list, rot, num_sms, stream)
                : append_dim<128, 1>(pool, format, k, v, qs, list, rot, num_sms, stream);
}

cudaError_t launch_kv_read(const KvPool &pool, int format, int head_dim, const Heads &k,
                           const Heads &v, const TokenList &list, int num_sms,
                           cudaStream_t stream) {
    return head_dim == 64 ? read_dim<64>(pool, format, k, v, list, num_sms, stream)
                          : read_dim<128>(pool, format, k, v, list, num_sms, stream);
}

}  // namespace w4
