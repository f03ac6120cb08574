// Attention of the new tokens over the paged cache (w4_paged_attn), or over listed
// blocks of it (w4_sparse_attn).
//
// Mathematics.  For one key/value head the queries that share it (new tokens
// x query heads of the group, "rows") meet every cached token once:
//   S^T = K Q^T (16 keys x 8 rows a tensor-core tile), p = exp2(y - m),
//   O^T += V^T P^T, l += sum of p,
// with y the scores in units of log2 and m a reference within a few powers of
// two of the running maximum, so one pass over the records is enough.  Pieces
// of the length have their own (m, l, O) and are joined by
//   m = max m_i, l = sum 2^(m_i - m) l_i, O = sum 2^(m_i - m) O_i.
//
// Why this way round.  Keys and values are the long operands; with them as the
// 16-row operand of mma.m16n8k16 the eight columns are the rows, and the 7
// (28/4, 14/2) query heads of a group fill 7 of 8 columns of one token.  S^T's
// accumulator, packed to 16 bits and transposed by movmatrix, is the second
// product's column operand: nothing goes through shared memory.
//
// Quantised records.  The bits of a code u (or 16 u, a high nibble) are the
// binary16 number u 2^-24 (16 u 2^-24; the 1/16 goes into q): a key's operand is
// one logic operation a pair, and its sum of q starts at -z sum q.  A value's
// code becomes 1024 + u by one operation and u - z, exact, by another: left to
// one correction of the sum, z would make the sum over a long cache many times
// larger than what is left of it, and fp32 accumulation loses the difference.
// (The keys' products are 8 long.  With 1024 + z left in the scores, they were
// rounded at 1024 times the codes' unit and the 4-bit log-sum-exp was off by
// 2e-4.)  A key's scale multiplies its scores; a value's scale goes into its
// probability, p s_v = exp2(y + log2 s_v - m), m taken over that sum, so that p
// fits binary16 whatever the scales are.
//
// Roundings.  Scores, m, l and O are fp32; the second product takes p in 16 bits.
// Beside bfloat16 values, whose range binary16 does not have, that is bfloat16 (8
// bits), and what it leaves of p goes through a product of its own: the result's
// error against fp64 is that of its own rounding, 0.00165, instead of 0.0022.
// Where memory sets the time (one new token) this costs nothing; 8 new tokens
// over 8 ragged sequences of up to 8192 take 31.5 us instead of 30.2, 5 over 48 x
// 4096 of 64 39.0 instead of 34.4.  Beside codes p is binary16 (11 bits): the
// error is 0.00163 and 0.00168 (8 and 4 bits), where a second product would make
// it 0.00163 and 0.00167 for 65.8 us instead of 60.2 at 4 x 131072 in 4 bits.  l
// sums p before any rounding.
//
// Schedule.  The blocks, one per SM, divide the list (sequence, head, record)
// evenly among themselves, from the lengths on the device: block c takes the
// records from cut c to cut c + 1.  A head counts for some records more than it
// has, what it costs to start and to finish one: without that, blocks with many
// short heads came last, and 64 ragged sequences of up to 8192 tokens in 8 bits
// took 64 us instead of 50.  A cut that would leave only a few records of a head
// on one side moves to the head's border on that side (w4_attn_plan.cuh).
// The pieces of cut heads are joined by a second kernel, a few rows a block,
// whose launch overlaps the first one's end: left to the block that finished a
// head last, the joining of 5 pieces of 56 rows took 7 us.  In a block, two
// warps issue the copies, a record a bulk copy, running ahead over the block's
// whole stretch; the others form KG groups of QG: a group takes every KG-th
// record through its own ring, and its QG warps hold 8 NT rows each.
//
// Listed blocks (w4_sparse_attn).  A sequence's records are those of its listed
// blocks; the copying warps find their numbers, and the pages by these, ahead, and tell
// the others each record's own first key, so that everything else is as above.
// Measured: 64 ragged sequences reading 4096 tokens each in 8 bits 51.0 us (numbers and
// pages asked for in one go 52.4; the whole attention over 64 x 4096 tokens 51.9);
// 64 blocks of 64 out of 131072 tokens in bf16, one sequence, 10.6.
//
// Measured (28 query and 4 key/value heads of 128, one new token, captured calls;
// a copy reaches 6788 GB/s).  bf16, bound by HBM: 32 x 16384 tokens 160 us =
// 6700 GB/s; one sequence of 65536, 108 records a block, 30.0 us = 4480 GB/s,
// 9 us of it around the records.  8 bits: 64 ragged sequences of up to 8192
// 48.7 us = 5700 GB/s (other lengths up to 55).  4 bits: 4 x 131072 60.2 us = 4740
// GB/s, most of it the instructions of conversion and softmax, though no unit is
// full (58 % of the issue slots, ALU 46 %, tensor pipe 23 %, DRAM 59 %).
#include <atomic>

#include "w4_attn_plan.cuh"
#include "w4_attn_query.cuh"

namespace w4 {
namespace {

constexpr float kNone = -3.0e38f;      // reference of a row that has seen no key
constexpr float kLn2 = 0.693147180559945309417f;

__device__ __forceinline__ void ldsm4_t(uint32_t *r, uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ uint32_t transposed(uint32_t v) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}
__device__ __forceinline__ float log2_fast(float x) {
    float r;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}
// Two numbers >= 0 in two bfloat16 parts each, within 2^-16 of them.  The upper
// part is cut off, not rounded, and the rest is 2^-20 of the number too large, so
// that neither is 0 or negative where the number is not: times an infinite value
// both parts give the same.
__device__ __forceinline__ uint32_t split_bf16(float x, float y, uint32_t *rest) {
    const uint32_t a = __float_as_uint(x), b = __float_as_uint(y);
    *rest = pack_bf16(fmaf(x, 1.f + 0x1p-20f, -__uint_as_float(a & 0xFFFF0000u)),
                      fmaf(y, 1.f + 0x1p-20f, -__uint_as_float(b & 0xFFFF0000u)));
    return __byte_perm(a, b, 0x7632);
}
__device__ __forceinline__ uint32_t half2_add(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("add.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t half2_fma(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t r;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
    return r;
}

// LISTED: of the listed blocks' records (the last block's past its end too).
template <bool LISTED>
__device__ __forceinline__ Seq sequence(const AttnArgs &a, int b) {
    int len = max(a.lens[b], 0);
    const int room = a.pool.width * a.pool.page_tokens;
    if (len > room) {
        if (a.pool.error) atomicOr(a.pool.error, W4_KV_ERR_LENGTH);
        len = room;
    }
    if constexpr (LISTED) {
        Seq s;
        s.len = len, s.first = 0;
        const int listed = min(max(a.counts[b], 0), a.most);
        s.records = len ? listed * a.pool.page_records : 0;
        return s;
    }
    return seen_records(len, a.tokens, a.window);
}

// A warp's NT tiles of 8 rows: its share of Q, and the running m, l, O.
template <int FMT, int D, int NT>
struct Tile : Queries<FMT, D, NT> {
    using L = KvLayout<FMT, D>;
    using Queries<FMT, D, NT>::KS;                 // k-steps of S, m-tiles of O
    using Queries<FMT, D, NT>::qf;
    using Queries<FMT, D, NT>::sc;
    using Queries<FMT, D, NT>::qs;
    static constexpr float kBias = FMT == W4_KV_BF16 ? 0.f : 6.f;
    static constexpr float kSlack = FMT == W4_KV_BF16 ? 8.f : 14.f;

    float o[NT][KS][4];
    float m[NT][2], l[NT][2];    // columns 2t, 2t + 1 of each tile
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int k = 0; k < KS; ++k)
#pragma unroll
                for (int c = 0; c < 4; ++c) o[n][k][c] = 0.f;
#pragma unroll
            for (int c = 0; c < 2; ++c) m[n][c] = kNone, l[n][c] = 0.f;
        }
    }

    // Values' operands of four codes: bytes 0, 2 (1, 3) of a word of 8-bit codes,
    // or the low (high) nibbles of bytes 0, 2; minus: -(1024 + z) of their keys
    // (high nibbles: (1024 + 16 u) / 16 - (64 + z)).
    __device__ static uint32_t even(uint32_t w, uint32_t minus) {
        return half2_add(and_or(w, 0x00FF00FFu, 0x64006400u), minus);
    }
    __device__ static uint32_t odd(uint32_t w, uint32_t minus) {
        return half2_add(__byte_perm(w, 0x64646464u, 0x4341), minus);
    }
    __device__ static uint32_t low(uint32_t w, uint32_t minus) {
        return half2_add(and_or(w, 0x000F000Fu, 0x64006400u), minus);
    }
    __device__ static uint32_t high(uint32_t w, uint32_t minus) {
        return half2_fma(and_or(w, 0x00F000F0u, 0x64006400u), 0x2C002C00u, minus);
    }

    // One record in shared memory, its first key j0 (kAbsent: there is none).
    // edge: some row does not see all of it.  (Two records a step, for more
    // independent instructions, measured 4 to 30 % slower: it halves what the
    // rings hold ahead.)
    __device__ __forceinline__ void record(const AttnArgs &a, uint32_t rec, int j0, bool edge,
                                           int len, int row0, int rows) {
        const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
        float s[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int c = 0; c < 4; ++c) s[n][c] = 0.f;
        // ---- S^T = K Q^T
        uint32_t mk[2], mv[2];                            // descriptors of keys g, g + 8
        if constexpr (FMT == W4_KV_BF16) {
            // piece 2 ks + hi of a row is stored at ^ (row & 7): only four
            // addresses differ, the others are 128 bytes on
            const uint32_t row = rec + (lane & 15) * L::kRow, swap = lane & 7, hi = lane >> 4;
#pragma unroll
            for (int ks = 0; ks < 4; ++ks) {
                const uint32_t at = row + (((2 * ks + hi) ^ swap) << 4);
                uint32_t k4[D / 64][4];
#pragma unroll
                for (int y = 0; y < D / 64; ++y) ldsm4(k4[y], at + 128 * y);
#pragma unroll
                for (int y = 0; y < D / 64; ++y)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
                        mma_bf16_16816(s[n], k4[y][0], k4[y][1], k4[y][2], k4[y][3],
                                       qf[n][ks + 4 * y][0], qf[n][ks + 4 * y][1]);
            }
        } else {
            uint32_t w0[D * L::kBits / 128], w1[D * L::kBits / 128];   // keys g, g + 8
            const uint32_t r0 = rec + g * L::kRow, r1 = r0 + 8 * L::kRow;
            if constexpr (FMT == W4_KV_INT8) {
#pragma unroll
                for (int i = 0; i < D / 64; ++i) {
                    const int piece = D == 128 ? (4 * i + t) ^ ((g & 1) << 2) : t;
                    lds128(w0 + 4 * i, r0 + piece * 16);
                    lds128(w1 + 4 * i, r1 + piece * 16);
                }
            } else if constexpr (D == 128) {
                lds128(w0, r0 + t * 16);
                lds128(w1, r1 + t * 16);
            } else {
                lds64(w0, r0 + t * 8);
                lds64(w1, r1 + t * 8);
            }
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                mk[r] = lds32(rec + L::kMeta + 4 * (g + 8 * r));
                mv[r] = lds32(rec + L::kMetaV + 4 * (g + 8 * r));
                const float z = __uint_as_float(__byte_perm(mk[r], 0x4B000000u, 0x7332)) - 0x1p23f;
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int c = 0; c < 2; ++c) s[n][2 * r + c] = z * qs[n][c];
            }
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                uint32_t a0, a1, a2, a3;
                if constexpr (FMT == W4_KV_INT8) {
                    a0 = w0[ks] & 0x00FF00FFu, a1 = w1[ks] & 0x00FF00FFu;
                    a2 = __byte_perm(w0[ks], 0u, 0x4341), a3 = __byte_perm(w1[ks], 0u, 0x4341);
                } else {
                    const uint32_t x0 = ks & 1 ? w0[ks >> 1] >> 8 : w0[ks >> 1];
                    const uint32_t x1 = ks & 1 ? w1[ks >> 1] >> 8 : w1[ks >> 1];
                    a0 = x0 & 0x000F000Fu, a1 = x1 & 0x000F000Fu;
                    a2 = x0 & 0x00F000F0u, a3 = x1 & 0x00F000F0u;
                }
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    mma_f16_16816(s[n], a0, a1, a2, a3, qf[n][ks][0], qf[n][ks][1]);
            }
        }
        // quantised values are on their way during the softmax
        uint32_t mt[2][2], vraw[FMT == W4_KV_BF16 ? 1 : L::kPart / 128];
        if constexpr (FMT != W4_KV_BF16) {
#pragma unroll
            for (int i = 0; i < L::kPart / 512; ++i)
                lds128(vraw + 4 * i, rec + L::kPart + i * 512 + lane * 16);
#pragma unroll
            for (int r = 0; r < 2; ++r) lds64(mt[r], rec + L::kMetaV + 4 * (2 * t + 8 * r));
        }
        // ---- scores in units of log2; quantised: with log2 s_v added
        float inv[2] = {1.f, 1.f};                        // 1 / s_v of keys g, g + 8
        if constexpr (FMT == W4_KV_BF16) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int c = 0; c < 4; ++c) s[n][c] *= sc[n][c & 1];
        } else {
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const float sk =
                    __half2float(__ushort_as_half((unsigned short)(mk[r] & 0xFFFFu)));
                // a value's scale of 0 goes with codes of 0: any factor does
                const float sv = fmaxf(
                    __half2float(__ushort_as_half((unsigned short)(mv[r] & 0xFFFFu))), 0x1p-24f);
                const float lv = log2_fast(sv);
                inv[r] = exp2_fast(-lv);
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int c = 0; c < 2; ++c)
                        s[n][2 * r + c] = fmaf(s[n][2 * r + c] * sc[n][c], sk, lv);
            }
        }
        uint32_t keep[2];
        bool apart = false;       // not finite, seen by some rows and not by others
        if (edge) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const int j = j0 + g + (c & 2) * 4;
                    const int last = len - a.tokens + token_of(a, n, c & 1, row0, rows);
                    if (j > last || (a.window > 0 && j <= last - a.window)) s[n][c] = -INFINITY;
                }
            if constexpr (FMT == W4_KV_BF16) {
                // values of keys that no row sees must not meet the product
                kept_keys(j0, a.window > 0 ? len - a.tokens - a.window : -1, len - 1, keep);
                if (a.tokens > 1) apart = __any_sync(0xFFFFFFFFu, !finite_values(rec, keep));
            }
        }
        // ---- a reference near the maximum: moved only when a score passes it by kSlack
        float top[NT][2];
        bool over = false;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                top[n][c] = fmaxf(s[n][c], s[n][c + 2]);
                over |= top[n][c] > m[n][c] + kSlack;
            }
        if (__any_sync(0xFFFFFFFFu, over)) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
#pragma unroll
                    for (int x = 4; x < 32; x <<= 1)
                        top[n][c] = fmaxf(top[n][c], __shfl_xor_sync(0xFFFFFFFFu, top[n][c], x));
                    const float now = fmaxf(m[n][c], top[n][c] - kBias);
                    const float f = exp2_fast(m[n][c] - now);
                    m[n][c] = now;
                    l[n][c] *= f;
#pragma unroll
                    for (int k = 0; k < KS; ++k) {
                        o[n][k][c] *= f;
                        o[n][k][c + 2] *= f;
                    }
                }
        }
        // ---- probabilities, their sums, and P^T as the column operand
        uint32_t p[NT][2], rest[FMT == W4_KV_BF16 ? NT : 1][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                s[n][c] = exp2_fast(s[n][c] - m[n][c & 1]);
                l[n][c & 1] = fmaf(s[n][c], inv[c >> 1], l[n][c & 1]);
            }
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                if constexpr (FMT == W4_KV_BF16) {
                    uint32_t less;
                    p[n][r] = transposed(split_bf16(s[n][2 * r], s[n][2 * r + 1], &less));
                    rest[n][r] = transposed(less);
                } else {
                    p[n][r] = transposed(pack_half(s[n][2 * r], s[n][2 * r + 1]));
                }
            }
        }
        // ---- O^T += V^T P^T
        if constexpr (FMT == W4_KV_BF16) {
            if (apart) {
#pragma unroll 1
                for (int part = 0; part < 2; ++part) {
                    tokens_apart(a, rec, j0, len, row0, rows, p);
#pragma unroll
                    for (int n = 0; n < NT; ++n) p[n][0] = rest[n][0], p[n][1] = rest[n][1];
                }
                return;
            }
            const uint32_t swap = lane & 7, hi = (lane >> 3) & 1;
            const uint32_t row = rec + L::kPart + ((lane >> 4) * 8 + swap) * L::kRow;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                uint32_t v4[D / 64][4];
                const uint32_t at = row + (((2 * k + hi) ^ swap) << 4);
#pragma unroll
                for (int y = 0; y < D / 64; ++y) {
                    ldsm4_t(v4[y], at + 128 * y);
                    if (edge)
#pragma unroll
                        for (int i = 0; i < 4; ++i) v4[y][i] &= keep[i >> 1];
                }
#pragma unroll
                for (int y = 0; y < D / 64; ++y)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
                        mma_bf16_16816(o[n][k + 4 * y], v4[y][0], v4[y][1], v4[y][2], v4[y][3],
                                       p[n][0], p[n][1]);
#pragma unroll
                for (int y = 0; y < D / 64; ++y)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
                        mma_bf16_16816(o[n][k + 4 * y], v4[y][0], v4[y][1], v4[y][2], v4[y][3],
                                       rest[n][0], rest[n][1]);
            }
        } else {
            uint32_t zlo[2], zhi[2];                      // -(1024 + z), -(64 + z)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                zlo[r] = (__byte_perm(mt[r][0], mt[r][1], 0x7632) & 0x00FF00FFu) | 0xE400E400u;
                zhi[r] = half2_add(zlo[r], 0x63806380u);
            }
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                uint32_t a0, a1, a2, a3;
                if constexpr (FMT == W4_KV_INT8) {
                    const uint32_t u = vraw[2 * k], v = vraw[2 * k + 1];
                    a0 = even(u, zlo[0]), a1 = even(v, zlo[0]);
                    a2 = odd(u, zlo[1]), a3 = odd(v, zlo[1]);
                } else {
                    const uint32_t u = vraw[k], v = vraw[k] >> 8;
                    a0 = low(u, zlo[0]), a1 = high(u, zhi[0]);
                    a2 = low(v, zlo[1]), a3 = high(v, zhi[1]);
                }
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    mma_f16_16816(o[n][k], a0, a1, a2, a3, p[n][0], p[n][1]);
            }
        }
    }

    // bf16: whether the kept values of a record that this lane takes are all
    // finite.
    __device__ static bool finite_values(uint32_t rec, const uint32_t (&keep)[2]) {
        const int lane = threadIdx.x & 31;
        bool ok = true;
#pragma unroll 1
        for (int k = 0; k < KS; ++k) {
            uint32_t v4[4];
            ldsm4_t(v4, value_piece(rec, lane, k));
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t v = v4[i] & keep[i >> 1];
                ok &= (v & 0x7F80u) != 0x7F80u && (v & 0x7F800000u) != 0x7F800000u;
            }
        }
        return ok;
    }

    // Address of the row that a lane gives for m-tile k of the values.
    __device__ static uint32_t value_piece(uint32_t rec, int lane, int k) {
        const uint32_t swap = lane & 7, hi = (lane >> 3) & 1;
        return rec + L::kPart + ((lane >> 4) * 8 + swap) * L::kRow + (((2 * k + hi) ^ swap) << 4);
    }

    // New token of column 2t + c of tile n.
    __device__ static int token_of(const AttnArgs &a, int n, int c, int row0, int rows) {
        return token_of_row(a, min(row0 + 8 * n + 2 * ((int)threadIdx.x & 3) + c, rows - 1));
    }

    // Masks of the keys 2t, 2t + 1 and 2t + 8, 2t + 9 of a record that lie in
    // (lo, last].
    __device__ static void kept_keys(int j0, int lo, int last, uint32_t (&keep)[2]) {
        const int t = threadIdx.x & 3;
        const auto seen = [&](int k) { return j0 + k <= last && j0 + k > lo; };
#pragma unroll
        for (int r = 0; r < 2; ++r)
            keep[r] = (seen(2 * t + 8 * r) ? 0xFFFFu : 0u) |
                      (seen(2 * t + 8 * r + 1) ? 0xFFFF0000u : 0u);
    }

    // The second product where a value that is not finite lies among keys that
    // some tokens see and others do not: 0 * inf would reach the rows that do
    // not see it, so each token's rows get a product of their own over the
    // keys that they see.
    __device__ __forceinline__ void tokens_apart(const AttnArgs &a, uint32_t rec, int j0, int len,
                                                 int row0, int rows, const uint32_t (&p)[NT][2]) {
        const int lane = threadIdx.x & 31;
#pragma unroll 1
        for (int i = 0; i < a.tokens; ++i) {
            const int last = len - a.tokens + i;
            uint32_t keep[2];
            kept_keys(j0, a.window > 0 ? last - a.window : -1, last, keep);
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                uint32_t v[4];
                ldsm4_t(v, value_piece(rec, lane, k));
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    float d[4] = {o[n][k][0], o[n][k][1], o[n][k][2], o[n][k][3]};
                    mma_bf16_16816(d, v[0] & keep[0], v[1] & keep[0], v[2] & keep[1],
                                   v[3] & keep[1], p[n][0], p[n][1]);
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        if (token_of(a, n, c & 1, row0, rows) == i) o[n][k][c] = d[c];
                }
            }
        }
    }

};

// The workspace: of every block, the head that it starts and others go on with
// (pieces = 0: none), then two pieces of rows: float [64][D], m [64], l [64].
struct CutHead {
    int b, h, tile0, pieces;
};
constexpr int kHeadBytes = kMaxGrid * sizeof(CutHead);
__device__ __forceinline__ CutHead *cut_head(const AttnArgs &a, int block) {
    return static_cast<CutHead *>(a.workspace) + block;
}
template <int D>
__device__ __forceinline__ float *slot_of(const AttnArgs &a, int block, bool starts) {
    return reinterpret_cast<float *>(static_cast<char *>(a.workspace) + kHeadBytes) +
           (size_t)(2 * block + (starts ? 1 : 0)) * kRowsMax * (D + 2);
}

// Four values of a row, l and m its sum and reference.  (With the approximate
// division and logarithm here the kernel's main loop, of all things, compiled
// to 40 % more time for 4-bit caches.)
__device__ __forceinline__ void store_row(const AttnArgs &a, int b, int h, int row, int d,
                                          float4 o, float m, float l) {
    const int i = token_of_row(a, row), hq = h * a.group + row - i * a.group;
    const long long t = (long long)b * a.tokens + i;
    const float f = l > 0.f ? 1.f / l : l;                     // 0 and NaN stay
    const long long at = t * a.out.token_stride + (long long)hq * a.out.head_stride + d;
    if (a.f32_out) {
        *reinterpret_cast<float4 *>(reinterpret_cast<float *>(a.out.data) + at) =
            make_float4(o.x * f, o.y * f, o.z * f, o.w * f);
    } else {
        *reinterpret_cast<uint2 *>(reinterpret_cast<__nv_bfloat16 *>(a.out.data) + at) =
            make_uint2(pack_bf16(o.x * f, o.y * f), pack_bf16(o.z * f, o.w * f));
    }
    if (a.lse && d == 0)
        a.lse[t * a.q_heads + hq] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

__device__ __forceinline__ void add_scaled(float4 &o, float f, const float4 &v) {
    o.x = fmaf(f, v.x, o.x), o.y = fmaf(f, v.y, o.y);
    o.z = fmaf(f, v.z, o.z), o.w = fmaf(f, v.w, o.w);
}

// The list, as a warp sees it: lane i holds sequences [b0, b1), whose items
// cost [before, before + mine) * per_seq.
template <bool LISTED>
struct List : Division {
    int b0, b1, before, mine;

    __device__ __forceinline__ int records(const AttnArgs &a, int b) const {
        return sequence<LISTED>(a, b).records;
    }

    __device__ __forceinline__ List(const AttnArgs &a, const Plan &plan) {
        const int lane = threadIdx.x & 31, each = (a.pool.seqs + 31) >> 5;
        extra = plan.extra;
        per_seq = a.pool.kv_heads * plan.row_tiles;
        b0 = min(lane * each, a.pool.seqs), b1 = min(b0 + each, a.pool.seqs);
        mine = 0;
#pragma unroll 4
        for (int b = b0; b < b1; ++b) mine += records(a, b) + extra;
        int upto = mine;
        if (a.pool.seqs > 1) {
#pragma unroll
            for (int x = 1; x < 32; x <<= 1) {
                const int v = __shfl_up_sync(0xFFFFFFFFu, upto, x);
                if (lane >= x) upto += v;
            }
        }
        before = upto - mine;
        const int all = __shfl_sync(0xFFFFFFFFu, upto, a.pool.seqs > 1 ? 31 : 0) * per_seq;
        divide(plan, a.pool.seqs, all, gridDim.x);
    }

    // The cut at cost u of the list.
    __device__ __forceinline__ Cut cut(const AttnArgs &a, int u) const {
        const bool here = u >= before * per_seq && u < (before + mine) * per_seq;
        int b = b0, n = mine - extra, in = u - before * per_seq;
        if (a.pool.seqs > 1) {
            if (here)
                for (;; ++b) {
                    n = records(a, b);
                    if (in < (n + extra) * per_seq) break;
                    in -= (n + extra) * per_seq;
                }
        }
        const unsigned found = __ballot_sync(0xFFFFFFFFu, here);
        const int src = found ? __ffs(found) - 1 : 0;
        b = __shfl_sync(0xFFFFFFFFu, b, src);
        n = __shfl_sync(0xFFFFFFFFu, n, src);
        in = __shfl_sync(0xFFFFFFFFu, in, src);
        if (found) return cut_inside(b, in, n);
        Cut end;                                              // of the list
        end.b = a.pool.seqs, end.item = 0, end.u = 0;
        return end;
    }
};

// Barrier over the warps that compute.
template <int WARPS>
__device__ __forceinline__ void warps_sync() {
    asm volatile("bar.sync 1, %0;" ::"n"(32 * WARPS) : "memory");
}

// Joins the pieces of the heads that blocks start and others go on with: block
// (c, y) rows ROWS y .. of block c's head, in the pieces' order.  256 / ROWS
// threads a row: groups of D / 4 take every other (or fourth) piece of it.  Bound
// by two trips to L2, about 2 us after the pieces are there.
template <int D, int ROWS>
__global__ void __launch_bounds__(256) join_kernel(const AttnArgs a, int block_rows) {
    constexpr int UNITS = D / 4, GROUPS = 256 / ROWS / UNITS;
    __shared__ float4 part[256];
    __shared__ float2 part_ml[256];
    begin_after_previous();
    const int4 head = __ldcg(reinterpret_cast<const int4 *>(cut_head(a, blockIdx.x)));
    const int tid = threadIdx.x, row = ROWS * blockIdx.y + tid / (GROUPS * UNITS);
    const int group = tid / UNITS % GROUPS, d = tid % UNITS * 4;
    if (head.w == 0) return;
    const bool there = row < min(block_rows, a.tokens * a.group - head.z);
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    float m = kNone, l = 0.f;
    if (there) {
        // AHEAD pieces are asked for together, however many there are: the
        // remainder of an unrolled loop would take a trip to L2 for each
        constexpr int AHEAD = 3;
        for (int c0 = group; c0 < head.w; c0 += GROUPS * AHEAD) {
            float4 v[AHEAD];
            float vm[AHEAD], vl[AHEAD];
#pragma unroll
            for (int x = 0; x < AHEAD; ++x) {
                const int c = c0 + x * GROUPS;
                const float *s = slot_of<D>(a, blockIdx.x + c, c == 0);
                v[x] = make_float4(0.f, 0.f, 0.f, 0.f);
                vm[x] = kNone, vl[x] = 0.f;
                if (c < head.w) {
                    v[x] = __ldcg(reinterpret_cast<const float4 *>(s + row * D + d));
                    vm[x] = __ldcg(s + kRowsMax * D + row);
                    vl[x] = __ldcg(s + kRowsMax * D + kRowsMax + row);
                }
            }
#pragma unroll
            for (int x = 0; x < AHEAD; ++x) {
                const float now = fmaxf(m, vm[x]), f = exp2_fast(m - now);
                const float g = exp2_fast(vm[x] - now);
                o = make_float4(o.x * f, o.y * f, o.z * f, o.w * f);
                add_scaled(o, g, v[x]);
                l = fmaf(l, f, vl[x] * g);
                m = now;
            }
        }
    }
    if (GROUPS > 1) {
        part[tid] = o, part_ml[tid] = make_float2(m, l);
        __syncthreads();
        if (group > 0) return;
#pragma unroll
        for (int x = 1; x < GROUPS; ++x) {
            const float2 ml = part_ml[tid + x * UNITS];
            const float now = fmaxf(m, ml.x), f = exp2_fast(m - now), g = exp2_fast(ml.x - now);
            o = make_float4(o.x * f, o.y * f, o.z * f, o.w * f);
            add_scaled(o, g, part[tid + x * UNITS]);
            l = fmaf(l, f, ml.y * g);
            m = now;
        }
    }
    if (there) store_row(a, head.x, head.y, head.z + row, d, o, m, l);
}

// A stretch's part of one head, as the copying warp tells the others.
struct Piece {
    int b;             // sequence; -1: no more pieces
    int h, tile0;      // key/value head, first row
    int u0, stop;      // records u0 .. stop - 1, from the sequence's first visible one
    int len;
    int whole;         // the head is not cut
    int starts;        // the piece starts the head
    int pieces;        // of a head that starts here and is cut
};

// The copying warps: lane i of warp w fills the ring of group 2 i + w.  Two of
// them, because a copy costs its warp about 100 cycles.
template <int FMT, int D, int WARPS, bool LISTED>
__device__ __forceinline__ void copy_records(const AttnArgs &a, const Plan &plan, int block_rows,
                                             unsigned char *smem, uint64_t *full, uint64_t *empty,
                                             int *first_key, Piece *piece, uint64_t *piece_full,
                                             uint64_t *piece_empty) {
    using L = KvLayout<FMT, D>;
    const int lane = threadIdx.x & 31, KG = plan.KG, stages = plan.stages;
    const int copier = (threadIdx.x >> 5) - WARPS, kg = kCopyWarps * lane + copier;
    const List<LISTED> list(a, plan);
    Cut c, to;
    c.b = 0, c.item = 0, c.u = 0;
    to = c;
    if ((int)blockIdx.x < list.blocks) {
        c = list.cut(a, list.start(blockIdx.x));
        to = list.cut(a, list.start(blockIdx.x + 1));
    }
    int put = 0, used = 0, told = 0;
    uint32_t phase = 1;
    bool ok = true;
    uint64_t *my_full = full + kg * stages, *my_empty = empty + kg * stages;
    unsigned char *ring = smem + kg * stages * L::kBytes;
    while (true) {
        const bool more = has_more(c, to, a.pool.seqs);
        const Seq seq = sequence<LISTED>(a, more ? c.b : 0);
        const bool last = c.b == to.b && c.item == to.item;
        const int stop = last ? to.u : seq.records;
        const int h = c.item / plan.row_tiles;
        const int32_t *pages = a.pool.table + (more ? c.b : 0) * a.pool.stride;
        constexpr int AHEAD = 4;
        int page[AHEAD];
        // LISTED: the block of page[x]; and the numbers of the one after, and of that
        // before it in the list, asked for as much earlier again
        constexpr int LISTS = LISTED ? AHEAD : 1;
        int block[LISTS], asked[LISTS], before[LISTS];
        const int32_t *blocks = nullptr;
        if constexpr (LISTED)
            blocks = a.blocks + ((long long)(more ? c.b : 0) * a.pool.kv_heads + h) * a.most;
        const auto ask = [&](int x, int u) {
            asked[x] = before[x] = -1;
            if (u < stop && kg < KG) {
                const int slot = page_slot(a.pool, u);
                asked[x] = blocks[slot];
                if (slot > 0) before[x] = blocks[slot - 1];
            }
        };
        const auto fetch = [&](int x, int u) {
            if constexpr (LISTED) {
                const int k = asked[x];
                const bool valid = u < stop && k > before[x] && k >= 0 &&
                                   (long long)k * a.pool.page_tokens < seq.len;
                block[x] = valid ? k : -1;
                page[x] = valid ? pages[k] : -1;
                ask(x, u + AHEAD * KG);
            } else {
                page[x] = u < stop && kg < KG ? pages[page_slot(a.pool, seq.first + u)] : 0;
            }
        };
        if (more) {
            if constexpr (LISTED) {
#pragma unroll
                for (int x = 0; x < AHEAD; ++x) ask(x, c.u + kg + x * KG);
            }
#pragma unroll
            for (int x = 0; x < AHEAD; ++x) fetch(x, c.u + kg + x * KG);
        }
        // tell the others, two pieces ahead at most (while the pages' numbers
        // are on their way)
        const int slot = told & 1;
        const bool tells = copier == 0 && lane == 0;
        if (copier == 0 && told >= 2 &&
            !__all_sync(0xFFFFFFFFu, mbar_wait(&piece_empty[slot], ((told >> 1) + 1) & 1))) {
            if (a.pool.error) atomicOr(a.pool.error, W4_KV_ERR_WAIT);   // never in normal operation
            break;
        }
        Piece &p = piece[slot];
        if (tells) {
            p.b = more ? c.b : -1;
            p.h = h, p.tile0 = (c.item - h * plan.row_tiles) * block_rows;
            p.u0 = c.u, p.stop = stop, p.len = seq.len;
            p.whole = c.u == 0 && stop == seq.records, p.starts = c.u == 0;
        }
        if (copier == 0 && more && c.u == 0 && stop != seq.records) {
            const bool mine = c.b >= list.b0 && c.b < list.b1;
            int head = list.before * list.per_seq + c.item * (seq.records + list.extra);
            if (mine)
                for (int x = list.b0; x < c.b; ++x)
                    head += (list.records(a, x) + list.extra) * list.per_seq;
            head = __shfl_sync(0xFFFFFFFFu, head, __ffs(__ballot_sync(0xFFFFFFFFu, mine)) - 1);
            const int pieces = list.pieces(head, seq.records);
            if (tells) p.pieces = pieces;
        }
        if (tells) mbar_arrive(&piece_full[slot]);
        ++told;
        if (!more) break;

        for (int u0 = c.u; u0 < stop; u0 += AHEAD * KG)
#pragma unroll
            for (int x = 0; x < AHEAD; ++x) {
                const int u = u0 + kg + x * KG, pg = page[x];
                // record of the sequence and of its page
                int r = seq.first + u, in_page = r - page_slot(a.pool, r) * a.pool.page_records;
                const int listed = LISTED ? block[x] : 0;
                if constexpr (LISTED) r = listed * a.pool.page_records + in_page;
                fetch(x, u + AHEAD * KG);
                const bool mine = kg < KG && u < stop && ok;
                // the lanes leave the wait one by one: without the barrier
                // each would go through the rest by itself
                if (mine && used >= stages) ok = mbar_wait(&my_empty[put], phase);
                __syncwarp();
                if (mine && ok) {
                    fence_proxy_async();
                    const bool known = pg >= 0 && pg < a.pool.pages;
                    // (records of the last listed block may lie past its end)
                    const bool valid = known && (!LISTED || r * kRecTokens < seq.len);
                    first_key[kg * stages + put] = valid ? r * kRecTokens : kAbsent;
                    if (valid) {
                        const char *src =
                            a.pool.records +
                            (((long long)pg * a.pool.kv_heads + h) * a.pool.page_records +
                             in_page) * L::kBytes;
                        mbar_expect_tx(&my_full[put], L::kBytes);
                        bulk_g2s(ring + put * L::kBytes, src, L::kBytes, &my_full[put]);
                    } else {
                        if (a.pool.error && !known)
                            atomicOr(a.pool.error, LISTED && listed < 0 ? W4_KV_ERR_BLOCK
                                                                        : W4_KV_ERR_PAGE);
                        mbar_arrive(&my_full[put]);
                    }
                    used = min(used + 1, stages);
                    if (++put == stages) put = 0, phase ^= 1;
                } else if (mine && a.pool.error) {
                    atomicOr(a.pool.error, W4_KV_ERR_WAIT);   // never in normal operation
                }
                __syncwarp();
            }
        __syncwarp();
        if (last) {
            c = to;
        } else {
            list.advance(c);
        }
    }
    // nothing of the block's own is under way when it ends
    phase ^= 1;
    for (int x = 0; x < used; ++x) {
        if (--put < 0) put = stages - 1, phase ^= 1;
        mbar_wait(&my_full[put], phase);
    }
}

template <int FMT, int D, int NT, bool LISTED>
__global__ void __launch_bounds__(32 * (compute_warps(D, NT) + kCopyWarps), 1)
attn_kernel(const AttnArgs a, const Plan plan) {
    extern __shared__ __align__(128) unsigned char smem[];
    using L = KvLayout<FMT, D>;
    constexpr int WARPS = compute_warps(D, NT);
    constexpr int OROW = D + 4;                               // floats; + 4: no bank conflicts
    __shared__ uint64_t full[WARPS * kMaxStages], empty[WARPS * kMaxStages];
    __shared__ uint64_t piece_full[2], piece_empty[2];
    __shared__ int first_key[WARPS * kMaxStages];             // of a stage's record, or kAbsent
    __shared__ float join_m[WARPS * 8 * NT], join_l[WARPS * 8 * NT];
    __shared__ Piece piece[2];
    const int block_rows = 8 * NT * plan.QG;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    for (int i = tid; i < plan.KG * plan.stages; i += 32 * (WARPS + kCopyWarps)) {
        mbar_init(&full[i], 1);
        mbar_init(&empty[i], plan.QG);
    }
    if (tid < 2) {
        mbar_init(&piece_full[tid], 1);
        mbar_init(&piece_empty[tid], WARPS);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    __syncthreads();
    begin_after_previous();
    if (warp >= WARPS) {
        copy_records<FMT, D, WARPS, LISTED>(a, plan, block_rows, smem, full, empty, first_key,
                                            piece, piece_full, piece_empty);
        return;
    }

    const int kg = warp / plan.QG, qg = warp - kg * plan.QG;
    const bool works = kg < plan.KG;                          // QG may not divide WARPS
    const uint32_t ring = smem_addr(smem) + kg * plan.stages * L::kBytes;
    int get = 0;
    uint32_t phase = 0;
    bool failed = false;
    CutHead started = {0, 0, 0, 0};
    Tile<FMT, D, NT> w;
    for (int told = 0;; ++told) {
        const Piece &p = piece[told & 1];
        if (!__all_sync(0xFFFFFFFFu, mbar_wait(&piece_full[told & 1], (told >> 1) & 1))) {
            if (a.pool.error) atomicOr(a.pool.error, W4_KV_ERR_WAIT);
            if (tid == 0) *cut_head(a, blockIdx.x) = {0, 0, 0, 0};
            return;                                           // every warp does
        }
        if (p.b < 0) {
            if (tid == 0) *cut_head(a, blockIdx.x) = started;
            return;
        }
        if (p.starts && !p.whole) started = {p.b, p.h, p.tile0, p.pieces};
        if (works && !failed) {
            const int rows = a.tokens * a.group, row0 = p.tile0 + qg * 8 * NT;
            w.load_q(a, p.b, p.h, row0, rows);
            w.clear();
            // every row sees all keys of [seen0, seen1)
            const int len = p.len, seen1 = len - a.tokens + 1;
            const int seen0 = a.window > 0 ? len - a.window : 0;
            uint64_t *my_full = full + kg * plan.stages, *my_empty = empty + kg * plan.stages;
            const int *keys = first_key + kg * plan.stages;
            for (int u = p.u0 + kg; u < p.stop; u += plan.KG) {
                if (!__all_sync(0xFFFFFFFFu, mbar_wait(&my_full[get], phase))) {
                    if (a.pool.error) atomicOr(a.pool.error, W4_KV_ERR_WAIT);
                    failed = true;                            // never in normal operation
                    break;
                }
                const int j0 = keys[get];
                w.record(a, ring + get * L::kBytes, j0, j0 + kRecTokens > seen1 || j0 < seen0, len,
                         row0, rows);
                __syncwarp();
                if (lane == 0) mbar_arrive(&my_empty[get]);
                if (++get == plan.stages) get = 0, phase ^= 1;
            }
        }

        // ---- join the groups of warps through shared memory
        float *join_o = reinterpret_cast<float *>(smem + plan.ring_bytes);
        if (works) {
            const int g = lane >> 2, t = lane & 3, own = kg * block_rows + qg * 8 * NT + 2 * t;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    float l = w.l[n][x];
#pragma unroll
                    for (int s = 4; s < 32; s <<= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, s);
                    const int r = own + 8 * n + x;
                    if (g == 0) join_m[r] = w.m[n][x], join_l[r] = l;
#pragma unroll
                    for (int k = 0; k < D / 16; ++k)
#pragma unroll
                        for (int y = 0; y < 2; ++y)
                            join_o[r * OROW + 16 * k + 8 * y + g] = w.o[n][k][2 * y + x];
                }
        }
        warps_sync<WARPS>();
        const int there = min(block_rows, a.tokens * a.group - p.tile0);
        float *slot = slot_of<D>(a, blockIdx.x, p.starts);
        for (int e = tid; e < there * (D / 4); e += 32 * WARPS) {
            const int r = e / (D / 4), d = e % (D / 4) * 4;
            float m = kNone, l = 0.f;
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
            for (int k = 0; k < plan.KG; ++k) m = fmaxf(m, join_m[k * block_rows + r]);
#pragma unroll 2
            for (int k = 0; k < plan.KG; ++k) {
                const int at = k * block_rows + r;
                const float f = exp2_fast(join_m[at] - m);
                l = fmaf(f, join_l[at], l);
                add_scaled(o, f, *reinterpret_cast<const float4 *>(&join_o[at * OROW + d]));
            }
            if (p.whole) {
                store_row(a, p.b, p.h, p.tile0 + r, d, o, m, l);
            } else {
                *reinterpret_cast<float4 *>(&slot[r * D + d]) = o;
                if (d == 0) slot[kRowsMax * D + r] = m, slot[kRowsMax * D + kRowsMax + r] = l;
            }
        }
        warps_sync<WARPS>();                                  // the join's memory is free again
        if (lane == 0) mbar_arrive(&piece_empty[told & 1]);
    }
}

template <int FMT, int D, int NT, bool LISTED>
cudaError_t launch(const AttnArgs &a, int num_sms, cudaStream_t stream) {
    constexpr int bytes = KvLayout<FMT, D>::kBytes, WARPS = compute_warps(D, NT);
    static std::atomic<bool> ready[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64 || !ready[dev].load(std::memory_order_relaxed)) {
        e = cudaFuncSetAttribute(attn_kernel<FMT, D, NT, LISTED>,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize, kSharedBytes);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) ready[dev].store(true, std::memory_order_relaxed);
    }
    const int rows = a.tokens * a.group;
    const Plan p =
        plan_of(D, NT, rows, bytes, LISTED ? listed_part(FMT == W4_KV_BF16, D) : kPart);
    const int grid = num_sms < kMaxGrid ? num_sms : kMaxGrid;
    e = launch_overlapped(attn_kernel<FMT, D, NT, LISTED>, dim3(grid), dim3(32 * (WARPS + kCopyWarps)),
                          kSharedBytes, stream, a, p);
    if (e != cudaSuccess) return e;
    if (nothing_to_join(p, a.pool.seqs, a.pool.kv_heads,
                        (long long)(LISTED ? a.most : a.pool.width) * a.pool.page_records, grid))
        return cudaSuccess;
    const int block_rows = 8 * NT * p.QG;
    constexpr int FEW = 2, MANY = 512 / D;                    // rows of a joining block
    if (rows <= 8)
        return launch_overlapped(join_kernel<D, FEW>, dim3(grid, (rows + FEW - 1) / FEW), dim3(256),
                                 0, stream, a, block_rows);
    return launch_overlapped(join_kernel<D, MANY>,
                             dim3(grid, ((rows < block_rows ? rows : block_rows) + MANY - 1) / MANY),
                             dim3(256), 0, stream, a, block_rows);
}

template <int FMT, int D, bool LISTED>
cudaError_t launch_rows(const AttnArgs &a, int num_sms, cudaStream_t stream) {
    return tiles_a_warp(D, a.tokens * a.group) == 2
               ? launch<FMT, D, 2, LISTED>(a, num_sms, stream)
               : launch<FMT, D, 1, LISTED>(a, num_sms, stream);
}

template <int D, bool LISTED>
cudaError_t launch_format(const AttnArgs &a, int format, int num_sms, cudaStream_t stream) {
    return format == W4_KV_BF16   ? launch_rows<W4_KV_BF16, D, LISTED>(a, num_sms, stream)
           : format == W4_KV_INT8 ? launch_rows<W4_KV_INT8, D, LISTED>(a, num_sms, stream)
                                  : launch_rows<W4_KV_INT4, D, LISTED>(a, num_sms, stream);
}

}  // namespace

size_t attn_workspace_bytes(int head_dim, int num_sms) {
    const int grid = num_sms < kMaxGrid ? num_sms : kMaxGrid;
    return kHeadBytes + (size_t)grid * 2 * kRowsMax * (head_dim + 2) * 4;
}

cudaError_t launch_paged_attn(const AttnArgs &a, int format, int head_dim, int num_sms,
                              cudaStream_t stream) {
    if (a.blocks)
        return head_dim == 128 ? launch_format<128, true>(a, format, num_sms, stream)
                               : launch_format<64, true>(a, format, num_sms, stream);
    return head_dim == 128 ? launch_format<128, false>(a, format, num_sms, stream)
                           : launch_format<64, false>(a, format, num_sms, stream);
}

}  // namespace w4
