// Attention of the new tokens over the paged cache (w4_paged_attn).
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
// Quantised records.  A code becomes the binary16 1024 + u (or 1024 + 16 u for
// a high nibble) by one logic operation a pair, and u - z, exact, by one
// addition (fma) a pair.  Leaving the products with 1024 + z to one correction
// per score would save the addition, but rounds the scores at 1024 times the
// codes' unit: the 4-bit log-sum-exp was then off by 2e-4.  A key's scale
// multiplies its scores; a value's scale goes into its probability,
// p s_v = exp2(y + log2 s_v - m), m taken over that sum, so that p fits
// binary16 whatever the scales are.
//
// Schedule.  The work, records x heads over all sequences, is divided evenly
// over the grid from the lengths on the device: block c takes records
// [c W / G, (c + 1) W / G) of the list (sequence, head, record).  A block's
// stretch may cover several heads or a part of one; the parts of a head are
// joined by the block that finishes it last, in block order.  In a block a
// group of warps takes every KG-th record through its own ring of bulk copies
// (one record is one copy).
#include <atomic>

#include "w4_device.cuh"
#include "w4_kv.cuh"

namespace w4 {
namespace {

constexpr float kNone = -3.0e38f;      // reference of a row that has seen no key
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.693147180559945309417f;

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
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
__device__ __forceinline__ float exp2_fast(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ uint32_t pack_half(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
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

// Shape of a block: KG groups of QG warps; a warp holds NT tiles of 8 rows.
template <int FMT_, int D_, int NT_, int QG_, int W_, int STAGES_, int BLOCKS_>
struct Cfg {
    static constexpr int FMT = FMT_, D = D_, NT = NT_, QG = QG_, W = W_, STAGES = STAGES_;
    static constexpr int BLOCKS = BLOCKS_;                // per SM
    static constexpr int KG = W / QG;
    static constexpr int THREADS = W * 32;
    static constexpr int ROWS = 8 * NT * QG;              // rows of a block
    using L = KvLayout<FMT, D>;
    static constexpr int RING = KG * STAGES * L::kBytes;
    static constexpr int OROW = D + 4;                    // floats; +4: no bank conflicts
    static constexpr int JOIN = KG * ROWS * OROW * 4;     // shares the ring's memory
    static constexpr int BUF = RING > JOIN ? RING : JOIN;
    static constexpr int ML = 2 * KG * ROWS * 4;
    static constexpr int SMEM = BUF + ML + 2 * KG * STAGES * 8 + 256;
    // floats of a joined piece in the workspace
    static constexpr int SLOT = 64 * (D + 2);
};

struct Seq {
    int len;           // visible tokens
    int first;         // first record with a visible key
    int records;       // records from there on (0: none)
};

__device__ __forceinline__ Seq sequence(const AttnArgs &a, int b) {
    Seq s;
    s.len = max(a.lens[b], 0);
    const int room = a.pool.width * a.pool.page_tokens;
    if (s.len > room) {
        if (a.pool.error) atomicOr(a.pool.error, W4_KV_ERR_LENGTH);
        s.len = room;
    }
    const long long lo = (long long)s.len - a.tokens + 1 - a.window;
    s.first = a.window > 0 && lo > 0 ? (int)(lo / kRecTokens) : 0;
    s.records = (s.len + kRecTokens - 1) / kRecTokens - s.first;
    return s;
}

template <typename C>
struct Warp {
    using L = typename C::L;
    static constexpr int D = C::D, NT = C::NT, FMT = C::FMT;
    static constexpr int KS = D / 16;                     // k-steps of S, m-tiles of O
    static constexpr float kBias = FMT == W4_KV_BF16 ? 0.f : 6.f;
    static constexpr float kSlack = FMT == W4_KV_BF16 ? 8.f : 14.f;

    uint32_t qf[NT][KS][2];      // Q as the column operand
    float o[NT][KS][4];
    float m[NT][2], l[NT][2];    // columns 2t, 2t + 1 of each tile
    float sc[NT][2];             // score factor of a column

    // Which value of the head goes with half e of register i of k-step ks.
    __device__ static int q_index(int ks, int i, int e, int t) {
        if (FMT == W4_KV_BF16) return 16 * ks + 8 * i + 2 * t + e;
        if (FMT == W4_KV_INT8) return 64 * (ks >> 2) + 16 * t + 4 * (ks & 3) + i + 2 * e;
        return (D / 4) * t + 8 * (ks >> 1) + 2 * (ks & 1) + i + 4 * e;
    }

    // row0: first row of this warp's tiles; rows: rows that there are.
    __device__ void load_q(const AttnArgs &a, int b, int h, int row0, int rows) {
        const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int r = row0 + 8 * n + g;
            const bool there = r < rows;
            const int i = there ? r / a.group : 0, hq = there ? r - i * a.group : 0;
            const __nv_bfloat16 *q = reinterpret_cast<const __nv_bfloat16 *>(a.q.data) +
                                     (long long)(b * a.tokens + i) * a.q.token_stride +
                                     (long long)(h * a.group + hq) * a.q.head_stride;
            if constexpr (FMT == W4_KV_BF16) {
#pragma unroll
                for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        qf[n][ks][j] = there ? *reinterpret_cast<const uint32_t *>(
                                                   q + q_index(ks, j, 0, t))
                                             : 0u;
                sc[n][0] = sc[n][1] = a.scale * kLog2e;
            } else {
                float v[KS][2][2], top = 0.f;
#pragma unroll
                for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                    for (int j = 0; j < 2; ++j)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            v[ks][j][e] =
                                there ? __bfloat162float(q[q_index(ks, j, e, t)]) : 0.f;
                            top = fmaxf(top, fabsf(v[ks][j][e]));
                        }
                top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
                // a power of two that brings the largest |q| into [2^14, 2^15):
                // q is exact in binary16 down to 2^-28 of it
                int e = 0;
                if (top > 0.f && top < INFINITY)
                    e = 14 - max(-86, (int)(__float_as_uint(top) >> 23) - 127);
                const float up = __int_as_float((127 + e) << 23);
#pragma unroll
                for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        qf[n][ks][j] = pack_half(v[ks][j][0] * up, v[ks][j][1] * up);
                const float f = a.scale * kLog2e * __int_as_float((127 - e) << 23);
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    sc[n][c] = __shfl_sync(0xFFFFFFFFu, f, 4 * (2 * t + c));
                }
            }
        }
    }

    __device__ void clear() {
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

    // Operands of four codes (two of key pair `lo`, two of the next): bytes 0, 2
    // and 1, 3 of a word of 8-bit codes; minus[]: -(1024 + z) of their keys.
    __device__ static uint32_t even(uint32_t w, uint32_t minus) {
        return half2_add(and_or(w, 0x00FF00FFu, 0x64006400u), minus);
    }
    __device__ static uint32_t low(uint32_t w, uint32_t minus) {
        return half2_add(and_or(w, 0x000F000Fu, 0x64006400u), minus);
    }
    // high nibbles: (1024 + 16 u) / 16 - (64 + z)
    __device__ static uint32_t high(uint32_t w, uint32_t minus) {
        return half2_fma(and_or(w, 0x00F000F0u, 0x64006400u), 0x2C002C00u, minus);
    }

    // One record in shared memory, its first key j0.  edge: some row does not
    // see all of it.
    __device__ void record(const AttnArgs &a, uint32_t rec, int j0, bool edge, int len, int row0,
                           int rows) {
        const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
        float s[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int c = 0; c < 4; ++c)
                s[n][c] = 0.f;
        // ---- S^T = K Q^T
        uint32_t mk[2], zk[2], zk16[2];      // keys g, g + 8: -(1024 + z), -(64 + z), twice each
        if constexpr (FMT != W4_KV_BF16) {
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                mk[r] = lds32(rec + L::kMeta + 4 * (g + 8 * r));
                const uint32_t z = __byte_perm(mk[r], 0u, 0x4242);
                zk[r] = z | 0xE400E400u;
                zk16[r] = half2_add(zk[r], 0x63806380u);  // + 960
            }
        }
        if constexpr (FMT == W4_KV_BF16) {
            const int r = ((lane >> 3) & 1) * 8 + (lane & 7), hi = lane >> 4;
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                uint32_t k4[4];
                ldsm4(k4, rec + r * L::kRow + (((2 * ks + hi) ^ (r & 7)) << 4));
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    mma_bf16_16816(s[n], k4[0], k4[1], k4[2], k4[3], qf[n][ks][0], qf[n][ks][1]);
            }
        } else if constexpr (FMT == W4_KV_INT8) {
#pragma unroll
            for (int i = 0; i < D / 64; ++i) {
                uint32_t w0[4], w1[4];
                const int piece = D == 128 ? (4 * i + t) ^ ((g & 1) << 2) : t;
                lds128(w0, rec + g * L::kRow + piece * 16);
                lds128(w1, rec + (g + 8) * L::kRow + piece * 16);
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    const uint32_t a0 = even(w0[w], zk[0]), a1 = even(w1[w], zk[1]);
                    const uint32_t a2 = even(w0[w] >> 8, zk[0]), a3 = even(w1[w] >> 8, zk[1]);
#pragma unroll
                    for (int n = 0; n < NT; ++n)
                        mma_f16_16816(s[n], a0, a1, a2, a3, qf[n][4 * i + w][0],
                                      qf[n][4 * i + w][1]);
                }
            }
        } else {
            uint32_t w0[D / 32], w1[D / 32];
            if constexpr (D == 128) {
                lds128(w0, rec + g * L::kRow + t * 16);
                lds128(w1, rec + (g + 8) * L::kRow + t * 16);
            } else {
                lds64(w0, rec + g * L::kRow + t * 8);
                lds64(w1, rec + (g + 8) * L::kRow + t * 8);
            }
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                const uint32_t x0 = ks & 1 ? w0[ks >> 1] >> 8 : w0[ks >> 1];
                const uint32_t x1 = ks & 1 ? w1[ks >> 1] >> 8 : w1[ks >> 1];
                const uint32_t a0 = low(x0, zk[0]), a1 = low(x1, zk[1]);
                const uint32_t a2 = high(x0, zk16[0]), a3 = high(x1, zk16[1]);
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    mma_f16_16816(s[n], a0, a1, a2, a3, qf[n][ks][0], qf[n][ks][1]);
            }
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
                const uint32_t mv = lds32(rec + L::kMetaV + 4 * (g + 8 * r));
                const float sk =
                    __half2float(__ushort_as_half((unsigned short)(mk[r] & 0xFFFFu)));
                // a value's scale of 0 goes with codes of 0: any factor does
                const float sv = fmaxf(
                    __half2float(__ushort_as_half((unsigned short)(mv & 0xFFFFu))), 0x1p-24f);
                const float lv = __log2f(sv);
                inv[r] = exp2_fast(-lv);
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int c = 0; c < 2; ++c)
                        s[n][2 * r + c] = fmaf(s[n][2 * r + c], sk * sc[n][c], lv);
            }
        }
        uint32_t keep0 = 0xFFFFFFFFu, keep1 = 0xFFFFFFFFu;    // keys 2t, 2t+1; 2t+8, 2t+9
        bool apart = false;       // a key that some rows see and some do not
        if (edge) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const int row = row0 + 8 * n + 2 * t + (c & 1), j = j0 + g + (c & 2) * 4;
                    const int last = len - a.tokens + min(row, rows - 1) / a.group;
                    if (j > last || (a.window > 0 && j <= last - a.window)) s[n][c] = -INFINITY;
                }
            if constexpr (FMT == W4_KV_BF16) {
                // values of keys that no row sees must not meet the product
                const int lo = a.window > 0 ? len - a.tokens - a.window : -1;
                const auto seen = [&](int k) { return j0 + k < len && j0 + k > lo; };
                keep0 = (seen(2 * t) ? 0xFFFFu : 0u) | (seen(2 * t + 1) ? 0xFFFF0000u : 0u);
                keep1 = (seen(2 * t + 8) ? 0xFFFFu : 0u) | (seen(2 * t + 9) ? 0xFFFF0000u : 0u);
                apart = a.tokens > 1;
            }
        }
        // ---- a reference near the maximum: moved only when a score passes it by kSlack
        bool over = false;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int c = 0; c < 4; ++c) over |= s[n][c] > m[n][c & 1] + kSlack;
        if (__any_sync(0xFFFFFFFFu, over)) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    float top = fmaxf(s[n][c], s[n][c + 2]);
#pragma unroll
                    for (int x = 4; x < 32; x <<= 1)
                        top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, x));
                    const float now = fmaxf(m[n][c], top - kBias);
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
        uint32_t p[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                s[n][c] = exp2_fast(s[n][c] - m[n][c & 1]);
                l[n][c & 1] = fmaf(s[n][c], inv[c >> 1], l[n][c & 1]);
            }
#pragma unroll
            for (int r = 0; r < 2; ++r)
                p[n][r] = transposed(FMT == W4_KV_BF16 ? pack_bf16(s[n][2 * r], s[n][2 * r + 1])
                                                       : pack_half(s[n][2 * r], s[n][2 * r + 1]));
        }
        // ---- O^T += V^T P^T
        if constexpr (FMT == W4_KV_BF16) {
            const int r = (lane >> 4) * 8 + (lane & 7), hi = (lane >> 3) & 1;
            const uint32_t base = rec + L::kPart + r * L::kRow;
            if (apart && __any_sync(0xFFFFFFFFu, !finite_values(base, r, hi, keep0, keep1))) {
                tokens_apart(a, base, r, hi, j0, len, row0, rows, p);
                return;
            }
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                uint32_t v4[4];
                ldsm4_t(v4, base + (((2 * k + hi) ^ (r & 7)) << 4));
                if (edge) v4[0] &= keep0, v4[1] &= keep0, v4[2] &= keep1, v4[3] &= keep1;
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    mma_bf16_16816(o[n][k], v4[0], v4[1], v4[2], v4[3], p[n][0], p[n][1]);
            }
        } else {
            uint32_t zlo[2], zhi[2];                      // minus (1024 + z), (64 + z)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                uint32_t mv[2];
                lds64(mv, rec + L::kMetaV + 4 * (2 * t + 8 * r));
                const uint32_t z = __byte_perm(mv[0], mv[1], 0x7632) & 0x00FF00FFu;
                zlo[r] = z | 0xE400E400u;
                zhi[r] = half2_add(zlo[r], 0x63806380u);  // + 960
            }
#pragma unroll
            for (int i = 0; i < L::kPart / 512; ++i) {
                uint32_t w[4];
                lds128(w, rec + L::kPart + i * 512 + lane * 16);
                if constexpr (FMT == W4_KV_INT8) {
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const uint32_t u = w[2 * x], v = w[2 * x + 1];
                        const uint32_t a0 = even(u, zlo[0]), a1 = even(v, zlo[0]);
                        const uint32_t a2 = even(u >> 8, zlo[1]), a3 = even(v >> 8, zlo[1]);
#pragma unroll
                        for (int n = 0; n < NT; ++n)
                            mma_f16_16816(o[n][2 * i + x], a0, a1, a2, a3, p[n][0], p[n][1]);
                    }
                } else {
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const uint32_t u = w[x], v = w[x] >> 8;
                        const uint32_t a0 = low(u, zlo[0]), a1 = high(u, zhi[0]);
                        const uint32_t a2 = low(v, zlo[1]), a3 = high(v, zhi[1]);
#pragma unroll
                        for (int n = 0; n < NT; ++n)
                            mma_f16_16816(o[n][4 * i + x], a0, a1, a2, a3, p[n][0], p[n][1]);
                    }
                }
            }
        }
    }

    __device__ static void lds128(uint32_t *r, uint32_t addr) {
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                     : "r"(addr)
                     : "memory");
    }
    __device__ static void lds64(uint32_t *r, uint32_t addr) {
        asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];"
                     : "=r"(r[0]), "=r"(r[1])
                     : "r"(addr)
                     : "memory");
    }
    __device__ static uint32_t lds32(uint32_t addr) {
        uint32_t r;
        asm volatile("ld.shared.u32 %0, [%1];" : "=r"(r) : "r"(addr) : "memory");
        return r;
    }

    // Whether the kept values that this lane takes are all finite.
    __device__ static bool finite_values(uint32_t base, int r, int hi, uint32_t keep0,
                                         uint32_t keep1) {
        bool ok = true;
        for (int k = 0; k < KS; ++k) {
            uint32_t v4[4];
            ldsm4_t(v4, base + (((2 * k + hi) ^ (r & 7)) << 4));
            for (int i = 0; i < 4; ++i) {
                const uint32_t v = v4[i] & (i < 2 ? keep0 : keep1);
                ok &= (v & 0x7F80u) != 0x7F80u && (v & 0x7F800000u) != 0x7F800000u;
            }
        }
        return ok;
    }

    // The second product where a value that is not finite lies among keys that
    // some tokens see and others do not: 0 * inf would reach the rows that do
    // not see it, so each token's rows get a product of their own over the
    // keys that they see.
    __device__ void tokens_apart(const AttnArgs &a, uint32_t base, int r, int hi, int j0, int len,
                                 int row0, int rows, const uint32_t (&p)[NT][2]) {
        const int t = threadIdx.x & 3;
        for (int i = 0; i < a.tokens; ++i) {
            const int last = len - a.tokens + i, lo = a.window > 0 ? last - a.window : -1;
            const auto seen = [&](int k) { return j0 + k <= last && j0 + k > lo; };
            const uint32_t k0 =
                (seen(2 * t) ? 0xFFFFu : 0u) | (seen(2 * t + 1) ? 0xFFFF0000u : 0u);
            const uint32_t k1 =
                (seen(2 * t + 8) ? 0xFFFFu : 0u) | (seen(2 * t + 9) ? 0xFFFF0000u : 0u);
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                uint32_t v4[4];
                ldsm4_t(v4, base + (((2 * k + hi) ^ (r & 7)) << 4));
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    float d[4] = {o[n][k][0], o[n][k][1], o[n][k][2], o[n][k][3]};
                    mma_bf16_16816(d, v4[0] & k0, v4[1] & k0, v4[2] & k1, v4[3] & k1, p[n][0],
                                   p[n][1]);
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const int row = row0 + 8 * n + 2 * t + (c & 1);
                        if (min(row, rows - 1) / a.group == i) o[n][k][c] = d[c];
                    }
                }
            }
        }
    }
};

// The workspace: a counter per block, then the pieces that are joined, two a
// block: float [64][D], then m [64], l [64].
constexpr int kCounterBytes = 4096;
template <typename C>
__device__ __forceinline__ float *slot_of(const AttnArgs &a, int block, int which) {
    return reinterpret_cast<float *>(static_cast<char *>(a.workspace) + kCounterBytes) +
           (size_t)(2 * block + which) * C::SLOT;
}

template <typename C>
__device__ void store_row(const AttnArgs &a, int b, int h, int row, int d, float4 o, float m,
                          float l) {
    const int i = row / a.group, hq = h * a.group + row - i * a.group;
    const long long t = (long long)b * a.tokens + i;
    const float f = l > 0.f ? 1.f / l : l == 0.f ? 0.f : l;    // NaN stays NaN
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

template <typename C>
__global__ void __launch_bounds__(C::THREADS, C::BLOCKS) attn_kernel(const AttnArgs a) {
    extern __shared__ __align__(128) unsigned char smem[];
    using L = typename C::L;
    float *join_o = reinterpret_cast<float *>(smem);
    float *join_m = reinterpret_cast<float *>(smem + C::BUF);
    float *join_l = join_m + C::KG * C::ROWS;
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + C::BUF + C::ML);
    uint64_t *empty = full + C::KG * C::STAGES;
    int *scratch = reinterpret_cast<int *>(empty + C::KG * C::STAGES);    // 64 words

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int kg = warp / C::QG, qg = warp % C::QG;
    if (tid == 0) {
        for (int i = 0; i < C::KG * C::STAGES; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], C::QG);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    begin_after_previous();

    // ---- this block's share of the list (sequence, head, rows, record)
    const int rows = a.tokens * a.group, row_tiles = (rows + C::ROWS - 1) / C::ROWS;
    const int per_seq = a.pool.kv_heads * row_tiles;          // items of a sequence
    const int each = (a.pool.seqs + C::THREADS - 1) / C::THREADS;
    const int b0 = min(tid * each, a.pool.seqs), b1 = min(b0 + each, a.pool.seqs);
    long long mine = 0;
    for (int b = b0; b < b1; ++b) mine += max(sequence(a, b).records, 1);
    long long upto = mine;                                    // inclusive scan
    for (int x = 1; x < 32; x <<= 1) {
        const long long v = __shfl_up_sync(0xFFFFFFFFu, upto, x);
        if (lane >= x) upto += v;
    }
    long long *sums = reinterpret_cast<long long *>(scratch);
    if (lane == 31) sums[warp] = upto;
    __syncthreads();
    long long total = 0;
    for (int w = 0; w < C::W; ++w) {
        if (w < warp) upto += sums[w];
        total += sums[w];
    }
    __syncthreads();
    const long long work = total * per_seq;
    const long long grid_ll = min((long long)gridDim.x, max(1LL, work / C::W));
    const int blocks = (int)grid_ll;
    if (blockIdx.x >= blocks) return;
    const long long begin = work * blockIdx.x / blocks, end = work * (blockIdx.x + 1) / blocks;
    if (begin >= (upto - mine) * per_seq && begin < upto * per_seq) {
        long long at = (upto - mine) * per_seq;
        int b = b0;
        for (;; ++b) {
            const long long n = (long long)max(sequence(a, b).records, 1) * per_seq;
            if (begin < at + n) break;
            at += n;
        }
        scratch[0] = b;
        reinterpret_cast<long long *>(scratch)[1] = begin - at;
    }
    __syncthreads();
    int b = scratch[0];
    long long in_seq = reinterpret_cast<long long *>(scratch)[1];
    __syncthreads();

    Warp<C> w;
    const uint32_t ring = smem_addr(smem) + kg * C::STAGES * L::kBytes;
    unsigned char *ring_ptr = smem + kg * C::STAGES * L::kBytes;
    uint64_t *my_full = full + kg * C::STAGES, *my_empty = empty + kg * C::STAGES;
    uint32_t turn = 0;           // records that this group's ring has taken so far
    bool failed = false;
    long long at = begin;
    while (at < end) {
        const Seq seq = sequence(a, b);
        const int n_seq = max(seq.records, 1);
        const int item = (int)(in_seq / n_seq), u0 = (int)(in_seq - (long long)item * n_seq);
        const int u1 = (int)min((long long)n_seq, u0 + (end - at));
        const int h = item / row_tiles, tile0 = (item - h * row_tiles) * C::ROWS;
        const int row0 = tile0 + qg * 8 * C::NT;
        w.load_q(a, b, h, row0, rows);
        w.clear();
        // records u0 + kg, u0 + kg + KG, ... of this piece
        const int stop = min(u1, seq.records);
        const int n =
            stop > u0 + kg && !failed ? (stop - u0 - kg + C::KG - 1) / C::KG : 0;
        const int32_t *pages = a.pool.table + b * a.pool.stride;
        const auto page_at = [&](int i) {
            if (i >= n) return -1;
            const int page = pages[(seq.first + u0 + kg + i * C::KG) / a.pool.page_records];
            return page >= 0 && page < a.pool.pages ? page : -1;
        };
        int here = page_at(lane), next = page_at(32 + lane);
        int batch = 0;                                        // here holds records 32 batch ..
        const auto page_of = [&](int i) {
            return __shfl_sync(0xFFFFFFFFu, (i >> 5) == batch ? here : next, i & 31);
        };
        // all lanes call; lane 0 of the group's first warp copies
        const auto request = [&](int i, uint32_t as) {
            const int page = page_of(i);
            if (qg == 0 && lane == 0) {
                const int st = as % C::STAGES;
                if (page < 0) {
                    mbar_arrive(&my_full[st]);
                    if (a.pool.error) atomicOr(a.pool.error, W4_KV_ERR_PAGE);
                } else {
                    const int r = seq.first + u0 + kg + i * C::KG;
                    const char *src =
                        a.pool.records +
                        (((long long)page * a.pool.kv_heads + h) * a.pool.page_records +
                         r % a.pool.page_records) * L::kBytes;
                    mbar_expect_tx(&my_full[st], L::kBytes);
                    bulk_g2s(ring_ptr + st * L::kBytes, src, L::kBytes, &my_full[st]);
                }
            }
        };
        if (qg == 0 && lane == 0) fence_proxy_async();
        for (int i = 0; i < min(n, C::STAGES); ++i) request(i, turn + i);
        for (int i = 0; i < n; ++i) {
            if ((i & 31) == 0 && i) {
                here = next;
                batch = i >> 5;
                next = page_at(i + 32 + lane);
            }
            const uint32_t as = turn + i;
            const int st = as % C::STAGES;
            if (!__all_sync(0xFFFFFFFFu, mbar_wait(&my_full[st], (as / C::STAGES) & 1))) {
                // never in normal operation: give up, after a bounded wait for
                // what is still under way
                failed = true;
                if (a.pool.error) atomicOr(a.pool.error, W4_KV_ERR_WAIT);
                for (int x = 1; x < C::STAGES && i + x < n; ++x)
                    mbar_wait(&my_full[(as + x) % C::STAGES], ((as + x) / C::STAGES) & 1);
                break;
            }
            const int j0 = (seq.first + u0 + kg + i * C::KG) * kRecTokens;
            const bool edge = j0 + kRecTokens > seq.len - a.tokens + 1 ||
                              (a.window > 0 && j0 < seq.len - a.window);
            if (page_of(i) >= 0)
                w.record(a, ring + st * L::kBytes, j0, edge, seq.len, row0, rows);
            __syncwarp();
            if constexpr (C::QG == 1) {
                if (i + C::STAGES < n) {
                    if (lane == 0) fence_proxy_async();
                    request(i + C::STAGES, as + C::STAGES);
                }
            } else {
                if (lane == 0) mbar_arrive(&my_empty[st]);
                // refill the stage of the record before: the others are done
                // with it, or soon will be
                if (i > 0 && i - 1 + C::STAGES < n) {
                    const uint32_t prev = as - 1;
                    if (qg == 0) {
                        // (a wait that gives up leaves the stage alone: the
                        // wait for its next record then gives up too)
                        if (!__all_sync(0xFFFFFFFFu, mbar_wait(&my_empty[prev % C::STAGES],
                                                               (prev / C::STAGES) & 1)))
                            continue;
                        if (lane == 0) fence_proxy_async();
                    }
                    request(i - 1 + C::STAGES, prev + C::STAGES);
                }
            }
        }
        turn += n;

        // ---- join the groups of warps through shared memory
        __syncthreads();
        {
            const int g = lane >> 2, t = lane & 3;
#pragma unroll
            for (int x = 0; x < C::NT; ++x) {
                const int r = kg * C::ROWS + qg * 8 * C::NT + 8 * x;
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    float l = w.l[x][c];
                    for (int s = 4; s < 32; s <<= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, s);
                    if (g == 0) join_m[r + 2 * t + c] = w.m[x][c], join_l[r + 2 * t + c] = l;
                }
#pragma unroll
                for (int k = 0; k < C::D / 16; ++k)
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        join_o[(r + 2 * t + (c & 1)) * C::OROW + 16 * k + g + (c & 2) * 4] =
                            w.o[x][k][c];
            }
        }
        __syncthreads();
        const bool whole = u0 == 0 && u1 == n_seq;
        float *slot = slot_of<C>(a, blockIdx.x, u0 == 0 ? 1 : 0);
        for (int e = tid; e < C::ROWS * (C::D / 4); e += C::THREADS) {
            const int r = e / (C::D / 4), d = e % (C::D / 4) * 4;
            if (tile0 + r >= rows) continue;
            float m = join_m[r];
#pragma unroll
            for (int k = 1; k < C::KG; ++k) m = fmaxf(m, join_m[k * C::ROWS + r]);
            float l = 0.f;
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int k = 0; k < C::KG; ++k) {
                const float f = exp2_fast(join_m[k * C::ROWS + r] - m);
                l = fmaf(f, join_l[k * C::ROWS + r], l);
                const float4 v =
                    *reinterpret_cast<const float4 *>(&join_o[(k * C::ROWS + r) * C::OROW + d]);
                o.x = fmaf(f, v.x, o.x), o.y = fmaf(f, v.y, o.y);
                o.z = fmaf(f, v.z, o.z), o.w = fmaf(f, v.w, o.w);
            }
            if (whole) {
                store_row<C>(a, b, h, tile0 + r, d, o, m, l);
            } else {
                *reinterpret_cast<float4 *>(&slot[r * C::D + d]) = o;
                if (d == 0) slot[64 * C::D + r] = m, slot[64 * C::D + 64 + r] = l;
            }
        }
        if (!whole) {
            // the blocks of this item: those whose shares hold its first and last unit
            const long long item0 = at - u0, item1 = item0 + n_seq;
            int c0 = (int)(item0 * blocks / work), c1 = (int)((item1 - 1) * blocks / work);
            while (work * (c0 + 1) / blocks <= item0) ++c0;
            while (work * c0 / blocks > item0) --c0;
            while (work * (c1 + 1) / blocks <= item1 - 1) ++c1;
            while (work * c1 / blocks > item1 - 1) --c1;
            uint32_t *counter = static_cast<uint32_t *>(a.workspace) + c0;
            __threadfence();
            __syncthreads();
            if (tid == 0) scratch[0] = atomicAdd(counter, 1u) == (uint32_t)(c1 - c0);
            __syncthreads();
            if (scratch[0]) {
                __threadfence();
                if (tid == 0) *counter = 0u;
                for (int e = tid; e < C::ROWS * (C::D / 4); e += C::THREADS) {
                    const int r = e / (C::D / 4), d = e % (C::D / 4) * 4;
                    if (tile0 + r >= rows) continue;
                    float m = kNone, l = 0.f;
                    for (int c = c0; c <= c1; ++c)
                        m = fmaxf(m, slot_of<C>(a, c, c == c0)[64 * C::D + r]);
                    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
                    for (int c = c0; c <= c1; ++c) {
                        const float *s = slot_of<C>(a, c, c == c0);
                        const float f = exp2_fast(s[64 * C::D + r] - m);
                        l = fmaf(f, s[64 * C::D + 64 + r], l);
                        const float4 v = *reinterpret_cast<const float4 *>(&s[r * C::D + d]);
                        o.x = fmaf(f, v.x, o.x), o.y = fmaf(f, v.y, o.y);
                        o.z = fmaf(f, v.z, o.z), o.w = fmaf(f, v.w, o.w);
                    }
                    store_row<C>(a, b, h, tile0 + r, d, o, m, l);
                }
            }
        }
        __syncthreads();                                      // the ring's memory is free again
        at += u1 - u0;
        in_seq += u1 - u0;
        if (in_seq == (long long)n_seq * per_seq) in_seq = 0, ++b;
    }
}

template <typename C>
cudaError_t launch_cfg(const AttnArgs &a, int num_sms, cudaStream_t stream) {
    if (num_sms * C::BLOCKS > kCounterBytes / 4) return cudaErrorInvalidConfiguration;
    static std::atomic<bool> ready[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64 || !ready[dev].load(std::memory_order_relaxed)) {
        e = cudaFuncSetAttribute(attn_kernel<C>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) ready[dev].store(true, std::memory_order_relaxed);
    }
    return launch_overlapped(attn_kernel<C>, dim3(num_sms * C::BLOCKS), dim3(C::THREADS), C::SMEM, stream,
                             a);
}

// Rows a block takes, and how: up to 8 in one tile a warp; more in two, with
// 1, 2 or 4 warps side by side on a record.
template <int FMT, int D, int STAGES1, int W1, int STAGES2>
cudaError_t launch_rows(const AttnArgs &a, int num_sms, cudaStream_t stream) {
    const int rows = a.tokens * a.group;
    if (rows <= 8) return launch_cfg<Cfg<FMT, D, 1, 1, W1, STAGES1, 2>>(a, num_sms, stream);
    if (rows <= 16) return launch_cfg<Cfg<FMT, D, 2, 1, 8, STAGES2, 1>>(a, num_sms, stream);
    if (rows <= 32)
        return launch_cfg<Cfg<FMT, D, 2, 2, 8, 2 * STAGES2, 1>>(a, num_sms, stream);
    return launch_cfg<Cfg<FMT, D, 2, 4, 8, 4 * STAGES2, 1>>(a, num_sms, stream);
}

}  // namespace

// Counters of the blocks, then two joined pieces of 64 rows a block.
size_t attn_workspace_bytes(int head_dim, int num_sms) {
    return kCounterBytes + (size_t)num_sms * 2 * 2 * 64 * (head_dim + 2) * 4;
}

cudaError_t launch_paged_attn(const AttnArgs &a, int format, int head_dim, int num_sms,
                              cudaStream_t stream) {
    if (head_dim == 128)
        return format == W4_KV_BF16 ? launch_rows<W4_KV_BF16, 128, 3, 4, 3>(a, num_sms, stream)
               : format == W4_KV_INT8
                   ? launch_rows<W4_KV_INT8, 128, 3, 8, 5>(a, num_sms, stream)
                   : launch_rows<W4_KV_INT4, 128, 5, 8, 8>(a, num_sms, stream);
    return format == W4_KV_BF16 ? launch_rows<W4_KV_BF16, 64, 3, 8, 5>(a, num_sms, stream)
           : format == W4_KV_INT8
               ? launch_rows<W4_KV_INT8, 64, 5, 8, 8>(a, num_sms, stream)
               : launch_rows<W4_KV_INT4, 64, 8, 8, 8>(a, num_sms, stream);
}

}  // namespace w4
