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
// Schedule.  The blocks, one per SM, divide the records among themselves from
// the lengths on the device.  With at most half as many heads (sequence x
// key/value head) as blocks, every head is cut into equal parts, as many as
// fit the grid, and a block takes one.  With more heads, block c takes records
// [c W / G, (c + 1) W / G) of the list (sequence, head, record): its stretch
// may cover several heads, the first and the last of them in part.  The parts
// of a head are joined by the block that finishes it last, in block order.
// In a block the warps form KG groups of QG: a group takes every KG-th record
// through its own ring of bulk copies (one record is one copy), and its QG
// warps hold 8 rows each.
#include <atomic>

#include "w4_device.cuh"
#include "w4_kv.cuh"

namespace w4 {
namespace {

constexpr int kAttnWarps = 16, kAttnThreads = 32 * kAttnWarps;
constexpr int kRowsMax = 64;           // rows of a block: 8 a warp, up to 8 warps a group
constexpr int kRingBytes = 196608;     // shared by the groups; the join uses it in between
constexpr int kMaxStages = 32;         // of one group's ring
constexpr int kMaxGrid = 256;
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

// A warp's tile of 8 rows: its share of Q, and the running m, l, O.
template <int FMT, int D>
struct Tile {
    using L = KvLayout<FMT, D>;
    static constexpr int KS = D / 16;                     // k-steps of S, m-tiles of O
    static constexpr float kBias = FMT == W4_KV_BF16 ? 0.f : 6.f;
    static constexpr float kSlack = FMT == W4_KV_BF16 ? 8.f : 14.f;

    uint32_t qf[KS][2];          // Q as the column operand
    float o[KS][4];
    float m[2], l[2];            // columns 2t, 2t + 1
    float sc[2];                 // score factor of a column

    // Which value of the head goes with half e of register i of k-step ks.
    __device__ static int q_index(int ks, int i, int e, int t) {
        if (FMT == W4_KV_BF16) return 16 * ks + 8 * i + 2 * t + e;
        if (FMT == W4_KV_INT8) return 64 * (ks >> 2) + 16 * t + 4 * (ks & 3) + i + 2 * e;
        return (D / 4) * t + 8 * (ks >> 1) + 2 * (ks & 1) + i + 4 * e;
    }

    // row0: first row of the warp's tile; rows: rows that there are.
    __device__ void load_q(const AttnArgs &a, int b, int h, int row0, int rows) {
        const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3, r = row0 + g;
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
                    qf[ks][j] =
                        there ? *reinterpret_cast<const uint32_t *>(q + q_index(ks, j, 0, t)) : 0u;
            sc[0] = sc[1] = a.scale * kLog2e;
        } else {
            // a lane's values lie in runs of RUN
            constexpr int RUN = FMT == W4_KV_INT8 ? 16 : D / 4, NRUN = D / 4 / RUN;
            uint4 raw[NRUN * RUN / 8];
#pragma unroll
            for (int x = 0; x < NRUN * RUN / 8; ++x)
                raw[x] = there ? *reinterpret_cast<const uint4 *>(
                                     q + (x / (RUN / 8)) * 64 + RUN * t + (x % (RUN / 8)) * 8)
                               : make_uint4(0u, 0u, 0u, 0u);
            const auto value = [&](int ks, int j, int e) {
                const int d = q_index(ks, j, e, 0);       // of lane t = 0
                const int at = (d / 64) * (FMT == W4_KV_INT8 ? RUN : 0) + d % 64;
                const uint4 v = raw[at / 8];
                const uint32_t w = at % 8 < 2 ? v.x : at % 8 < 4 ? v.y : at % 8 < 6 ? v.z : v.w;
                return __uint_as_float(at & 1 ? w & 0xFFFF0000u : w << 16);
            };
            float top = 0.f;
#pragma unroll
            for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    top = fmaxf(top, fmaxf(fabsf(value(ks, j, 0)), fabsf(value(ks, j, 1))));
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
                    qf[ks][j] = pack_half(value(ks, j, 0) * up, value(ks, j, 1) * up);
            const float f = a.scale * kLog2e * __int_as_float((127 - e) << 23);
#pragma unroll
            for (int c = 0; c < 2; ++c) sc[c] = __shfl_sync(0xFFFFFFFFu, f, 4 * (2 * t + c));
        }
    }

    __device__ void clear() {
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
            for (int c = 0; c < 4; ++c) o[k][c] = 0.f;
#pragma unroll
        for (int c = 0; c < 2; ++c) m[c] = kNone, l[c] = 0.f;
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
        float s[4];
#pragma unroll
            for (int c = 0; c < 4; ++c)
                s[c] = 0.f;
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
                    mma_bf16_16816(s, k4[0], k4[1], k4[2], k4[3], qf[ks][0], qf[ks][1]);
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
                        mma_f16_16816(s, a0, a1, a2, a3, qf[4 * i + w][0],
                                      qf[4 * i + w][1]);
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
                    mma_f16_16816(s, a0, a1, a2, a3, qf[ks][0], qf[ks][1]);
            }
        }
        // ---- scores in units of log2; quantised: with log2 s_v added
        float inv[2] = {1.f, 1.f};                        // 1 / s_v of keys g, g + 8
        if constexpr (FMT == W4_KV_BF16) {
#pragma unroll
                for (int c = 0; c < 4; ++c) s[c] *= sc[c & 1];
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
                    for (int c = 0; c < 2; ++c)
                        s[2 * r + c] = fmaf(s[2 * r + c], sk * sc[c], lv);
            }
        }
        uint32_t keep0 = 0xFFFFFFFFu, keep1 = 0xFFFFFFFFu;    // keys 2t, 2t+1; 2t+8, 2t+9
        bool apart = false;       // a key that some rows see and some do not
        if (edge) {
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const int row = row0 + 2 * t + (c & 1), j = j0 + g + (c & 2) * 4;
                    const int last = len - a.tokens + min(row, rows - 1) / a.group;
                    if (j > last || (a.window > 0 && j <= last - a.window)) s[c] = -INFINITY;
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
            for (int c = 0; c < 4; ++c) over |= s[c] > m[c & 1] + kSlack;
        if (__any_sync(0xFFFFFFFFu, over)) {
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    float top = fmaxf(s[c], s[c + 2]);
#pragma unroll
                    for (int x = 4; x < 32; x <<= 1)
                        top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, x));
                    const float now = fmaxf(m[c], top - kBias);
                    const float f = exp2_fast(m[c] - now);
                    m[c] = now;
                    l[c] *= f;
#pragma unroll
                    for (int k = 0; k < KS; ++k) {
                        o[k][c] *= f;
                        o[k][c + 2] *= f;
                    }
                }
        }
        // ---- probabilities, their sums, and P^T as the column operand
        uint32_t p[2];
        {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                s[c] = exp2_fast(s[c] - m[c & 1]);
                l[c & 1] = fmaf(s[c], inv[c >> 1], l[c & 1]);
            }
#pragma unroll
            for (int r = 0; r < 2; ++r)
                p[r] = transposed(FMT == W4_KV_BF16 ? pack_bf16(s[2 * r], s[2 * r + 1])
                                                       : pack_half(s[2 * r], s[2 * r + 1]));
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
                    mma_bf16_16816(o[k], v4[0], v4[1], v4[2], v4[3], p[0], p[1]);
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
                            mma_f16_16816(o[2 * i + x], a0, a1, a2, a3, p[0], p[1]);
                    }
                } else {
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const uint32_t u = w[x], v = w[x] >> 8;
                        const uint32_t a0 = low(u, zlo[0]), a1 = high(u, zhi[0]);
                        const uint32_t a2 = low(v, zlo[1]), a3 = high(v, zhi[1]);
                            mma_f16_16816(o[4 * i + x], a0, a1, a2, a3, p[0], p[1]);
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
                                 int row0, int rows, const uint32_t (&p)[2]) {
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
                {
                    float d[4] = {o[k][0], o[k][1], o[k][2], o[k][3]};
                    mma_bf16_16816(d, v4[0] & k0, v4[1] & k0, v4[2] & k1, v4[3] & k1, p[0],
                                   p[1]);
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const int row = row0 + 2 * t + (c & 1);
                        if (min(row, rows - 1) / a.group == i) o[k][c] = d[c];
                    }
                }
            }
        }
    }
};

// The workspace: a counter per block, then the pieces that are joined, two a
// block: float [64][D], then m [64], l [64].
constexpr int kCounterBytes = 4 * kMaxGrid;
template <int D>
__device__ __forceinline__ float *slot_of(const AttnArgs &a, int block, bool starts) {
    return reinterpret_cast<float *>(static_cast<char *>(a.workspace) + kCounterBytes) +
           (size_t)(2 * block + (starts ? 1 : 0)) * kRowsMax * (D + 2);
}

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

__device__ __forceinline__ void add_scaled(float4 &o, float f, const float4 &v) {
    o.x = fmaf(f, v.x, o.x), o.y = fmaf(f, v.y, o.y);
    o.z = fmaf(f, v.z, o.z), o.w = fmaf(f, v.w, o.w);
}

// A block's stretch of the list.
struct Share {
    int b;                 // sequence of the first piece
    int item;              // head (x row tile) of the first piece in it
    int u0;                // first record of that
    long long units;       // records to go (over all pieces)
    int parts;             // parts of every head, or 0: the stretch may cover several heads
    int part;              // which of them this is
    long long work;        // all records of the list
    long long at;          // the stretch's start in the list
    int blocks;            // blocks that have a stretch
};

// Every warp works it out for itself, without a barrier.  false: nothing to do.
__device__ bool share_of(const AttnArgs &a, int row_tiles, int least, Share *s) {
    const int lane = threadIdx.x & 31, per_seq = a.pool.kv_heads * row_tiles;
    const int each = (a.pool.seqs + 31) / 32;
    const int b0 = min(lane * each, a.pool.seqs), b1 = min(b0 + each, a.pool.seqs);
    const int grid = (int)gridDim.x;
    long long mine = 0;
    int longest = 0;
#pragma unroll 4
    for (int b = b0; b < b1; ++b) {
        const int n = max(sequence(a, b).records, 1);
        mine += n;
        longest = max(longest, n);
    }
    long long upto = mine;                                    // inclusive scan
#pragma unroll
    for (int x = 1; x < 32; x <<= 1) {
        const long long v = __shfl_up_sync(0xFFFFFFFFu, upto, x);
        if (lane >= x) upto += v;
    }
    s->work = __shfl_sync(0xFFFFFFFFu, upto, 31) * per_seq;
    if ((long long)a.pool.seqs * per_seq * 2 <= grid) {
        // parts of at most `size` records, the smallest that fit the grid
        longest = __reduce_max_sync(0xFFFFFFFFu, longest);
        int size = max(least, (int)((s->work + grid - 1) / grid));
        int cuts, before;
        while (true) {
            cuts = 0;
            for (int b = b0; b < b1; ++b)
                cuts += (max(sequence(a, b).records, 1) + size - 1) / size;
            before = cuts;
#pragma unroll
            for (int x = 1; x < 32; x <<= 1) {
                const int v = __shfl_up_sync(0xFFFFFFFFu, before, x);
                if (lane >= x) before += v;
            }
            if (__shfl_sync(0xFFFFFFFFu, before, 31) * per_seq <= grid || size >= longest) break;
            size += max(1, size / 8);
        }
        const int c = blockIdx.x;
        before = (before - cuts) * per_seq;                   // parts before this lane's
        const bool here = c >= before && c < before + cuts * per_seq;
        int b = b0, parts = 1, n = 1;
        if (here)
            for (;; ++b) {
                n = max(sequence(a, b).records, 1);
                parts = (n + size - 1) / size;
                if (c < before + parts * per_seq) break;
                before += parts * per_seq;
            }
        const unsigned found = __ballot_sync(0xFFFFFFFFu, here);
        if (!found) return false;
        const int src = __ffs(found) - 1;
        s->b = __shfl_sync(0xFFFFFFFFu, b, src);
        s->parts = __shfl_sync(0xFFFFFFFFu, parts, src);
        n = __shfl_sync(0xFFFFFFFFu, n, src);
        const int in = c - __shfl_sync(0xFFFFFFFFu, before, src);
        s->item = in / s->parts;
        s->part = in - s->item * s->parts;
        s->u0 = (int)((long long)n * s->part / s->parts);
        s->units = (long long)n * (s->part + 1) / s->parts - s->u0;
        s->at = 0;
        s->blocks = grid;
        return true;
    }
    s->parts = s->part = 0;
    s->blocks = (int)min((long long)grid, s->work);
    if ((int)blockIdx.x >= s->blocks) return false;
    s->at = s->work * blockIdx.x / s->blocks;
    s->units = s->work * (blockIdx.x + 1) / s->blocks - s->at;
    long long before = (upto - mine) * per_seq;
    const bool here = s->at >= before && s->at < upto * per_seq;
    int b = b0, n = 1;
    if (here)
        for (;; ++b) {
            n = max(sequence(a, b).records, 1);
            if (s->at < before + (long long)n * per_seq) break;
            before += (long long)n * per_seq;
        }
    const int src = __ffs(__ballot_sync(0xFFFFFFFFu, here)) - 1;
    s->b = __shfl_sync(0xFFFFFFFFu, b, src);
    n = __shfl_sync(0xFFFFFFFFu, n, src);
    const long long in = s->at - __shfl_sync(0xFFFFFFFFu, before, src);
    s->item = (int)(in / n);
    s->u0 = (int)(in - (long long)s->item * n);
    return true;
}

// The block that finished a head last joins its n pieces, those of blocks c0 ..
// c0 + n - 1, in that order.  buf: the ring's shared memory.
template <int D>
__device__ void join_pieces(const AttnArgs &a, int c0, int n, int b, int h, int tile0, int rows,
                            int block_rows, float *buf) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int there = min(block_rows, rows - tile0);
    float *fac = buf, *mx = buf + n * kRowsMax, *sum = mx + kRowsMax, *half = sum + kRowsMax;
    for (int r = warp; r < there; r += kAttnWarps) {          // a warp per row: factors
        float m = kNone;
        for (int c = lane; c < n; c += 32)
            m = fmaxf(m, __ldcg(&slot_of<D>(a, c0 + c, c == 0)[kRowsMax * D + r]));
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, x));
        float l = 0.f;
        for (int c = lane; c < n; c += 32) {
            const float *s = slot_of<D>(a, c0 + c, c == 0);
            const float f = exp2_fast(__ldcg(&s[kRowsMax * D + r]) - m);
            fac[c * kRowsMax + r] = f;
            l = fmaf(f, __ldcg(&s[kRowsMax * D + kRowsMax + r]), l);
        }
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, x);
        if (lane == 0) mx[r] = m, sum[r] = l;
    }
    __syncthreads();
    // two threads per 4 values take every other piece
    const int values = there * (D / 4);
    for (int e0 = 0; e0 < values; e0 += kAttnThreads / 2) {
        const int e = e0 + (tid & (kAttnThreads / 2 - 1)), side = tid / (kAttnThreads / 2);
        const int r = e / (D / 4), d = e % (D / 4) * 4;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        if (e < values) {
#pragma unroll 8
            for (int c = side; c < n; c += 2)
                add_scaled(o, fac[c * kRowsMax + r],
                           __ldcg(reinterpret_cast<const float4 *>(
                               &slot_of<D>(a, c0 + c, c == 0)[r * D + d])));
        }
        float4 *other = reinterpret_cast<float4 *>(half) + (tid & (kAttnThreads / 2 - 1));
        if (side) *other = o;
        __syncthreads();
        if (!side && e < values) {
            add_scaled(o, 1.f, *other);
            store_row(a, b, h, tile0 + r, d, o, mx[r], sum[r]);
        }
        __syncthreads();
    }
}

template <int FMT, int D>
__global__ void __launch_bounds__(kAttnThreads, 1)
attn_kernel(const AttnArgs a, const int row_tiles, const int QG, const int KG, const int stages) {
    extern __shared__ __align__(128) unsigned char smem[];
    using L = KvLayout<FMT, D>;
    constexpr int OROW = D + 4;                               // floats; + 4: no bank conflicts
    __shared__ uint64_t full[kAttnWarps * kMaxStages], empty[kAttnWarps * kMaxStages];
    __shared__ float join_m[kAttnWarps * 8], join_l[kAttnWarps * 8];
    __shared__ int is_last;
    float *join_o = reinterpret_cast<float *>(smem);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int kg = warp / QG, qg = warp - kg * QG;
    const bool works = kg < KG;                               // QG may not divide 16
    const int block_rows = 8 * QG;
    for (int i = tid; i < KG * stages; i += kAttnThreads) {
        mbar_init(&full[i], 1);
        mbar_init(&empty[i], QG);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    __syncthreads();
    begin_after_previous();

    Share share;
    if (!share_of(a, row_tiles, 4 * KG, &share)) return;
    const int rows = a.tokens * a.group, per_seq = a.pool.kv_heads * row_tiles;
    const uint32_t ring = smem_addr(smem) + kg * stages * L::kBytes;
    unsigned char *ring_ptr = smem + kg * stages * L::kBytes;
    uint64_t *my_full = full + kg * stages, *my_empty = empty + kg * stages;
    int get = 0, put = 0;                                     // stages next taken and filled
    uint32_t get_phase = 0;
    bool failed = false;
    Tile<FMT, D> w;
    int b = share.b, item = share.item, u0 = share.u0;
    long long at = share.at;
    while (share.units > 0) {
        const Seq seq = sequence(a, b);
        const int n_seq = max(seq.records, 1);
        const int u1 = (int)min((long long)n_seq, u0 + share.units);
        const int h = item / row_tiles, tile0 = (item - h * row_tiles) * block_rows;
        const int row0 = tile0 + qg * 8;
        // records u0 + kg, u0 + kg + KG, ... of this piece
        const int stop = min(u1, seq.records);
        const int n = works && stop > u0 + kg && !failed ? (stop - u0 - kg + KG - 1) / KG : 0;
        const int rec0 = seq.first + u0 + kg;
        const int32_t *pages = a.pool.table + b * a.pool.stride;
        const auto page_at = [&](int i) {
            if (i >= n) return -1;
            const int page = pages[(rec0 + i * KG) / a.pool.page_records];
            return page >= 0 && page < a.pool.pages ? page : -1;
        };
        int here = page_at(lane), next = page_at(32 + lane);
        int batch = 0;                                        // here holds records 32 batch ..
        const auto page_of = [&](int i) {
            return __shfl_sync(0xFFFFFFFFu, (i >> 5) == batch ? here : next, i & 31);
        };
        // all lanes call; lane 0 of the group's first warp copies record i
        const auto request = [&](int i) {
            const int page = page_of(i);
            if (qg == 0 && lane == 0) {
                if (page < 0) {
                    mbar_arrive(&my_full[put]);
                    if (a.pool.error) atomicOr(a.pool.error, W4_KV_ERR_PAGE);
                } else {
                    const int r = rec0 + i * KG;
                    const char *src =
                        a.pool.records +
                        (((long long)page * a.pool.kv_heads + h) * a.pool.page_records +
                         r % a.pool.page_records) * L::kBytes;
                    mbar_expect_tx(&my_full[put], L::kBytes);
                    bulk_g2s(ring_ptr + put * L::kBytes, src, L::kBytes, &my_full[put]);
                }
            }
            if (++put == stages) put = 0;
        };
        if (qg == 0 && lane == 0) fence_proxy_async();
        for (int i = 0; i < min(n, stages); ++i) request(i);
        if (works) w.load_q(a, b, h, row0, rows);
        w.clear();
        int prev = 0;
        uint32_t prev_phase = 0;
        for (int i = 0; i < n; ++i) {
            if ((i & 31) == 0 && i) {
                here = next;
                batch = i >> 5;
                next = page_at(i + 32 + lane);
            }
            if (!__all_sync(0xFFFFFFFFu, mbar_wait(&my_full[get], get_phase))) {
                // never in normal operation: give up, after a bounded wait for
                // what is still under way
                failed = true;
                if (a.pool.error) atomicOr(a.pool.error, W4_KV_ERR_WAIT);
                for (int x = 1; x < stages && i + x < n; ++x) {
                    if (++get == stages) get = 0, get_phase ^= 1;
                    mbar_wait(&my_full[get], get_phase);
                }
                break;
            }
            const int j0 = (rec0 + i * KG) * kRecTokens;
            const bool edge = j0 + kRecTokens > seq.len - a.tokens + 1 ||
                              (a.window > 0 && j0 < seq.len - a.window);
            if (page_of(i) >= 0)
                w.record(a, ring + get * L::kBytes, j0, edge, seq.len, row0, rows);
            __syncwarp();
            if (QG == 1) {
                if (i + stages < n) {
                    if (lane == 0) fence_proxy_async();
                    request(i + stages);
                }
            } else {
                if (lane == 0) mbar_arrive(&my_empty[get]);
                // refill the stage of the record before: the others are done
                // with it, or soon will be
                if (i > 0 && i - 1 + stages < n) {
                    // (a wait that gives up leaves the stage alone: the wait
                    // for its next record then gives up too)
                    if (qg != 0 ||
                        __all_sync(0xFFFFFFFFu, mbar_wait(&my_empty[prev], prev_phase))) {
                        if (qg == 0 && lane == 0) fence_proxy_async();
                        request(i - 1 + stages);
                    }
                }
            }
            prev = get, prev_phase = get_phase;
            if (++get == stages) get = 0, get_phase ^= 1;
        }

        // ---- join the groups of warps through shared memory
        __syncthreads();
        if (works) {
            const int g = lane >> 2, t = lane & 3, r = kg * block_rows + qg * 8 + 2 * t;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                float l = w.l[c];
#pragma unroll
                for (int s = 4; s < 32; s <<= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, s);
                if (g == 0) join_m[r + c] = w.m[c], join_l[r + c] = l;
            }
#pragma unroll
            for (int k = 0; k < D / 16; ++k)
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    join_o[(r + (c & 1)) * OROW + 16 * k + g + (c & 2) * 4] = w.o[k][c];
        }
        __syncthreads();
        const bool whole = u0 == 0 && u1 == n_seq;
        float *slot = slot_of<D>(a, blockIdx.x, u0 == 0);
        for (int e = tid; e < block_rows * (D / 4); e += kAttnThreads) {
            const int r = e / (D / 4), d = e % (D / 4) * 4;
            if (tile0 + r >= rows) continue;
            float m = join_m[r];
            for (int k = 1; k < KG; ++k) m = fmaxf(m, join_m[k * block_rows + r]);
            float l = 0.f;
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
            for (int k = 0; k < KG; ++k) {
                const int at = k * block_rows + r;
                const float f = exp2_fast(join_m[at] - m);
                l = fmaf(f, join_l[at], l);
                add_scaled(o, f, *reinterpret_cast<const float4 *>(&join_o[at * OROW + d]));
            }
            if (whole) {
                store_row(a, b, h, tile0 + r, d, o, m, l);
            } else {
                *reinterpret_cast<float4 *>(&slot[r * D + d]) = o;
                if (d == 0) slot[kRowsMax * D + r] = m, slot[kRowsMax * D + kRowsMax + r] = l;
            }
        }
        if (!whole) {
            int c0, pieces;
            if (share.parts) {
                c0 = blockIdx.x - share.part;
                pieces = share.parts;
            } else {
                // the blocks whose stretches hold the head's first and last record
                const long long first = at - u0, last = first + n_seq - 1;
                const auto owner = [&](long long u) {
                    int c = (int)(u * share.blocks / share.work);
                    while (share.work * (c + 1) / share.blocks <= u) ++c;
                    while (share.work * c / share.blocks > u) --c;
                    return c;
                };
                c0 = owner(first);
                pieces = owner(last) - c0 + 1;
            }
            uint32_t *counter = static_cast<uint32_t *>(a.workspace) + c0;
            __threadfence();
            __syncthreads();
            if (tid == 0) is_last = atomicAdd(counter, 1u) == (uint32_t)(pieces - 1);
            __syncthreads();
            if (is_last) {
                __threadfence();
                if (tid == 0) *counter = 0u;
                join_pieces<D>(a, c0, pieces, b, h, tile0, rows, block_rows, join_o);
            }
        }
        __syncthreads();                                      // the ring's memory is free again
        at += u1 - u0;
        share.units -= u1 - u0;
        u0 = 0;
        if (u1 == n_seq && ++item == per_seq) item = 0, ++b;
    }
}

template <int FMT, int D>
cudaError_t launch(const AttnArgs &a, int num_sms, cudaStream_t stream) {
    constexpr int bytes = KvLayout<FMT, D>::kBytes;
    static std::atomic<bool> ready[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64 || !ready[dev].load(std::memory_order_relaxed)) {
        e = cudaFuncSetAttribute(attn_kernel<FMT, D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 kRingBytes);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) ready[dev].store(true, std::memory_order_relaxed);
    }
    const int tiles = (a.tokens * a.group + 7) / 8, row_tiles = (tiles + 7) / 8;
    const int QG = (tiles + row_tiles - 1) / row_tiles;
    // groups of at least three stages (64-KB rings of bf16 records: 8 groups)
    const int most = kRingBytes / (3 * bytes);
    const int KG = kAttnWarps / QG < most ? kAttnWarps / QG : most;
    int stages = kRingBytes / (KG * bytes);
    if (stages > kMaxStages) stages = kMaxStages;
    const int grid = num_sms < kMaxGrid ? num_sms : kMaxGrid;
    return launch_overlapped(attn_kernel<FMT, D>, dim3(grid), dim3(kAttnThreads), kRingBytes,
                             stream, a, row_tiles, QG, KG, stages);
}

}  // namespace

size_t attn_workspace_bytes(int head_dim, int num_sms) {
    const int grid = num_sms < kMaxGrid ? num_sms : kMaxGrid;
    return kCounterBytes + (size_t)grid * 2 * kRowsMax * (head_dim + 2) * 4;
}

cudaError_t launch_paged_attn(const AttnArgs &a, int format, int head_dim, int num_sms,
                              cudaStream_t stream) {
    if (head_dim == 128)
        return format == W4_KV_BF16   ? launch<W4_KV_BF16, 128>(a, num_sms, stream)
               : format == W4_KV_INT8 ? launch<W4_KV_INT8, 128>(a, num_sms, stream)
                                      : launch<W4_KV_INT4, 128>(a, num_sms, stream);
    return format == W4_KV_BF16   ? launch<W4_KV_BF16, 64>(a, num_sms, stream)
           : format == W4_KV_INT8 ? launch<W4_KV_INT8, 64>(a, num_sms, stream)
                                  : launch<W4_KV_INT4, 64>(a, num_sms, stream);
}

}  // namespace w4
