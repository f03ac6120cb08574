// What every cached token gets of the new tokens' attention (w4_attn_weights).
//
// With the attention's log-sum-exp known, a token's weight is
//   w_j = sum over the rows that see j of exp2(y_j - lse log2 e),
// y the scores in units of log2, so the keys are read once more, the values not at
// all, and no token needs another one's result: nothing is joined.
//
// Roundings.  Operands are those of the attention (bf16, or exact codes against binary16
// queries), scores, exponents and sums fp32; exp2 is off by 2^-22, and what it gives
// under 2^-126 is 0.  No probability is rounded to fewer bits.
//
// The blocks divide the list (sequence, head, record) evenly, from the lengths on
// the device.  A warp takes every fourth unit of 1 to 4 records of its block's
// stretch through a ring of its own, which asynchronous copies of 16 bytes fill
// across the heads' borders, with the records' keys and what their tokens had
// before; a record's lanes find its page.  One tile of 8 rows of queries stays in
// registers, more of them are shared by the block's warps.
//
// Measured (28 query and 4 key/value heads of 128, one new token, captured calls):
// 32 x 16384 tokens in bf16 86.8 us, 95 % of a copy's rate for keys and weights; 64
// ragged sequences of up to 8192 in 8 bits 28.3 us (78 %), where the instructions
// around 2 KB of codes count; in 4 bits 32 x 16384 39.5 us (61 %): conversion and
// products, 230 instructions a record and warp.  Four blocks of four warps and rings of
// two stages; two blocks of eight 29.9, 88.4 and 38.8 us; three stages 31.5, 91.9 and
// 39.5; three blocks of eight at 80 registers 42.3, 88.8 and 56.5 (spills); units of
// half the size 34.8 and 45.0 in 8 and 4 bits.
#include <atomic>

#include "w4_attn_query.cuh"
#include "w4_kv_work.cuh"

namespace w4 {
namespace {

constexpr int kTilesMax = 8;             // tiles of 8 rows that a launch takes
constexpr int kWeightWarps = 4;          // of a block
constexpr int kWeightBlocks = 4;         // an SM
constexpr int kWeightStages = 2;         // of a warp's ring

struct Weights {
    const float *before;                 // NULL: none
    float *after;
    float decay;
    int columns;
    int row0;                            // first row of this launch; from the second
                                         // on it adds to what the one before left
};

// Operands of one tile of rows in shared memory, by lane.
template <int D>
struct SharedTile {
    uint4 q[D / 32][32];                 // two k-steps each
    float4 factors[32];                  // sc, qs of columns 2t, 2t + 1
    float2 minus[32];                    // their lse in units of log2; infinite: no row
};

// A unit is RECS neighbouring records, 4 KB of keys where D is 128: what a warp does
// at a time.
template <int FMT, int D>
struct Stage {
    using L = KvLayout<FMT, D>;
    static constexpr int kRecs = L::kPart >= 4096 ? 1 : L::kPart >= 2048 ? 2 : 4;
    static constexpr int kTokens = kRecs * kRecTokens;
    // of a stage of a warp's ring: keys, their descriptors, weights before
    static constexpr int kMetaAt = kRecs * L::kPart, kBeforeAt = kMetaAt + 64 * kRecs,
                         kBytes = kBeforeAt + 4 * kTokens;
};

// Units of a sequence.
template <int TOKENS>
struct Units {
    const AttnArgs &a;

    __device__ __forceinline__ int len(int b) const {
        return cached_len(a.pool, a.lens, b, a.most);
    }
    __device__ __forceinline__ int operator()(int b) const {
        return (len(b) + TOKENS - 1) / TOKENS;
    }
};

__device__ __forceinline__ void copy16(uint32_t to, const void *from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
// 4 bytes, or zeros.
__device__ __forceinline__ void copy4(uint32_t to, const void *from, bool there) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(to), "l"(from),
                 "r"(there ? 4 : 0)
                 : "memory");
}
__device__ __forceinline__ void copies_end() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int LEFT>
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory");
}

// 2 R sums over the lanes of a quad, each of which ends up with the ones that it
// stores: of records of a unit tokens g + 8 r.  R = 4: lane t's of record t; 2: of
// record t / 2 the token r = t % 2; 1: token r = t / 2.
template <int R>
__device__ __forceinline__ void quad_sums(float (&v)[R][2], float (&out)[2]) {
    const int t = threadIdx.x & 3;
    const auto both = [](float keep, float give, int lane) {
        return keep + __shfl_xor_sync(0xFFFFFFFFu, give, lane);
    };
    if constexpr (R == 4) {
        float w[2][2];
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int r = 0; r < 2; ++r)
                w[x][r] = both(t < 2 ? v[x][r] : v[x + 2][r], t < 2 ? v[x + 2][r] : v[x][r], 2);
#pragma unroll
        for (int r = 0; r < 2; ++r)
            out[r] = both(t & 1 ? w[1][r] : w[0][r], t & 1 ? w[0][r] : w[1][r], 1);
    } else if constexpr (R == 2) {
        float w[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) w[r] = both(t < 2 ? v[0][r] : v[1][r], t < 2 ? v[1][r] : v[0][r], 2);
        out[0] = both(t & 1 ? w[1] : w[0], t & 1 ? w[0] : w[1], 1);
    } else {
        const float w = both(t < 2 ? v[0][0] : v[0][1], t < 2 ? v[0][1] : v[0][0], 2);
        out[0] = both(w, w, 1);
    }
}

// ONE: one tile of rows, whose operands stay in registers.
template <int FMT, int D, bool ONE>
__global__ void __launch_bounds__(32 * kWeightWarps, kWeightBlocks)
weights_kernel(const AttnArgs a, const Weights out, int n_tiles) {
    using L = KvLayout<FMT, D>;
    using S = Stage<FMT, D>;
    constexpr int KS = D / 16, R = S::kRecs, LANES = 32 / R, WARPS = kWeightWarps;
    extern __shared__ __align__(128) unsigned char smem[];
    SharedTile<D> *tiles = reinterpret_cast<SharedTile<D> *>(smem);
    begin_after_previous();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const uint32_t ring = smem_addr(smem) + n_tiles * (int)sizeof(SharedTile<D>) +
                          warp * kWeightStages * S::kBytes;
    const int rows = a.tokens * a.group, heads = a.pool.kv_heads;
    const Units<S::kTokens> units = {a};
    Share s(units, a.pool.seqs, heads, blockIdx.x, gridDim.x);
    if (s.left == 0) return;

    // ---- the warp's copies, ahead of its products: unit `ahead` is the next.  A
    // record's LANES lanes find its page and copy its keys.
    Share ahead = s;
    ahead.next(units, heads, warp);
    // records that are there: bit x * LANES of stage 0, the others' shifted by theirs
    constexpr unsigned FIRST = R == 4 ? 0x01010101u : R == 2 ? 0x00010001u : 1u;
    unsigned valid = 0;
    int page = -1, ahead_len = 0, seen_b = -1;
    bool wanted = false;
    const int part = lane % LANES, own = lane / LANES;
    const auto look = [&]() {                                 // the page of the next record
        if (ahead.left <= 0) return;
        if (ahead.b != seen_b) seen_b = ahead.b, ahead_len = units.len(ahead.b);
        const int r = R * ahead.u + own;
        // (no row sees a key before the window of the first one)
        const int upto = kRecTokens * (r + 1);
        wanted = upto - kRecTokens < ahead_len &&
                 (a.window == 0 || upto > ahead_len - a.tokens - a.window + 1);
        if (wanted) page = a.pool.table[ahead.b * a.pool.stride + page_slot(a.pool, r)];
    };
    const auto fetch = [&](int put) {
        if (ahead.left > 0) {
            const uint32_t to = ring + put * S::kBytes;
            const int r = R * ahead.u + own;
            const char *rec = nullptr;
            if (wanted) rec = page_records(a.pool, page, ahead.h, L::kBytes);
            valid = (valid & ~(FIRST << put)) |
                    (__ballot_sync(0xFFFFFFFFu, rec != nullptr) & FIRST) << put;
            if (rec) {
                rec += (r - page_slot(a.pool, r) * a.pool.page_records) * L::kBytes;
                const uint32_t keys = to + own * L::kPart + part * 16;
#pragma unroll
                for (int i = 0; i < L::kPart / (16 * LANES); ++i)
                    copy16(keys + i * 16 * LANES, rec + part * 16 + i * 16 * LANES);
                if (FMT != W4_KV_BF16 && part < 4)
                    copy16(to + S::kMetaAt + own * 64 + part * 16, rec + L::kMeta + part * 16);
            }
            const float *old = out.row0 > 0 ? out.after : out.before;
            if (old && (out.row0 > 0 || out.decay != 0.f)) {
                const int upto = out.row0 > 0 ? ahead_len : ahead_len - a.tokens;
                old += ((long long)ahead.b * heads + ahead.h) * out.columns;
#pragma unroll
                for (int i = 0; i < (S::kTokens + 31) / 32; ++i) {
                    const int k = lane + 32 * i, j = S::kTokens * ahead.u + k;
                    if (k < S::kTokens)
                        copy4(to + S::kBeforeAt + 4 * k, j < upto ? old + j : old, j < upto);
                }
            }
            ahead.next(units, heads, WARPS);
            look();
        }
        copies_end();
    };
    look();
#pragma unroll
    for (int i = 0; i < kWeightStages - 1; ++i) fetch(i);

    int mine = warp;                                          // units until the warp's next one
    int b = 0, h = 0, len = 0, stop = 0, u = 0, stage = 0;
    long long at = 0;
    uint4 q1[ONE ? D / 32 : 1];
    float4 f1;
    float2 m1;
    while (s.left > 0) {
        b = s.b, h = s.h, len = units.len(b), stop = min(s.n, s.u + s.left);
        at = ((long long)b * heads + h) * out.columns;
        // every row sees all keys of [seen0, seen1)
        const int seen1 = len - a.tokens + 1, seen0 = a.window > 0 ? len - a.window : 0;
        const auto load_tile = [&](int n, uint4 *q4, float4 &f, float2 &m) {
            Queries<FMT, D, 1> q;
            q.load_q(a, b, h, out.row0 + 8 * n, rows);
#pragma unroll
            for (int j = 0; j < D / 32; ++j)
                q4[j] = make_uint4(q.qf[0][2 * j][0], q.qf[0][2 * j][1], q.qf[0][2 * j + 1][0],
                                   q.qf[0][2 * j + 1][1]);
            f = FMT == W4_KV_BF16 ? make_float4(q.sc[0][0], q.sc[0][1], 0.f, 0.f)
                                  : make_float4(q.sc[0][0], q.sc[0][1], q.qs[0][0], q.qs[0][1]);
            float minus[2];
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int r = out.row0 + 8 * n + 2 * t + c;
                minus[c] = INFINITY;
                if (r < rows) {
                    const int i = token_of_row(a, r);
                    const float lse = a.lse[((long long)b * a.tokens + i) * a.q_heads +
                                            h * a.group + r - i * a.group];
                    minus[c] = lse == -INFINITY ? INFINITY : lse * kLog2e;
                }
            }
            m = make_float2(minus[0], minus[1]);
        };
        u = s.u + mine;
        if constexpr (ONE) {
            if (u < stop) load_tile(0, q1, f1, m1);
        } else {
            __syncthreads();                                  // no warp is in the last head
            for (int n = warp; n < n_tiles; n += WARPS) {
                uint4 q4[D / 32];
                load_tile(n, q4, tiles[n].factors[lane], tiles[n].minus[lane]);
#pragma unroll
                for (int j = 0; j < D / 32; ++j) tiles[n].q[j][lane] = q4[j];
            }
            __syncthreads();
        }
        for (; u < stop; u += WARPS) {
            copies_wait<kWeightStages - 2>();
            __syncwarp();                                     // everyone's copies are there, and
                                                              // the stage before is free
            const unsigned here = valid >> stage;
            fetch(stage == 0 ? kWeightStages - 1 : stage - 1);
            const uint32_t at_stage = ring + stage * S::kBytes;
            if (++stage == kWeightStages) stage = 0;
            float sum[R][2];
#pragma unroll
            for (int x = 0; x < R; ++x) {
                sum[x][0] = sum[x][1] = 0.f;
                if (!(here >> (x * LANES) & 1)) continue;
                const uint32_t rec = at_stage + x * L::kPart;
                uint32_t k[KS][4];                            // the keys' operands
                float sk[2] = {1.f, 1.f}, z[2];
                if constexpr (FMT == W4_KV_BF16) {
                    const uint32_t row = rec + (lane & 15) * L::kRow, swap = lane & 7;
#pragma unroll
                    for (int ks = 0; ks < KS; ++ks)
                        ldsm4(k[ks], row + (((2 * ks + (lane >> 4)) ^ swap) << 4));
                } else {
                    constexpr int WORDS = D * L::kBits / 128;
                    uint32_t w[2][WORDS];
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const uint32_t row = rec + (g + 8 * r) * L::kRow;
                        if constexpr (WORDS == 2) {
                            lds64(w[r], row + t * 8);
                        } else {
#pragma unroll
                            for (int i = 0; i < WORDS / 4; ++i) {
                                const int piece =
                                    (4 * i + t) ^ (FMT == W4_KV_INT8 && D == 128 ? (g & 1) << 2 : 0);
                                lds128(w[r] + 4 * i, row + piece * 16);
                            }
                        }
                        const uint32_t meta =
                            lds32(at_stage + S::kMetaAt + 64 * x + 4 * (g + 8 * r));
                        sk[r] = __half2float(__ushort_as_half((unsigned short)(meta & 0xFFFFu)));
                        z[r] = __uint_as_float(__byte_perm(meta, 0x4B000000u, 0x7332)) - 0x1p23f;
                    }
#pragma unroll
                    for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                        for (int r = 0; r < 2; ++r) {
                            if constexpr (FMT == W4_KV_INT8) {
                                k[ks][r] = w[r][ks] & 0x00FF00FFu;
                                k[ks][2 + r] = __byte_perm(w[r][ks], 0u, 0x4341);
                            } else {
                                const uint32_t v = ks & 1 ? w[r][ks >> 1] >> 8 : w[r][ks >> 1];
                                k[ks][r] = v & 0x000F000Fu;
                                k[ks][2 + r] = v & 0x00F000F0u;
                            }
                        }
                }
                const int j0 = kRecTokens * (R * u + x);
                const bool edge = j0 + kRecTokens > seen1 || j0 < seen0;
                for (int n = 0; n < (ONE ? 1 : n_tiles); ++n) {
                    const float4 f = ONE ? f1 : tiles[n].factors[lane];
                    const float2 m = ONE ? m1 : tiles[n].minus[lane];
                    // (two sums, so that half as many products wait for one another)
                    float y[4] = {0.f, 0.f, 0.f, 0.f}, y1[4] = {0.f, 0.f, 0.f, 0.f};
                    if constexpr (FMT != W4_KV_BF16) {
#pragma unroll
                        for (int c = 0; c < 4; ++c) y[c] = z[c >> 1] * (c & 1 ? f.w : f.z);
                    }
#pragma unroll
                    for (int i = 0; i < D / 32; ++i) {
                        const uint4 q = ONE ? q1[i] : tiles[n].q[i][lane];
                        const uint32_t (&ka)[4] = k[2 * i], (&kb)[4] = k[2 * i + 1];
                        if constexpr (FMT == W4_KV_BF16) {
                            mma_bf16_16816(y, ka[0], ka[1], ka[2], ka[3], q.x, q.y);
                            mma_bf16_16816(y1, kb[0], kb[1], kb[2], kb[3], q.z, q.w);
                        } else {
                            mma_f16_16816(y, ka[0], ka[1], ka[2], ka[3], q.x, q.y);
                            mma_f16_16816(y1, kb[0], kb[1], kb[2], kb[3], q.z, q.w);
                        }
                    }
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const float minus = c & 1 ? m.y : m.x;
                        float p = exp2_fast(
                            fmaf((y[c] + y1[c]) * sk[c >> 1], c & 1 ? f.y : f.x, -minus));
                        if (minus == INFINITY) p = 0.f;
                        if (edge) {
                            const int r = min(out.row0 + 8 * n + 2 * t + (c & 1), rows - 1);
                            const int last = len - a.tokens + token_of_row(a, r);
                            const int j = j0 + g + 8 * (c >> 1);
                            if (j > last || (a.window > 0 && j <= last - a.window)) p = 0.f;
                        }
                        sum[x][c >> 1] += p;
                    }
                }
            }
            float w[2];
            quad_sums<R>(sum, w);
            const int x = R == 4 ? t : R == 2 ? t >> 1 : 0;
#pragma unroll
            for (int i = 0; i < (R == 4 ? 2 : 1); ++i) {
                const int k = kRecTokens * x + g + 8 * (R == 4 ? i : R == 2 ? t & 1 : t >> 1);
                const int j = S::kTokens * u + k;
                if (j < len && (R > 1 || (t & 1) == 0)) {
                    float old = 0.f;
                    if (out.row0 > 0)
                        old = __uint_as_float(lds32(at_stage + S::kBeforeAt + 4 * k));
                    else if (out.before && out.decay != 0.f)
                        old = out.decay * __uint_as_float(lds32(at_stage + S::kBeforeAt + 4 * k));
                    out.after[at + j] = old + w[i];
                }
            }
        }
        mine = u - stop;
        s.next(units, heads, stop - s.u);
    }
    copies_wait<0>();
}

template <int FMT, int D, bool ONE>
cudaError_t launch(const AttnArgs &a, const Weights &out, int n_tiles, int num_sms,
                   cudaStream_t stream) {
    using S = Stage<FMT, D>;
    const auto bytes = [](int tiles) {
        return tiles * (int)sizeof(SharedTile<D>) + kWeightWarps * kWeightStages * S::kBytes;
    };
    static std::atomic<bool> ready[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64 || !ready[dev].load(std::memory_order_relaxed)) {
        e = cudaFuncSetAttribute(weights_kernel<FMT, D, ONE>,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize, bytes(kTilesMax));
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) ready[dev].store(true, std::memory_order_relaxed);
    }
    const long long most = (long long)(a.most + S::kTokens - 1) / S::kTokens * a.pool.seqs *
                           a.pool.kv_heads;
    const long long blocks = (most + kWeightWarps - 1) / kWeightWarps;
    const long long held = (long long)kWeightBlocks * num_sms;
    const int grid = (int)(blocks < held ? blocks : held);
    return launch_overlapped(weights_kernel<FMT, D, ONE>, dim3(grid), dim3(32 * kWeightWarps),
                             bytes(ONE ? 0 : n_tiles), stream, a, out, ONE ? 0 : n_tiles);
}

template <int FMT, int D>
cudaError_t launch_tiles(const AttnArgs &a, const Weights &out, int n_tiles, int num_sms,
                         cudaStream_t stream) {
    return n_tiles == 1 ? launch<FMT, D, true>(a, out, n_tiles, num_sms, stream)
                        : launch<FMT, D, false>(a, out, n_tiles, num_sms, stream);
}

}  // namespace

cudaError_t launch_attn_weights(const AttnArgs &a, int format, int head_dim, const float *before,
                                float decay, float *weights, int columns, int num_sms,
                                cudaStream_t stream) {
    const int rows = a.tokens * a.group;
    for (int row0 = 0; row0 < rows; row0 += 8 * kTilesMax) {
        const Weights out = {before, weights, decay, columns, row0};
        const int left = (rows - row0 + 7) / 8, n_tiles = left < kTilesMax ? left : kTilesMax;
        const auto run = [&](auto f) { return f(a, out, n_tiles, num_sms, stream); };
        const cudaError_t e =
            head_dim == 128
                ? (format == W4_KV_BF16   ? run(launch_tiles<W4_KV_BF16, 128>)
                   : format == W4_KV_INT8 ? run(launch_tiles<W4_KV_INT8, 128>)
                                          : run(launch_tiles<W4_KV_INT4, 128>))
                : (format == W4_KV_BF16   ? run(launch_tiles<W4_KV_BF16, 64>)
                   : format == W4_KV_INT8 ? run(launch_tiles<W4_KV_INT8, 64>)
                                          : run(launch_tiles<W4_KV_INT4, 64>));
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace w4
