// What every cached token gets of the new tokens' attention (w4_attn_weights).
//
// With the attention's log-sum-exp known, a token's weight is
//   w_j = sum over the rows that see j of exp2(y_j - lse log2 e),
// y the scores in units of log2, so the keys are read once more, the values not at
// all, and no token needs another one's result: nothing is joined.
//
// The blocks divide the list (sequence, head, record) evenly, from the lengths on
// the device.  A block holds the queries of one head in shared memory as the
// tensor cores' column operands; its warps take every other record of the head's
// stretch, straight from memory into registers in the layout that the products
// take, the next ones on their way meanwhile.
#include "w4_attn_query.cuh"
#include "w4_kv_work.cuh"

namespace w4 {
namespace {

constexpr int kWeightWarps = 8;
constexpr int kTilesMax = 8;             // tiles of 8 rows in shared memory

struct Weights {
    const float *before;                 // NULL: none
    float *after;
    float decay;
    int columns;
};

// Records of a sequence.
struct Records {
    const AttnArgs &a;

    __device__ __forceinline__ int len(int b) const {
        return cached_len(a.pool, a.lens, b, a.most);
    }
    __device__ __forceinline__ int operator()(int b) const {
        return (len(b) + kRecTokens - 1) / kRecTokens;
    }
};

// A lane's part of a record's keys: tokens g and g + 8.
template <int FMT, int D>
struct Keys {
    using L = KvLayout<FMT, D>;
    static constexpr int KS = D / 16, WORDS = D * L::kBits / 128;
    uint32_t w[2][WORDS];
    uint32_t meta[2];

    __device__ __forceinline__ void load(const char *rec) {
        const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const char *row = rec + (g + 8 * r) * L::kRow;
            if constexpr (WORDS == 2) {
                const uint2 v = *reinterpret_cast<const uint2 *>(row + t * 8);
                w[r][0] = v.x, w[r][1] = v.y;
            } else {
#pragma unroll
                for (int i = 0; i < WORDS / 4; ++i) {
                    int piece = 4 * i + t;
                    if (FMT == W4_KV_BF16) piece ^= g;
                    if (FMT == W4_KV_INT8 && D == 128) piece ^= (g & 1) << 2;
                    const uint4 v = *reinterpret_cast<const uint4 *>(row + piece * 16);
                    w[r][4 * i] = v.x, w[r][4 * i + 1] = v.y;
                    w[r][4 * i + 2] = v.z, w[r][4 * i + 3] = v.w;
                }
            }
            if (FMT != W4_KV_BF16)
                meta[r] = *reinterpret_cast<const uint32_t *>(rec + L::kMeta + 4 * (g + 8 * r));
        }
    }

    // s += K q of a tile whose operands are q.
    __device__ __forceinline__ void product(float (&s)[4], const uint32_t (&q)[KS][2]) const {
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            if constexpr (FMT == W4_KV_BF16) {
                const int at = 4 * (ks >> 1) + 2 * (ks & 1);
                mma_bf16_16816(s, w[0][at], w[1][at], w[0][at + 1], w[1][at + 1], q[ks][0],
                               q[ks][1]);
            } else if constexpr (FMT == W4_KV_INT8) {
                mma_f16_16816(s, w[0][ks] & 0x00FF00FFu, w[1][ks] & 0x00FF00FFu,
                              __byte_perm(w[0][ks], 0u, 0x4341),
                              __byte_perm(w[1][ks], 0u, 0x4341), q[ks][0], q[ks][1]);
            } else {
                const uint32_t x0 = ks & 1 ? w[0][ks >> 1] >> 8 : w[0][ks >> 1];
                const uint32_t x1 = ks & 1 ? w[1][ks >> 1] >> 8 : w[1][ks >> 1];
                mma_f16_16816(s, x0 & 0x000F000Fu, x1 & 0x000F000Fu, x0 & 0x00F000F0u,
                              x1 & 0x00F000F0u, q[ks][0], q[ks][1]);
            }
        }
    }
};

// Operands of one tile of rows in shared memory, by lane.
template <int D>
struct SharedTile {
    uint4 q[D / 32][32];                 // two k-steps each
    float4 factors[32];                  // sc, qs of columns 2t, 2t + 1
    float2 minus[32];                    // their lse in units of log2; infinite: no row
};

template <int FMT, int D>
__global__ void __launch_bounds__(32 * kWeightWarps, 2)
weights_kernel(const AttnArgs a, const Weights out) {
    using L = KvLayout<FMT, D>;
    constexpr int KS = D / 16;
    constexpr int R = L::kPart >= 4096 ? 1 : L::kPart >= 2048 ? 2 : 4;   // records a round
    __shared__ SharedTile<D> tiles[kTilesMax];
    begin_after_previous();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int rows = a.tokens * a.group;
    const Records records = {a};
    Share s(records, a.pool.seqs, a.pool.kv_heads, blockIdx.x, gridDim.x);
    while (s.left > 0) {
        const int b = s.b, h = s.h, len = records.len(b), stop = min(s.n, s.u + s.left);
        const int32_t *pages = a.pool.table + b * a.pool.stride;
        const long long at = ((long long)b * a.pool.kv_heads + h) * out.columns;
        // every row sees all keys of [seen0, seen1), none sees a key before unseen
        const int seen1 = len - a.tokens + 1, seen0 = a.window > 0 ? len - a.window : 0;
        const int unseen = a.window > 0 ? len - a.tokens - a.window + 1 : 0;
        for (int row0 = 0; row0 < rows; row0 += 8 * kTilesMax) {
            const int n_tiles = min(kTilesMax, (rows - row0 + 7) / 8);
            __syncthreads();
            for (int n = warp; n < n_tiles; n += kWeightWarps) {
                Queries<FMT, D, 1, true> q;
                q.load_q(a, b, h, row0 + 8 * n, rows);
#pragma unroll
                for (int j = 0; j < D / 32; ++j)
                    tiles[n].q[j][lane] = make_uint4(q.qf[0][2 * j][0], q.qf[0][2 * j][1],
                                                     q.qf[0][2 * j + 1][0], q.qf[0][2 * j + 1][1]);
                tiles[n].factors[lane] = FMT == W4_KV_BF16
                                             ? make_float4(q.sc[0][0], q.sc[0][1], 0.f, 0.f)
                                             : make_float4(q.sc[0][0], q.sc[0][1], q.qs[0][0],
                                                           q.qs[0][1]);
                float minus[2];
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const int r = row0 + 8 * n + 2 * t + c;
                    minus[c] = INFINITY;
                    if (r < rows) {
                        const int i = token_of_row(a, r);
                        const float lse = a.lse[((long long)b * a.tokens + i) * a.q_heads +
                                                h * a.group + r - i * a.group];
                        minus[c] = lse == -INFINITY ? INFINITY : lse * kLog2e;
                    }
                }
                tiles[n].minus[lane] = make_float2(minus[0], minus[1]);
            }
            __syncthreads();
            // a lane's weight: of token g (lanes 0 of a quad) or g + 8 (lanes 1)
            const auto page_of = [&](int u) { return u < stop ? pages[page_slot(a.pool, u)] : -1; };
            const auto record_of = [&](int u, int page) -> const char * {
                if (u >= stop || 16 * u + kRecTokens <= unseen) return nullptr;
                const char *first = page_records(a.pool, page, h, L::kBytes);
                return first ? first + (u - page_slot(a.pool, u) * a.pool.page_records) * L::kBytes
                             : nullptr;
            };
            constexpr int STEP = R * kWeightWarps;
            Keys<FMT, D> next[R];
            bool there[R];
            int page[R];
            const int first = s.u + warp * R;
#pragma unroll
            for (int x = 0; x < R; ++x) {
                const char *rec = record_of(first + x, page_of(first + x));
                there[x] = rec != nullptr;
                if (rec) next[x].load(rec);
            }
#pragma unroll
            for (int x = 0; x < R; ++x) page[x] = page_of(first + STEP + x);
            for (int u0 = first; u0 < stop; u0 += STEP) {
                Keys<FMT, D> keys[R];
                bool here[R];
                float old[R];
#pragma unroll
                for (int x = 0; x < R; ++x) keys[x] = next[x], here[x] = there[x];
#pragma unroll
                for (int x = 0; x < R; ++x) {
                    const int j = kRecTokens * (u0 + x) + g + 8 * t;
                    old[x] = 0.f;
                    if (t < 2 && j < len && u0 + x < stop) {
                        if (row0 > 0)
                            old[x] = out.after[at + j];
                        else if (j < len - a.tokens && out.before && out.decay != 0.f)
                            old[x] = out.decay * out.before[at + j];
                    }
                    const char *rec = record_of(u0 + STEP + x, page[x]);
                    there[x] = rec != nullptr;
                    if (rec) next[x].load(rec);
                    page[x] = page_of(u0 + 2 * STEP + x);
                }
                float sum[R][2];
#pragma unroll
                for (int x = 0; x < R; ++x) sum[x][0] = sum[x][1] = 0.f;
                for (int n = 0; n < n_tiles; ++n) {
                    uint32_t q[KS][2];
#pragma unroll
                    for (int j = 0; j < D / 32; ++j) {
                        const uint4 v = tiles[n].q[j][lane];
                        q[2 * j][0] = v.x, q[2 * j][1] = v.y;
                        q[2 * j + 1][0] = v.z, q[2 * j + 1][1] = v.w;
                    }
                    const float4 f = tiles[n].factors[lane];
                    const float2 m = tiles[n].minus[lane];
#pragma unroll
                    for (int x = 0; x < R; ++x) {
                        if (!here[x]) continue;
                        float y[4] = {0.f, 0.f, 0.f, 0.f};
                        float sk[2] = {1.f, 1.f};
                        if constexpr (FMT != W4_KV_BF16) {
#pragma unroll
                            for (int r = 0; r < 2; ++r) {
                                const uint32_t meta = keys[x].meta[r];
                                sk[r] = __half2float(
                                    __ushort_as_half((unsigned short)(meta & 0xFFFFu)));
                                const float z = (float)(meta >> 16);
                                y[2 * r] = z * f.z, y[2 * r + 1] = z * f.w;
                            }
                        }
                        keys[x].product(y, q);
                        const int j0 = kRecTokens * (u0 + x);
                        const bool edge = j0 + kRecTokens > seen1 || j0 < seen0;
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            const float minus = c & 1 ? m.y : m.x;
                            float p = exp2_fast(fmaf(y[c] * sk[c >> 1], c & 1 ? f.y : f.x, -minus));
                            if (minus == INFINITY) p = 0.f;
                            if (edge) {
                                const int r = min(row0 + 8 * n + 2 * t + (c & 1), rows - 1);
                                const int last = len - a.tokens + token_of_row(a, r);
                                const int j = j0 + g + 8 * (c >> 1);
                                if (j > last || (a.window > 0 && j <= last - a.window)) p = 0.f;
                            }
                            sum[x][c >> 1] += p;
                        }
                    }
                }
#pragma unroll
                for (int x = 0; x < R; ++x) {
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        sum[x][r] += __shfl_xor_sync(0xFFFFFFFFu, sum[x][r], 1);
                        sum[x][r] += __shfl_xor_sync(0xFFFFFFFFu, sum[x][r], 2);
                    }
                    const int j = kRecTokens * (u0 + x) + g + 8 * t;
                    if (t < 2 && j < len && u0 + x < stop)
                        out.after[at + j] = old[x] + (t ? sum[x][1] : sum[x][0]);
                }
            }
        }
        s.next(records, a.pool.kv_heads, stop - s.u);
    }
}

}  // namespace

cudaError_t launch_attn_weights(const AttnArgs &a, int format, int head_dim, const float *before,
                                float decay, float *weights, int columns, int num_sms,
                                cudaStream_t stream) {
    const Weights out = {before, weights, decay, columns};
    const long long most = (long long)(a.most + kRecTokens - 1) / kRecTokens * a.pool.seqs *
                           a.pool.kv_heads;
    const long long blocks = (most + kWeightWarps - 1) / kWeightWarps;
    const int grid = (int)(blocks < 2 * num_sms ? blocks : 2 * num_sms);
    const auto run = [&](auto kernel) {
        return launch_overlapped(kernel, dim3(grid), dim3(32 * kWeightWarps), 0, stream, a, out);
    };
    if (head_dim == 128)
        return format == W4_KV_BF16   ? run(weights_kernel<W4_KV_BF16, 128>)
               : format == W4_KV_INT8 ? run(weights_kernel<W4_KV_INT8, 128>)
                                      : run(weights_kernel<W4_KV_INT4, 128>);
    return format == W4_KV_BF16   ? run(weights_kernel<W4_KV_BF16, 64>)
           : format == W4_KV_INT8 ? run(weights_kernel<W4_KV_INT8, 64>)
                                  : run(weights_kernel<W4_KV_INT4, 64>);
}

}  // namespace w4
