// The paged key-value cache: writing tokens (w4_kv_append: rotation of q and
// k, quantisation, scatter into records) and reading them back (w4_kv_read).
//
// Mathematics of a (token, head) group: w4_quantize's asymmetric rule with
// Q = 255 or 15 (include/w4.h), every operation rounded to nearest in fp32, so
// the codes are those of any other evaluation of the rule bit for bit.
#include "w4_kv.cuh"

namespace w4 {
namespace {

constexpr int kKvThreads = 256;

__device__ __forceinline__ float clampf(float v, float a, float b) {
    return fminf(fmaxf(v, a), b);
}

__device__ __forceinline__ float2 load_pair(const Heads &x, int t, int h, int d) {
    const __nv_bfloat16 *p = reinterpret_cast<const __nv_bfloat16 *>(x.data) +
                             t * x.token_stride + h * x.head_stride + d;
    return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(p));
}

__device__ __forceinline__ void store_pair(const Heads &x, int t, int h, int d, float2 v) {
    __nv_bfloat16 *p = reinterpret_cast<__nv_bfloat16 *>(x.data) + t * x.token_stride +
                       h * x.head_stride + d;
    *reinterpret_cast<__nv_bfloat162 *>(p) = __floats2bfloat162_rn(v.x, v.y);
}

// Values d, d + 1 (d even) of a head, rotated by row pos.
__device__ __forceinline__ float2 load_turned(const Heads &x, int t, int h, int d,
                                              const Rotation &rot, int pos) {
    const float2 own = load_pair(x, t, h, d);
    if (!rot.table || d >= 2 * rot.pairs) return own;
    const float *row = rot.table + 2LL * pos * rot.pairs;
    if (rot.layout == W4_ROPE_INTERLEAVED) {
        const float2 cs = *reinterpret_cast<const float2 *>(row + d);
        return make_float2(__fsub_rn(__fmul_rn(own.x, cs.x), __fmul_rn(own.y, cs.y)),
                           __fadd_rn(__fmul_rn(own.y, cs.x), __fmul_rn(own.x, cs.y)));
    }
    const bool first = d < rot.pairs;
    const int i = first ? d : d - rot.pairs;
    const float2 other = load_pair(x, t, h, first ? d + rot.pairs : i);
    const float4 cs = *reinterpret_cast<const float4 *>(row + 2 * i);
    if (first)
        return make_float2(__fsub_rn(__fmul_rn(own.x, cs.x), __fmul_rn(other.x, cs.y)),
                           __fsub_rn(__fmul_rn(own.y, cs.z), __fmul_rn(other.y, cs.w)));
    return make_float2(__fadd_rn(__fmul_rn(own.x, cs.x), __fmul_rn(other.x, cs.y)),
                       __fadd_rn(__fmul_rn(own.y, cs.z), __fmul_rn(other.y, cs.w)));
}

// One warp per (token, head of k, v or q).
template <int FMT, int D>
__global__ void __launch_bounds__(kKvThreads)
append_kernel(KvPool pool, Heads k, Heads v, Heads q, Heads q_out, int q_heads, TokenList list,
              Rotation rot) {
    using L = KvLayout<FMT, D>;
    begin_after_previous();
    const int lane = threadIdx.x & 31;
    const int heads = 2 * pool.kv_heads + q_heads;
    const long long n = (long long)list.tokens * heads;
    for (long long w = ((long long)blockIdx.x * kKvThreads + threadIdx.x) >> 5; w < n;
         w += (long long)gridDim.x * (kKvThreads / 32)) {
        const int t = (int)(w / heads), row = (int)(w % heads);
        TokenPlace at;
        if (!kv_place(pool, list, t, rot.table ? rot.rows : 0x7FFFFFFF, &at)) continue;
        float2 x[D / 64];
        if (row >= 2 * pool.kv_heads) {
            const int h = row - 2 * pool.kv_heads;
#pragma unroll
            for (int j = 0; j < D / 64; ++j)
                x[j] = load_turned(q, t, h, 64 * j + 2 * lane, rot, at.position);
            __syncwarp();                  // q_out may be q: all loads before any store
#pragma unroll
            for (int j = 0; j < D / 64; ++j) store_pair(q_out, t, h, 64 * j + 2 * lane, x[j]);
            continue;
        }
        const bool is_v = row >= pool.kv_heads;
        const int h = is_v ? row - pool.kv_heads : row;
#pragma unroll
        for (int j = 0; j < D / 64; ++j)
            x[j] = is_v ? load_pair(v, t, h, 64 * j + 2 * lane)
                        : load_turned(k, t, h, 64 * j + 2 * lane, rot, at.position);
        const int r = at.in_page % kRecTokens;
        char *rec = pool.records + (at.page_record + (long long)h * pool.page_records +
                                    at.in_page / kRecTokens) * L::kBytes;
        if constexpr (FMT == W4_KV_BF16) {
#pragma unroll
            for (int j = 0; j < D / 64; ++j) {
                const int d = 64 * j + 2 * lane;
                *reinterpret_cast<__nv_bfloat162 *>(rec + (is_v ? L::value(r, d) : L::key(r, d))) =
                    __floats2bfloat162_rn(x[j].x, x[j].y);
            }
        } else {
            float lo = 0.f, hi = 0.f;
#pragma unroll
            for (int j = 0; j < D / 64; ++j) {
                lo = fminf(lo, fminf(x[j].x, x[j].y));
                hi = fmaxf(hi, fmaxf(x[j].x, x[j].y));
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                lo = fminf(lo, __shfl_xor_sync(0xFFFFFFFFu, lo, o));
                hi = fmaxf(hi, __shfl_xor_sync(0xFFFFFFFFu, hi, o));
            }
            constexpr float top = (float)L::kLevels;
            const __half sh =
                __float2half_rn(fminf(__fdiv_rn(__fsub_rn(hi, lo), top), 65504.f));
            const float s = __half2float(sh);
            const float z = s == 0.f ? 0.f : clampf(rintf(__fdiv_rn(-lo, s)), 0.f, top);
            const auto code = [&](float w) {
                if (s == 0.f) return 0;
                // NaN: rintf gives NaN, and clampf's fmaxf takes 0 for it after z
                return (int)clampf((w == w ? rintf(__fdiv_rn(w, s)) : 0.f) + z, 0.f, top);
            };
#pragma unroll
            for (int j = 0; j < D / 64; ++j) {
                const int d = 64 * j + 2 * lane;
                const int c0 = code(x[j].x), c1 = code(x[j].y);
                if constexpr (FMT == W4_KV_INT8) {
                    if (is_v) {
                        rec[L::value(r, d)] = (char)c0;
                        rec[L::value(r, d + 1)] = (char)c1;
                    } else {
                        *reinterpret_cast<uint16_t *>(rec + L::key(r, d)) =
                            (uint16_t)(c0 | c1 << 8);
                    }
                } else {
                    const int up0 = __shfl_down_sync(0xFFFFFFFFu, c0, 4);
                    const int up1 = __shfl_down_sync(0xFFFFFFFFu, c1, 4);
                    if (!is_v) {
                        rec[L::key(r, d)] = (char)(c0 | c1 << 4);
                    } else if (!(d & 8)) {
                        rec[L::value(r, d)] = (char)(c0 | up0 << 4);
                        rec[L::value(r, d + 1)] = (char)(c1 | up1 << 4);
                    }
                }
            }
            if (lane == 0)
                *reinterpret_cast<uint32_t *>(rec + (is_v ? L::kMetaV : L::kMeta) + 4 * r) =
                    (uint32_t)__half_as_ushort(sh) | (uint32_t)z << 16;
        }
    }
}

template <int FMT, int D>
__global__ void __launch_bounds__(kKvThreads)
read_kernel(KvPool pool, Heads k, Heads v, TokenList list) {
    using L = KvLayout<FMT, D>;
    begin_after_previous();
    const int lane = threadIdx.x & 31;
    const int heads = 2 * pool.kv_heads;
    const long long n = (long long)list.tokens * heads;
    for (long long w = ((long long)blockIdx.x * kKvThreads + threadIdx.x) >> 5; w < n;
         w += (long long)gridDim.x * (kKvThreads / 32)) {
        const int t = (int)(w / heads), row = (int)(w % heads);
        const bool is_v = row >= pool.kv_heads;
        const int h = is_v ? row - pool.kv_heads : row;
        if (!(is_v ? v : k).data) continue;
        TokenPlace at;
        if (!kv_place(pool, list, t, 0x7FFFFFFF, &at)) continue;
        const int r = at.in_page % kRecTokens;
        const char *rec = pool.records + (at.page_record + (long long)h * pool.page_records +
                                          at.in_page / kRecTokens) * L::kBytes;
        float s = 0.f;
        int z = 0;
        if constexpr (FMT != W4_KV_BF16) {
            const uint32_t m = *reinterpret_cast<const uint32_t *>(
                rec + (is_v ? L::kMetaV : L::kMeta) + 4 * r);
            s = __half2float(__ushort_as_half((unsigned short)(m & 0xFFFFu)));
            z = (int)(m >> 16);
        }
#pragma unroll
        for (int j = 0; j < D / 64; ++j) {
            const int d = 64 * j + 2 * lane;
            const int at0 = is_v ? L::value(r, d) : L::key(r, d);
            const int at1 = is_v ? L::value(r, d + 1) : L::key(r, d + 1);
            float2 x;
            if constexpr (FMT == W4_KV_BF16) {
                x = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(rec + at0));
            } else {
                int c0 = (uint8_t)rec[at0], c1 = (uint8_t)rec[at1];
                if constexpr (FMT == W4_KV_INT4) {
                    c0 = is_v ? (d & 8 ? c0 >> 4 : c0 & 15) : c0 & 15;
                    c1 = is_v ? (d & 8 ? c1 >> 4 : c1 & 15) : c1 >> 4;
                }
                x = make_float2(__fmul_rn((float)(c0 - z), s), __fmul_rn((float)(c1 - z), s));
            }
            store_pair(is_v ? v : k, t, h, d, x);
        }
    }
}

int grid_for(long long warps, int num_sms) {
    const long long blocks = (warps + kKvThreads / 32 - 1) / (kKvThreads / 32);
    const long long cap = 8LL * num_sms;
    return (int)(blocks < cap ? blocks : cap);
}

template <int D>
cudaError_t append_dim(const KvPool &pool, int format, const Heads &k, const Heads &v,
                       const Heads &q, const Heads &q_out, int q_heads, const TokenList &list,
                       const Rotation &rot, int num_sms, cudaStream_t stream) {
    const dim3 grid(grid_for((long long)list.tokens * (2 * pool.kv_heads + q_heads), num_sms));
    const auto kernel = format == W4_KV_BF16   ? append_kernel<W4_KV_BF16, D>
                        : format == W4_KV_INT8 ? append_kernel<W4_KV_INT8, D>
                                               : append_kernel<W4_KV_INT4, D>;
    return launch_overlapped(kernel, grid, dim3(kKvThreads), 0, stream, pool, k, v, q, q_out,
                             q_heads, list, rot);
}

template <int D>
cudaError_t read_dim(const KvPool &pool, int format, const Heads &k, const Heads &v,
                     const TokenList &list, int num_sms, cudaStream_t stream) {
    const dim3 grid(grid_for((long long)list.tokens * 2 * pool.kv_heads, num_sms));
    const auto kernel = format == W4_KV_BF16   ? read_kernel<W4_KV_BF16, D>
                        : format == W4_KV_INT8 ? read_kernel<W4_KV_INT8, D>
                                               : read_kernel<W4_KV_INT4, D>;
    return launch_overlapped(kernel, grid, dim3(kKvThreads), 0, stream, pool, k, v, list);
}

}  // namespace

cudaError_t launch_kv_append(const KvPool &pool, int format, int head_dim, const Heads &k,
                             const Heads &v, const Heads &q, const Heads &q_out, int q_heads,
                             const TokenList &list, const Rotation &rot, int num_sms,
                             cudaStream_t stream) {
    return head_dim == 64 ? append_dim<64>(pool, format, k, v, q, q_out, q_heads, list, rot,
                                           num_sms, stream)
                          : append_dim<128>(pool, format, k, v, q, q_out, q_heads, list, rot,
                                            num_sms, stream);
}

cudaError_t launch_kv_read(const KvPool &pool, int format, int head_dim, const Heads &k,
                           const Heads &v, const TokenList &list, int num_sms,
                           cudaStream_t stream) {
    return head_dim == 64 ? read_dim<64>(pool, format, k, v, list, num_sms, stream)
                          : read_dim<128>(pool, format, k, v, list, num_sms, stream);
}

}  // namespace w4
