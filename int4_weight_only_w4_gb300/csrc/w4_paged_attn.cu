// Attention of the new tokens over the paged cache (w4_paged_attn).
#include "w4_kv.cuh"

namespace w4 {
namespace {

constexpr int kThreads = 128;

// Key (which = 0) or value (1) d of token r of a record.
template <int FMT, int D>
__device__ __forceinline__ float cached(const char *rec, int which, int r, int d) {
    using L = KvLayout<FMT, D>;
    const char *at = rec + (which ? L::value(r, d) : L::key(r, d));
    if constexpr (FMT == W4_KV_BF16) {
        return __bfloat162float(*reinterpret_cast<const __nv_bfloat16 *>(at));
    } else {
        int c = (uint8_t)*at;
        if constexpr (FMT == W4_KV_INT4) c = (which ? d & 8 : d & 1) ? c >> 4 : c & 15;
        const uint32_t m =
            *reinterpret_cast<const uint32_t *>(rec + (which ? L::kMetaV : L::kMeta) + 4 * r);
        return (float)(c - (int)(m >> 16)) *
               __half2float(__ushort_as_half((unsigned short)(m & 0xFFFFu)));
    }
}

__device__ __forceinline__ float block_reduce(float v, bool is_max, float *tmp) {
    for (int o = 16; o > 0; o >>= 1) {
        const float w = __shfl_xor_sync(0xFFFFFFFFu, v, o);
        v = is_max ? fmaxf(v, w) : v + w;
    }
    __syncthreads();
    if ((threadIdx.x & 31) == 0) tmp[threadIdx.x >> 5] = v;
    __syncthreads();
    v = tmp[0];
    for (int i = 1; i < kThreads / 32; ++i) v = is_max ? fmaxf(v, tmp[i]) : v + tmp[i];
    return v;
}

// One block per (new token, query head): a thread scores one key of a tile of
// 128, then sums one value column.
template <int FMT, int D, bool F32>
__global__ void __launch_bounds__(kThreads) attn_kernel(AttnArgs a) {
    using L = KvLayout<FMT, D>;
    __shared__ float qs[D], p[kThreads], tmp[kThreads / 32];
    __shared__ const char *recs[kThreads];
    begin_after_previous();
    const int h = blockIdx.x, row = blockIdx.y, b = row / a.tokens, i = row % a.tokens;
    const int kvh = h / a.group, tid = threadIdx.x;
    int len = max(a.lens[b], 0);
    const long long room = (long long)a.pool.width * a.pool.page_tokens;
    if (len > room) {
        if (a.pool.error && tid == 0) atomicOr(a.pool.error, W4_KV_ERR_LENGTH);
        len = (int)room;
    }
    const int last = len - a.tokens + i;
    const int first = a.window > 0 ? max(0, last - a.window + 1) : 0;
    if (tid < D)
        qs[tid] = __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(
            a.q.data)[row * a.q.token_stride + h * a.q.head_stride + tid]);
    __syncthreads();
    float m = -INFINITY, l = 0.f, acc = 0.f;
    for (int j0 = first; j0 <= last; j0 += kThreads) {
        const int j = j0 + tid;
        float s = -INFINITY;
        const char *rec = nullptr;
        if (j <= last) {
            const int slot = j / a.pool.page_tokens;
            const int page = a.pool.table[b * a.pool.stride + slot];
            if (page < 0 || page >= a.pool.pages) {
                if (a.pool.error) atomicOr(a.pool.error, W4_KV_ERR_PAGE);
            } else {
                const int in = j - slot * a.pool.page_tokens;
                rec = a.pool.records +
                      (((long long)page * a.pool.kv_heads + kvh) * a.pool.page_records +
                       in / kRecTokens) * L::kBytes;
                s = 0.f;
                for (int d = 0; d < D; ++d) s += qs[d] * cached<FMT, D>(rec, 0, j % kRecTokens, d);
                s *= a.scale;
            }
        }
        const float mt = fmaxf(m, block_reduce(s, true, tmp));
        const float base = mt == -INFINITY ? 0.f : mt;
        const float e = expf(s - base), keep = expf(m - base);
        l = l * keep + block_reduce(e, false, tmp);
        p[tid] = e;
        recs[tid] = rec;
        __syncthreads();
        if (tid < D) {
            acc *= keep;
            for (int c = 0; c < kThreads && j0 + c <= last; ++c)
                if (recs[c]) acc += p[c] * cached<FMT, D>(recs[c], 1, (j0 + c) % kRecTokens, tid);
        }
        m = mt;
        __syncthreads();
    }
    if (tid < D) {
        const float o = l > 0.f ? acc / l : 0.f;
        const long long at = row * a.out.token_stride + h * a.out.head_stride + tid;
        if constexpr (F32)
            reinterpret_cast<float *>(a.out.data)[at] = o;
        else
            reinterpret_cast<__nv_bfloat16 *>(a.out.data)[at] = __float2bfloat16_rn(o);
    }
    if (a.lse && tid == 0)
        a.lse[(long long)row * a.q_heads + h] = l > 0.f ? m + logf(l) : -INFINITY;
}

template <int FMT, int D>
cudaError_t launch(const AttnArgs &a, bool f32_out, cudaStream_t stream) {
    const dim3 grid(a.q_heads, a.pool.seqs * a.tokens);
    return launch_overlapped(f32_out ? attn_kernel<FMT, D, true> : attn_kernel<FMT, D, false>,
                             grid, dim3(kThreads), 0, stream, a);
}

template <int D>
cudaError_t launch_dim(const AttnArgs &a, int format, bool f32_out, cudaStream_t stream) {
    return format == W4_KV_BF16   ? launch<W4_KV_BF16, D>(a, f32_out, stream)
           : format == W4_KV_INT8 ? launch<W4_KV_INT8, D>(a, f32_out, stream)
                                  : launch<W4_KV_INT4, D>(a, f32_out, stream);
}

}  // namespace

size_t attn_workspace_bytes(int head_dim, int num_sms) { return 512; }

cudaError_t launch_paged_attn(const AttnArgs &a, int format, int head_dim, bool f32_out,
                              int num_sms, cudaStream_t stream) {
    return head_dim == 64 ? launch_dim<64>(a, format, f32_out, stream)
                          : launch_dim<128>(a, format, f32_out, stream);
}

}  // namespace w4
