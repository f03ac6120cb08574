// Record layout of the paged key-value cache (include/w4.h, "Paged key-value
// cache") and the launches of the kernels that use it.  Internal to libw4.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "w4_attn_plan.cuh"
#include "w4_internal.cuh"

namespace w4 {

// Byte offsets inside a record of format FMT (W4_KV_*) and head dimension D.
template <int FMT, int D>
struct KvLayout {
    static constexpr int kBits = FMT == W4_KV_BF16 ? 16 : FMT == W4_KV_INT8 ? 8 : 4;
    static constexpr int kLevels = FMT == W4_KV_INT8 ? 255 : 15;
    static constexpr int kRow = D * kBits / 8;              // bytes of a token's key
    static constexpr int kPart = kRecTokens * kRow;         // bytes of all keys (values)
    static constexpr int kMeta = 2 * kPart;                 // descriptors of the keys
    static constexpr int kMetaV = kMeta + 4 * kRecTokens;   // descriptors of the values
    static constexpr int kBytes = FMT == W4_KV_BF16 ? kMeta : kMeta + 8 * kRecTokens;

    // Byte of value d of token r's key, from the start of the record (int4:
    // nibble d & 1 of it).
    __host__ __device__ static constexpr int key(int r, int d) {
        if (FMT == W4_KV_BF16) return r * kRow + (((d >> 3) ^ (r & 7)) << 4) + (d & 7) * 2;
        if (FMT == W4_KV_INT8)
            return r * kRow + (((d >> 4) ^ (D == 128 ? (r & 1) << 2 : 0)) << 4) + (d & 15);
        return r * kRow + (d >> 1);
    }
    // The same of its value (int4: nibble (d >> 3) & 1 of it).
    __host__ __device__ static constexpr int value(int r, int d) {
        if (FMT == W4_KV_BF16) return kPart + key(r, d);
        const int lane = 4 * (d & 7) + ((r & 7) >> 1), byte = 2 * (r & 1) + (r >> 3);
        if (FMT == W4_KV_INT8)
            return kPart + (d >> 5) * 512 + lane * 16 + ((d >> 3) & 3) * 4 + byte;
        return kPart + (d >> 6) * 512 + lane * 16 + ((d >> 4) & 3) * 4 + byte;
    }
};

inline int kv_record_bytes(int format, int head_dim) {
    return format == W4_KV_BF16 ? 64 * head_dim
           : format == W4_KV_INT8 ? 32 * head_dim + 128
                                  : 16 * head_dim + 128;
}

// What the kernels need of w4_kv_cache and w4_block_table.
struct KvPool {
    char *records;
    int kv_heads;
    int page_records;     // records of a page and head
    int page_shift;       // its log2, or -1
    int page_tokens;
    int pages;
    uint32_t *error;
    const int32_t *table;
    int seqs;
    int width;
    long long stride;
};

struct Heads {
    char *data;
    long long token_stride;    // in elements
    long long head_stride;
};

struct Rotation {
    const float *table;        // NULL: none
    int rows;
    int pairs;                 // rotary_dim / 2
    int layout;
};

// Tokens of w4_kv_append and w4_kv_read: token t is at positions[t] of
// sequence seq_ids[t], or of t / run without seq_ids.
struct TokenList {
    const int32_t *positions;
    const int32_t *seq_ids;
    int tokens;
    int run;                   // tokens of one sequence in a row (with seq_ids: all)
};

cudaError_t launch_rope_table(const unsigned long long *turns, int pairs, double amplitude,
                              int rows, float *table, cudaStream_t stream);
cudaError_t launch_rope(const Heads &x, const Heads &y, int tokens, int heads, int head_dim,
                        const int32_t *positions, const Rotation &rot, uint32_t *error,
                        bool wide, int num_sms, cudaStream_t stream);
cudaError_t launch_kv_append(const KvPool &pool, int format, int head_dim, const Heads &k,
                             const Heads &v, const Heads &q, const Heads &q_out, int q_heads,
                             const TokenList &list, const Rotation &rot, int num_sms,
                             cudaStream_t stream);
cudaError_t launch_kv_read(const KvPool &pool, int format, int head_dim, const Heads &k,
                           const Heads &v, const TokenList &list, int num_sms,
                           cudaStream_t stream);

// First key of a record that is not there.  The host refuses tables with room for a
// longer sequence, so it is past every length.
constexpr int kAbsent = 0x7FFFFF00;

struct AttnArgs {
    KvPool pool;
    Heads q, out;
    float *lse;
    bool f32_out;    // out is float, not bfloat16
    const int32_t *lens;
    int q_heads;
    int group;       // query heads per key/value head
    unsigned group_magic;    // 2^32 / group, rounded up: rows below 2^16 divide by it
    int tokens;      // new tokens per sequence
    float scale;
    int window;      // 0: none
    const int32_t *blocks;    // the blocks to look at, `most` a head, or NULL: all
    const int32_t *counts;    // how many of them, by sequence
    int most;
    void *workspace;
};
size_t attn_workspace_bytes(int head_dim, int num_sms);
// (a.lse is read; a.most: columns or the table's room, the smaller one)
cudaError_t launch_attn_weights(const AttnArgs &a, int format, int head_dim, const float *before,
                                float decay, float *weights, int columns, int num_sms,
                                cudaStream_t stream);
cudaError_t launch_paged_attn(const AttnArgs &a, int format, int head_dim, int num_sms,
                              cudaStream_t stream);

cudaError_t launch_key_bounds(const KvPool &pool, int format, int head_dim, void *bounds,
                              int tokens, const int32_t *lens, int num_sms, cudaStream_t stream);
cudaError_t launch_block_scores(const KvPool &pool, int head_dim, const void *bounds,
                                const Heads &q, int group, unsigned group_magic, int tokens,
                                const int32_t *lens, float *scores, int columns, int num_sms,
                                cudaStream_t stream);

cudaError_t launch_kv_gather(const KvPool &from, const KvPool &to, int format, int head_dim,
                             const int32_t *lens, const int32_t *index, const int32_t *counts,
                             int most, const float *weights, int columns, float *weights_out,
                             int columns_out, int num_sms, cudaStream_t stream);
cudaError_t launch_select(const float *scores, int seqs, int heads, int columns,
                          const int32_t *lens, int unit, int first, int last, int count,
                          int32_t *index, int32_t *counts, int num_sms, cudaStream_t stream);

// Launch with programmatic stream serialisation: the grid may start while the
// previous kernel of the stream drains; every kernel launched this way calls
// griddepcontrol.wait before it touches memory that another kernel writes.
template <typename... Params, typename... Args>
cudaError_t launch_overlapped(void (*kernel)(Params...), dim3 grid, dim3 block, size_t smem,
                              cudaStream_t stream, Args &&...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...);
}

inline bool same_place(const Heads &x, const Heads &y) {
    return x.data == y.data && x.token_stride == y.token_stride && x.head_stride == y.head_stride;
}

// Units of a head that turn_unit takes (in place nothing is copied).
inline int turn_units(const Heads &x, const Heads &y, int head_dim, const Rotation &rot) {
    return (rot.layout == W4_ROPE_HALF ? rot.pairs / 8 : rot.pairs / 4) +
           (same_place(x, y) ? 0 : (head_dim - 2 * rot.pairs) / 8);
}

#ifdef __CUDACC__
__device__ __forceinline__ void begin_after_previous() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

// A pair turned by cs = (cos, sin): every operation rounded once, so that the
// result is that of any other evaluation of the formula bit for bit.
__device__ __forceinline__ float2 turn_pair(float a, float b, float2 cs) {
    return make_float2(__fsub_rn(__fmul_rn(a, cs.x), __fmul_rn(b, cs.y)),
                       __fadd_rn(__fmul_rn(b, cs.x), __fmul_rn(a, cs.y)));
}
__device__ __forceinline__ float bf16_low(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_high(uint32_t w) {
    return __uint_as_float(w & 0xFFFF0000u);
}
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}
// 8 bfloat16 values and their 8 partners.
__device__ __forceinline__ void turn_halves(uint4 &a, uint4 &b, const float2 (&cs)[8]) {
    uint32_t *wa = &a.x, *wb = &b.x;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 r0 = turn_pair(bf16_low(wa[i]), bf16_low(wb[i]), cs[2 * i]);
        const float2 r1 = turn_pair(bf16_high(wa[i]), bf16_high(wb[i]), cs[2 * i + 1]);
        wa[i] = bf16_pair(r0.x, r1.x);
        wb[i] = bf16_pair(r0.y, r1.y);
    }
}
// 4 pairs of neighbours.
__device__ __forceinline__ void turn_neighbours(uint4 &a, const float2 (&cs)[8]) {
    uint32_t *w = &a.x;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 r = turn_pair(bf16_low(w[i]), bf16_high(w[i]), cs[i]);
        w[i] = bf16_pair(r.x, r.y);
    }
}

// What one thread turns with 16-byte accesses: unit u of the heads h0, h0 +
// groups, ... of a token, HEADS of them at most, all their loads under way
// together and the unit's (cos, sin) in registers.  A unit is 8 values and their
// 8 partners (half), 4 pairs (interleaved), or past the rotated part 8 values
// to copy.  row: the table's; back: the transposed rotation.
template <int LAYOUT, int HEADS>
__device__ __forceinline__ void turn_unit(const Heads &x, const Heads &y, long long t, int u,
                                          int h0, int groups, int heads, const Rotation &rot,
                                          unsigned row, bool back) {
    const int turned = LAYOUT == W4_ROPE_HALF ? rot.pairs / 8 : rot.pairs / 4;
    const bool turns = u < turned;
    const int d = LAYOUT == W4_ROPE_HALF && !turns ? 8 * (u + turned) : 8 * u;
    float2 cs[8];
    if (turns) {
        const float4 *tab = reinterpret_cast<const float4 *>(
            rot.table + 2 * ((long long)row * rot.pairs + (LAYOUT == W4_ROPE_HALF ? d : d / 2)));
#pragma unroll
        for (int i = 0; i < (LAYOUT == W4_ROPE_HALF ? 4 : 2); ++i) {
            const float4 v = tab[i];
            cs[2 * i] = make_float2(v.x, back ? -v.y : v.y);
            cs[2 * i + 1] = make_float2(v.z, back ? -v.w : v.w);
        }
    }
    const __nv_bfloat16 *in =
        reinterpret_cast<const __nv_bfloat16 *>(x.data) + t * x.token_stride + d;
    __nv_bfloat16 *out = reinterpret_cast<__nv_bfloat16 *>(y.data) + t * y.token_stride + d;
    uint4 a[HEADS], b[HEADS];
#pragma unroll
    for (int i = 0; i < HEADS; ++i) {
        const int h = h0 + i * groups;
        if (h >= heads) continue;
        a[i] = *reinterpret_cast<const uint4 *>(in + h * x.head_stride);
        if (LAYOUT == W4_ROPE_HALF && turns)
            b[i] = *reinterpret_cast<const uint4 *>(in + h * x.head_stride + rot.pairs);
    }
#pragma unroll
    for (int i = 0; i < HEADS; ++i) {
        const int h = h0 + i * groups;
        if (h >= heads) continue;
        if (turns) {
            if constexpr (LAYOUT == W4_ROPE_HALF)
                turn_halves(a[i], b[i], cs);
            else
                turn_neighbours(a[i], cs);
        }
        *reinterpret_cast<uint4 *>(out + h * y.head_stride) = a[i];
        if (LAYOUT == W4_ROPE_HALF && turns)
            *reinterpret_cast<uint4 *>(out + h * y.head_stride + rot.pairs) = b[i];
    }
}

// Where token t of a list is kept: the first record of its page for head 0,
// and the token's place; false (and a bit of the error word) if it is
// nowhere, false without one for padding.
struct TokenPlace {
    long long page_record;     // page * kv_heads * page_records
    int in_page;               // token of the page
    int position;
};

__device__ __forceinline__ bool kv_place(const KvPool &pool, const TokenList &list, int t,
                                         int rotation_rows, TokenPlace *at) {
    const int pos = list.positions[t];
    if (pos < 0) return false;
    const int seq = list.seq_ids ? list.seq_ids[t] : t / list.run;
    uint32_t bad = 0;
    int page = 0;
    const int slot = pos / pool.page_tokens;
    if (seq < 0 || seq >= pool.seqs)
        bad = W4_KV_ERR_SEQUENCE;
    else if (slot >= pool.width || pos >= rotation_rows)
        bad = W4_KV_ERR_POSITION;
    else {
        page = pool.table[seq * pool.stride + slot];
        if (page < 0 || page >= pool.pages) bad = W4_KV_ERR_PAGE;
    }
    if (bad) {
        if (pool.error) atomicOr(pool.error, bad);
        return false;
    }
    at->page_record = (long long)page * pool.kv_heads * pool.page_records;
    at->in_page = pos - slot * pool.page_tokens;
    at->position = pos;
    return true;
}
#endif

}  // namespace w4
