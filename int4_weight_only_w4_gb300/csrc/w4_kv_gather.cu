// Moves listed tokens of the paged cache to other pages, every key/value head its
// own ones (w4_kv_gather): codes, scales and zero points as they are.
//
// A warp makes one record of 16 new places.  Keys and bf16 values are rows, copied
// in 16-byte pieces whose exchange inside a row depends on the token's place.  Of
// quantised values 16 bytes belong to 4 tokens, 4 bytes of each, at the same place
// in all records but for the tokens' lane and byte: a lane loads the four pieces
// that its own four tokens come from and picks its bytes.  A place that gets no
// token keeps what it holds: it comes from itself.
//
// Bound by DRAM, and by what the layout makes it fetch.  bf16 rows are whole sectors:
// 4096 of 16384 tokens of 16 sequences and 4 heads of 128 take 49.9 us, 81 % of a
// copy's rate.  A quantised value's bytes lie in every second sector of its record's
// values, so in 4 bits a token that is kept by itself makes DRAM move 640 bytes for its
// 136: 4096 of 32768 tokens, 200 MB and 30 us at a copy's rate instead of 11, take
// 40.0 us (DRAM busy 63 % of them, all in single sectors); one in two kept 25.6 us;
// in 8 bits 63.7.
// What a unit comes from (list, then page) is asked for two and one units earlier:
// without that, and with a grid larger than the device holds, 46.7 us.
#include "w4_kv_work.cuh"

namespace w4 {
namespace {

constexpr int kGatherWarps = 4;

// Blocks an SM, by what a lane holds of a record.
template <int FMT, int D>
constexpr int kGatherBlocks = D == 64 ? 8 : FMT == W4_KV_BF16 ? 4 : FMT == W4_KV_INT8 ? 5 : 8;

struct Lists {
    KvPool to;                    // the pool, by the table of the new places
    const int32_t *counts;
    int most;

    __device__ __forceinline__ int count(int b) const {
        return cached_len(to, counts, b, min(most, to.width * to.page_tokens));
    }
    __device__ __forceinline__ int operator()(int b) const {
        return (count(b) + kRecTokens - 1) / kRecTokens;
    }
};

struct Moved {
    const int32_t *index;
    const float *weights;         // NULL: none
    float *weights_out;
    int columns, columns_out;
};

template <int FMT, int D>
__global__ void __launch_bounds__(32 * kGatherWarps, kGatherBlocks<FMT, D>)
gather_kernel(const KvPool from, const int32_t *lens, const Lists lists, const Moved m) {
    using L = KvLayout<FMT, D>;
    begin_after_previous();
    const int lane = threadIdx.x & 31;
    const KvPool &to = lists.to;
    Share s(lists, to.seqs, to.kv_heads, blockIdx.x * kGatherWarps + (threadIdx.x >> 5),
            gridDim.x * kGatherWarps);
    // What a lane knows of a unit, asked for while the one before is moved: places
    // there are, the new page, and the token of place r = lane % 16 with its old page.
    struct Ahead {
        int there, page, token, from_page;
    };
    const int r = lane & 15;
    const auto token_of = [&](const Share &s, Ahead &x) {
        const int first = kRecTokens * s.u;
        x.there = min(lists.count(s.b) - first, kRecTokens);
        x.page = to.table[s.b * to.stride + s.u / to.page_records];
        x.token = -1;
        if (r < x.there)
            x.token = m.index[((long long)s.b * to.kv_heads + s.h) * lists.most + first + r];
    };
    const auto page_of = [&](const Share &s, Ahead &x) {
        if (x.token < 0) return;
        int len = cached_len(from, lens, s.b, from.width * from.page_tokens);
        if (m.weights) len = min(len, m.columns);
        if (x.token >= len) {
            if (from.error) atomicOr(from.error, W4_KV_ERR_POSITION);
            x.token = -1;
        } else {
            x.from_page = from.table[s.b * from.stride + x.token / from.page_tokens];
        }
    };
    Share ahead = s, after = s;
    Ahead next, third;
    if (s.left > 0) token_of(s, next), page_of(s, next);
    after.next(lists, to.kv_heads);
    if (after.left > 0) token_of(after, third);
    for (; s.left > 0; s.next(lists, to.kv_heads)) {
        const Ahead now = next;
        next = third;
        ahead = after;
        if (ahead.left > 0) {
            page_of(ahead, next);
            after.next(lists, to.kv_heads);
            if (after.left > 0) token_of(after, third);
        }
        const int first = kRecTokens * s.u, slot = s.u / to.page_records;
        char *dst = page_records(to, now.page, s.h, L::kBytes);
        if (!dst) continue;
        dst += (s.u - slot * to.page_records) * L::kBytes;
        // lane r (and r + 16): the record that place r's token comes from, and its
        // place there
        const long long row = (long long)s.b * to.kv_heads + s.h;
        const char *src = nullptr;
        int src_r = r;
        if (now.token >= 0) {
            const int in_page = now.token % from.page_tokens;
            src = page_records(from, now.from_page, s.h, L::kBytes);
            if (src) {
                src += in_page / kRecTokens * L::kBytes, src_r = in_page % kRecTokens;
                if (m.weights && lane < 16)
                    m.weights_out[row * m.columns_out + first + r] =
                        m.weights[row * m.columns + now.token];
            }
        }
        const unsigned comes = __ballot_sync(0xFFFFFFFFu, src != nullptr) & 0xFFFFu;
        if (!comes) continue;
        if (!src) src = dst;
        const unsigned long long src_at = reinterpret_cast<unsigned long long>(src);
        const auto source = [&](int x) {
            return reinterpret_cast<const char *>(__shfl_sync(0xFFFFFFFFu, src_at, x));
        };
        // ---- rows: keys, and values in bf16
        constexpr int PIECES = L::kRow / 16, ROWS = 32 / PIECES, EACH = kRecTokens / ROWS;
        constexpr int SIDES = FMT == W4_KV_BF16 ? 2 : 1;
        const int piece = lane % PIECES;
        const auto at = [&](int x) { return L::key(x, piece * 128 / L::kBits); };
        uint4 v[SIDES][EACH];
#pragma unroll
        for (int k = 0; k < EACH; ++k) {
            const int x = lane / PIECES + k * ROWS;
            const char *p = source(x) + at(__shfl_sync(0xFFFFFFFFu, src_r, x));
#pragma unroll
            for (int y = 0; y < SIDES; ++y)
                v[y][k] = *reinterpret_cast<const uint4 *>(p + y * L::kPart);
        }
        // ---- quantised values, and descriptors
        constexpr int PARTS = FMT == W4_KV_BF16 ? 1 : L::kPart / 512;
        uint4 out[PARTS];
        uint32_t meta = 0;
        if constexpr (FMT != W4_KV_BF16) {
            // bytes 0 .. 3 of a word: tokens 2t, 2t + 8, 2t + 1, 2t + 9
            const int t2 = 2 * (lane & 3);
            const char *p[4];
            int byte[4];
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                const int x = t2 + 8 * (y & 1) + (y >> 1);
                const int sr = __shfl_sync(0xFFFFFFFFu, src_r, x);
                p[y] = source(x) + L::kPart + ((lane & ~3) + ((sr & 7) >> 1)) * 16;
                byte[y] = 2 * (sr & 1) + (sr >> 3);
            }
            const uint32_t low = byte[0] | (4 + byte[1]) << 4, high = byte[2] | (4 + byte[3]) << 4;
#pragma unroll
            for (int i = 0; i < PARTS; ++i) {
                uint4 w[4];
#pragma unroll
                for (int y = 0; y < 4; ++y) w[y] = *reinterpret_cast<const uint4 *>(p[y] + i * 512);
                const auto pick = [&](uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
                    return __byte_perm(__byte_perm(a, b, low), __byte_perm(c, d, high), 0x5410);
                };
                out[i] = make_uint4(pick(w[0].x, w[1].x, w[2].x, w[3].x),
                                    pick(w[0].y, w[1].y, w[2].y, w[3].y),
                                    pick(w[0].z, w[1].z, w[2].z, w[3].z),
                                    pick(w[0].w, w[1].w, w[2].w, w[3].w));
            }
            meta = *reinterpret_cast<const uint32_t *>(
                src + (lane < 16 ? L::kMeta : L::kMetaV) + 4 * src_r);
        }
#pragma unroll
        for (int k = 0; k < EACH; ++k) {
            const int x = lane / PIECES + k * ROWS;
            if (!(comes >> x & 1)) continue;
#pragma unroll
            for (int y = 0; y < SIDES; ++y)
                *reinterpret_cast<uint4 *>(dst + y * L::kPart + at(x)) = v[y][k];
        }
        if constexpr (FMT != W4_KV_BF16) {
#pragma unroll
            for (int i = 0; i < PARTS; ++i)
                *reinterpret_cast<uint4 *>(dst + L::kPart + i * 512 + lane * 16) = out[i];
            if (comes >> r & 1)
                *reinterpret_cast<uint32_t *>(dst + (lane < 16 ? L::kMeta : L::kMetaV) + 4 * r) =
                    meta;
        }
        __syncwarp();
    }
}

}  // namespace

cudaError_t launch_kv_gather(const KvPool &from, const KvPool &to, int format, int head_dim,
                             const int32_t *lens, const int32_t *index, const int32_t *counts,
                             int most, const float *weights, int columns, float *weights_out,
                             int columns_out, int num_sms, cudaStream_t stream) {
    const Lists lists = {to, counts, most};
    const Moved moved = {index, weights, weights_out, columns, columns_out};
    const long long room = (long long)to.width * to.page_records,
                    listed = ((long long)most + kRecTokens - 1) / kRecTokens;
    const long long units = (room < listed ? room : listed) * to.seqs * to.kv_heads;
    const long long blocks = (units + kGatherWarps - 1) / kGatherWarps;
    const auto run = [&](auto kernel, int held) {
        const long long most = (long long)held * num_sms;
        return launch_overlapped(kernel, dim3((unsigned)(blocks < most ? blocks : most)),
                                 dim3(32 * kGatherWarps), 0, stream, from, lens, lists, moved);
    };
    if (head_dim == 128)
        return format == W4_KV_BF16
                   ? run(gather_kernel<W4_KV_BF16, 128>, kGatherBlocks<W4_KV_BF16, 128>)
               : format == W4_KV_INT8
                   ? run(gather_kernel<W4_KV_INT8, 128>, kGatherBlocks<W4_KV_INT8, 128>)
                   : run(gather_kernel<W4_KV_INT4, 128>, kGatherBlocks<W4_KV_INT4, 128>);
    return format == W4_KV_BF16
               ? run(gather_kernel<W4_KV_BF16, 64>, kGatherBlocks<W4_KV_BF16, 64>)
           : format == W4_KV_INT8
               ? run(gather_kernel<W4_KV_INT8, 64>, kGatherBlocks<W4_KV_INT8, 64>)
               : run(gather_kernel<W4_KV_INT4, 64>, kGatherBlocks<W4_KV_INT4, 64>);
}

}  // namespace w4
