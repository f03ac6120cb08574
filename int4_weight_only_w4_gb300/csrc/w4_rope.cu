// Rotary positions: the table of rotations (w4_rope_table) and its
// application to the heads of token rows (w4_rope).
//
// Mathematics.  Pair i of a head, (a, b), at position p becomes
// (a c - b s, b c + a s) with (c, s) = amplitude * (cos, sin)(p f_i).  The
// table holds (c, s) in fp32; its angles are products of an integer and a
// frequency, and fp32 would leave p f_i with an error that grows with p (at
// p = 10^5 the cosine would keep three digits).  So the host writes f_i / 2 pi
// as a fraction of 2^64 turns and the kernel multiplies it by p modulo 2^64:
// the whole turns drop out exactly, and what is left is an angle in one turn
// with an error below p * 2^-65 turns.  sincospi in fp64 then gives the pair.
// That is one launch per model, not per call.
#include "w4_kv.cuh"

namespace w4 {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kMaxPairs = 256;

struct Turns {
    unsigned long long f[kMaxPairs];
};

__global__ void __launch_bounds__(kRopeThreads)
rope_table_kernel(const __grid_constant__ Turns turns, int pairs, double amplitude, int rows,
                  float2 *__restrict__ table) {
    begin_after_previous();
    const long long n = (long long)rows * pairs;
    for (long long e = (long long)blockIdx.x * kRopeThreads + threadIdx.x; e < n;
         e += (long long)gridDim.x * kRopeThreads) {
        const int p = (int)(e / pairs), i = (int)(e - (long long)p * pairs);
        const long long phase = (long long)((unsigned long long)p * turns.f[i]);
        double s, c;
        sincospi((double)phase * 0x1p-63, &s, &c);
        table[e] = make_float2((float)(amplitude * c), (float)(amplitude * s));
    }
}

// Any alignment: one thread per (token, head, pair), then per value past the
// rotated ones.
__global__ void __launch_bounds__(kRopeThreads)
rope_kernel(Heads x, Heads y, int tokens, int heads, int head_dim,
            const int32_t *positions, Rotation rot, uint32_t *error) {
    begin_after_previous();
    const int units = rot.pairs + head_dim - 2 * rot.pairs;
    const long long n = (long long)tokens * heads * units;
    for (long long e = (long long)blockIdx.x * kRopeThreads + threadIdx.x; e < n;
         e += (long long)gridDim.x * kRopeThreads) {
        const long long th = e / units;
        const int u = (int)(e - th * units), t = (int)(th / heads), h = (int)(th % heads);
        const int pos = positions[t];
        const unsigned row = pos < 0 ? 0u - (unsigned)pos : (unsigned)pos;
        if (row >= (unsigned)rot.rows) {
            if (error && u == 0 && h == 0) atomicOr(error, W4_KV_ERR_POSITION);
            continue;
        }
        const __nv_bfloat16 *in = reinterpret_cast<const __nv_bfloat16 *>(x.data) +
                                  t * x.token_stride + h * x.head_stride;
        __nv_bfloat16 *out = reinterpret_cast<__nv_bfloat16 *>(y.data) + t * y.token_stride +
                             h * y.head_stride;
        if (u >= rot.pairs) {
            const int d = u + rot.pairs;
            out[d] = in[d];
            continue;
        }
        const float2 cs =
            reinterpret_cast<const float2 *>(rot.table)[(long long)row * rot.pairs + u];
        const int da = rot.layout == W4_ROPE_HALF ? u : 2 * u;
        const int db = rot.layout == W4_ROPE_HALF ? u + rot.pairs : 2 * u + 1;
        const float2 r = turn_pair(__bfloat162float(in[da]), __bfloat162float(in[db]),
                                   make_float2(cs.x, pos < 0 ? -cs.y : cs.y));
        out[da] = __float2bfloat16_rn(r.x);
        out[db] = __float2bfloat16_rn(r.y);
    }
}

// Rows on 16-byte boundaries: a thread per unit of HEADS heads (turn_unit).
// Bound by HBM: 8192 tokens of 32 heads of 128 in 23.4 us = 5830 GB/s, 86 % of
// the measured copy; the pair kernel above takes 112 us, with its 2-byte
// accesses.
template <int LAYOUT, int HEADS>
__global__ void __launch_bounds__(kRopeThreads)
rope_wide_kernel(Heads x, Heads y, unsigned units_all, int heads, unsigned groups, unsigned units,
                 const int32_t *positions, Rotation rot, uint32_t *error) {
    begin_after_previous();
    const unsigned e = blockIdx.x * kRopeThreads + threadIdx.x;
    if (e >= units_all) return;
    const unsigned tg = e / units, u = e - tg * units, t = tg / groups, h0 = tg - t * groups;
    const int pos = positions[t];
    const unsigned row = pos < 0 ? 0u - (unsigned)pos : (unsigned)pos;
    if (row >= (unsigned)rot.rows) {
        if (error && u == 0 && h0 == 0) atomicOr(error, W4_KV_ERR_POSITION);
        return;
    }
    turn_unit<LAYOUT, HEADS>(x, y, t, u, h0, groups, heads, rot, row, pos < 0);
}

int grid_for(long long units, int num_sms) {
    const long long blocks = (units + kRopeThreads - 1) / kRopeThreads, cap = 8LL * num_sms;
    return (int)(blocks < 1 ? 1 : blocks < cap ? blocks : cap);
}

template <int HEADS>
cudaError_t launch_wide(const Heads &x, const Heads &y, long long units_all, int heads,
                        unsigned groups, unsigned units, const int32_t *positions,
                        const Rotation &rot, uint32_t *error, cudaStream_t stream) {
    const auto kernel = rot.layout == W4_ROPE_HALF
                            ? rope_wide_kernel<W4_ROPE_HALF, HEADS>
                            : rope_wide_kernel<W4_ROPE_INTERLEAVED, HEADS>;
    return launch_overlapped(kernel, dim3((unsigned)((units_all + kRopeThreads - 1) / kRopeThreads)),
                             dim3(kRopeThreads), 0, stream, x, y, (unsigned)units_all, heads, groups,
                             units, positions, rot, error);
}

}  // namespace

cudaError_t launch_rope_table(const unsigned long long *turns, int pairs, double amplitude,
                              int rows, float *table, cudaStream_t stream) {
    Turns t = {};
    for (int i = 0; i < pairs; ++i) t.f[i] = turns[i];
    const long long blocks = ((long long)rows * pairs + kRopeThreads - 1) / kRopeThreads;
    return launch_overlapped(rope_table_kernel, dim3((unsigned)(blocks < 65536 ? blocks : 65536)),
                             dim3(kRopeThreads), 0, stream, t, pairs, amplitude, rows,
                             reinterpret_cast<float2 *>(table));
}

cudaError_t launch_rope(const Heads &x, const Heads &y, int tokens, int heads, int head_dim,
                        const int32_t *positions, const Rotation &rot, uint32_t *error,
                        bool wide, int num_sms, cudaStream_t stream) {
    if (wide) {
        const int units = turn_units(x, y, head_dim, rot);
        // four heads a thread once that still gives every SM two blocks
        const long long by_head = (long long)tokens * heads * units;
        const long long by_four = (long long)tokens * ((heads + 3) / 4) * units;
        if (by_four >= 2LL * num_sms * kRopeThreads && by_four < (1LL << 31))
            return launch_wide<4>(x, y, by_four, heads, (heads + 3) / 4, units, positions, rot,
                                  error, stream);
        if (by_head < (1LL << 31))
            return launch_wide<1>(x, y, by_head, heads, heads, units, positions, rot, error,
                                  stream);
    }
    const long long units = (long long)tokens * heads * (head_dim - rot.pairs);
    return launch_overlapped(rope_kernel, dim3(grid_for(units, num_sms)), dim3(kRopeThreads), 0,
                             stream, x, y, tokens, heads, head_dim, positions, rot, error);
}

}  // namespace w4
