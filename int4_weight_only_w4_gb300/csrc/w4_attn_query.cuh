// Queries of the paged attention as the column operand of the tensor cores, and
// small device functions around them: shared by the attention's kernels and by
// those that use its scores alone.  Internal to libw4.
#pragma once

#include "w4_device.cuh"
#include "w4_kv.cuh"

namespace w4 {

constexpr float kCodeUnit = 0x1p-24f;  // what the bits of a code are in binary16
constexpr float kLog2e = 1.44269504088896340736f;

__device__ __forceinline__ float exp2_fast(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ uint32_t pack_half(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ void ldsm4(uint32_t *r, uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void lds128(uint32_t *r, uint32_t addr) {
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void lds64(uint32_t *r, uint32_t addr) {
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];"
                 : "=r"(r[0]), "=r"(r[1])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
    uint32_t r;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(r) : "r"(addr) : "memory");
    return r;
}

// Block-table column of record r of a sequence.
__device__ __forceinline__ int page_slot(const KvPool &pool, int r) {
    return pool.page_shift >= 0 ? r >> pool.page_shift : r / pool.page_records;
}

// New token of a row.
__device__ __forceinline__ int token_of_row(const AttnArgs &a, int row) {
    return a.group == 1 ? row : (int)__umulhi((unsigned)row, a.group_magic);
}

// A warp's NT tiles of 8 rows of queries.
template <int FMT, int D, int NT>
struct Queries {
    static constexpr int KS = D / 16;                     // k-steps of a score
    uint32_t qf[NT][KS][2];      // Q as the column operand
    float sc[NT][2];             // score factor of a column
    float qs[NT][2];             // quantised: -(sum of its q), in the products' unit

    // Which value of the head goes with half e of register i of k-step ks.
    __device__ static constexpr int q_index(int ks, int i, int e, int t) {
        if (FMT == W4_KV_BF16) return 16 * ks + 8 * i + 2 * t + e;
        if (FMT == W4_KV_INT8) return 64 * (ks >> 2) + 16 * t + 4 * (ks & 3) + i + 2 * e;
        return (D / 4) * t + 8 * (ks >> 1) + 2 * (ks & 1) + i + 4 * e;
    }

    // row0: first row of the warp's tiles; rows: rows that there are.
    __device__ __forceinline__ void load_q(const AttnArgs &a, int b, int h, int row0, int rows) {
        const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int r = row0 + 8 * n + g;
            const bool there = r < rows;
            const int i = there ? token_of_row(a, r) : 0, hq = there ? r - i * a.group : 0;
            const __nv_bfloat16 *q = reinterpret_cast<const __nv_bfloat16 *>(a.q.data) +
                                     (long long)(b * a.tokens + i) * a.q.token_stride +
                                     (long long)(h * a.group + hq) * a.q.head_stride;
            if constexpr (FMT == W4_KV_BF16) {
#pragma unroll
                for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        qf[n][ks][j] =
                            there ? *reinterpret_cast<const uint32_t *>(q + q_index(ks, j, 0, t))
                                  : 0u;
                sc[n][0] = sc[n][1] = a.scale * kLog2e;
            } else {
                // a lane's values lie in runs of RUN
                constexpr int RUN = FMT == W4_KV_INT8 ? 16 : D / 4, PIECES = D / 32;
                uint4 raw[PIECES];
#pragma unroll
                for (int x = 0; x < PIECES; ++x)
                    raw[x] = there ? *reinterpret_cast<const uint4 *>(
                                         q + (x / (RUN / 8)) * 64 + RUN * t + (x % (RUN / 8)) * 8)
                                   : make_uint4(0u, 0u, 0u, 0u);
                const auto value = [&](int ks, int j, int e) {
                    const int d = q_index(ks, j, e, 0);   // of lane t = 0
                    const int at = (d / 64) * (FMT == W4_KV_INT8 ? RUN : 0) + d % 64;
                    const uint4 v = raw[at / 8];
                    const uint32_t w =
                        at % 8 < 2 ? v.x : at % 8 < 4 ? v.y : at % 8 < 6 ? v.z : v.w;
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
                // a power of two that brings the largest |q| into [2^14, 2^15);
                // in 4 bits what meets high nibbles (16 u) is 1/16 of that: q is
                // exact in binary16 down to 2^-27 of the largest
                int e = 0;
                if (top > 0.f && top < INFINITY)
                    e = 14 - max(-86, (int)(__float_as_uint(top) >> 23) - 127);
                const float up = __int_as_float((127 + e) << 23);
                float sum = 0.f;
#pragma unroll
                for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const float x = value(ks, j, 0) * up, y = value(ks, j, 1) * up;
                        const float less = FMT == W4_KV_INT4 && j == 1 ? 0.0625f : 1.f;
                        sum += x + y;
                        qf[n][ks][j] = pack_half(x * less, y * less);
                    }
                sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 1);
                sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 2);
                sum *= -kCodeUnit;
                // (finite: a score of 0 stays 0 whatever q is)
                float f = a.scale * kLog2e * __int_as_float((127 - e) << 23) / kCodeUnit;
                f = fminf(fmaxf(f, -3.0e38f), 3.0e38f);
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    sc[n][c] = __shfl_sync(0xFFFFFFFFu, f, 4 * (2 * t + c));
                    qs[n][c] = __shfl_sync(0xFFFFFFFFu, sum, 4 * (2 * t + c));
                }
            }
        }
    }
};

}  // namespace w4
