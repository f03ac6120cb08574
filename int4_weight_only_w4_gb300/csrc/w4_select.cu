// The best items of every row of scores, in ascending order (w4_select).
//
// A score becomes an unsigned key in the scores' order.  The count-th largest key
// is found digit by digit (11, 11 and 10 bits): a histogram of the keys that
// share the digits found so far, and a sum over its bins from the top until
// `count` is reached.  Then an item is chosen if its key is above that one, or
// equal to it and among the first of those; how many are chosen before it is its
// place in the list, so nothing is sorted.
//
// A row is shared by a cluster of up to 8 blocks, whose keys stay in registers
// through all passes (131072 items at 16 a thread; longer rows are read again by
// each pass); the blocks add up each other's histograms through distributed
// shared memory.
#include "w4_device.cuh"
#include "w4_kv.cuh"

namespace w4 {
namespace {

constexpr int kKeys = 16;                 // items of a thread that stays resident
constexpr int kBins = 2048;
constexpr uint32_t kAlways = 0xFFFFFFFFu, kNan = 0xFFFFFFFEu;

struct Job {
    const float *scores;
    const int32_t *lens;
    int32_t *index, *counts;
    int heads, columns, unit, first, last, count;
};

__device__ __forceinline__ int items_of(const Job &j, int b) {
    const int len = max(j.lens[b], 0);
    return min(len / j.unit + (len % j.unit != 0), j.columns);
}

// Larger scores have larger keys, -0 and 0 the same one, NaN the largest.  (0 is
// no score's key.)
__device__ __forceinline__ uint32_t key_of(float s) {
    const uint32_t b = __float_as_uint(s + 0.f);
    if (s != s) return kNan;
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile(
        "barrier.cluster.arrive.release.aligned;\n\t"
        "barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// A word of block `rank`'s shared memory, by its address in the own one.
__device__ __forceinline__ int cluster_load(const int *p, int rank) {
    uint32_t at;
    int r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_addr(p)), "r"(rank));
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(r) : "r"(at) : "memory");
    return r;
}

template <int THREADS, bool RESIDENT>
__global__ void __launch_bounds__(THREADS) select_kernel(const Job j, int blocks) {
    constexpr int WARPS = THREADS / 32, EACH = kBins / THREADS;
    __shared__ int hist[3][kBins];
    __shared__ int sums[WARPS], above[WARPS], equal[WARPS], total[2];
    __shared__ int found_bin, found_need, found_in;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    for (int i = tid; i < 3 * kBins; i += THREADS) (&hist[0][0])[i] = 0;
    begin_after_previous();
    const int rank = blocks > 1 ? cluster_rank() : 0;
    const long long row = blockIdx.x / blocks;
    const int b = (int)(row / j.heads), n = items_of(j, b);
    int32_t *out = j.index + row * j.count;
    if (rank == 0 && tid == 0 && row % j.heads == 0) j.counts[b] = min(n, j.count);
    if (n <= j.count) {                                       // all of them, in every block
        for (int i = rank * THREADS + tid; i < n; i += blocks * THREADS) out[i] = i;
        return;
    }
    // a block, and a warp of it, has neighbouring items: 32 a round
    const int rounds = ((n + blocks - 1) / blocks + THREADS - 1) / THREADS;
    const int start = (rank * WARPS + warp) * 32 * rounds;
    const float *in = j.scores + row * j.columns;
    const auto key_at = [&](int k) -> uint32_t {
        const int i = start + 32 * k + lane;
        if (i >= n) return 0u;
        return i < j.first || i >= n - j.last ? kAlways : key_of(in[i]);
    };
    uint32_t keys[RESIDENT ? kKeys : 1];
    if constexpr (RESIDENT) {
#pragma unroll
        for (int k = 0; k < kKeys; ++k) keys[k] = k < rounds ? key_at(k) : 0u;
    }
    // f(key) of each of the thread's items, all lanes of a warp together
    const auto each_key = [&](auto f) {
        if constexpr (RESIDENT) {
#pragma unroll
            for (int k = 0; k < kKeys; ++k)
                if (k < rounds) f(keys[k], k);
        } else {
            for (int k = 0; k < rounds; ++k) f(key_at(k), k);
        }
    };

    // ---- the count-th largest key, and how many equal to it are chosen
    uint32_t found = 0;                                       // its upper digits
    int need = j.count, shift = 32;
    __syncthreads();
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
        const int bits = pass < 2 ? 11 : 10, top = shift;
        shift -= bits;
        int *h = hist[pass];
        each_key([&](uint32_t key, int) {
            const bool counts = top == 32 || key >> top == found >> top;
            const int bin = counts ? (int)(key >> shift & ((1u << bits) - 1)) : -1;
            if (__all_sync(0xFFFFFFFFu, bin == __shfl_sync(0xFFFFFFFFu, bin, 0))) {
                // often, where many scores are equal
                if (lane == 0 && counts) atomicAdd(&h[bin], 32);
            } else if (counts) {
                atomicAdd(&h[bin], 1);
            }
        });
        if (blocks > 1)
            cluster_sync();
        else
            __syncthreads();
        // thread t: bins from the top, EACH of them
        const int bin0 = kBins - 1 - tid * EACH;
        int in_bin[EACH], mine = 0;
#pragma unroll
        for (int x = 0; x < EACH; ++x) {
            in_bin[x] = 0;
            if (blocks > 1)
                for (int r = 0; r < blocks; ++r) in_bin[x] += cluster_load(&h[bin0 - x], r);
            else
                in_bin[x] = h[bin0 - x];
            mine += in_bin[x];
        }
        int upto = mine;
#pragma unroll
        for (int x = 1; x < 32; x <<= 1) {
            const int v = __shfl_up_sync(0xFFFFFFFFu, upto, x);
            if (lane >= x) upto += v;
        }
        if (lane == 31) sums[warp] = upto;
        __syncthreads();
        int before = upto - mine;
        for (int w = 0; w < warp; ++w) before += sums[w];
        if (before < need && need <= before + mine) {
#pragma unroll
            for (int x = 0; x < EACH; ++x) {
                if (before < need && need <= before + in_bin[x])
                    found_bin = bin0 - x, found_need = need - before, found_in = in_bin[x];
                before += in_bin[x];
            }
        }
        __syncthreads();
        found |= (uint32_t)found_bin << shift;
        need = found_need;
        if (need == found_in) break;                          // every one of the bin
    }
    if (need == found_in) --found, need = 0;                  // (found is no score's 0)

    // ---- how many are above it, or equal to it, before a warp's first item
    int n_above = 0, n_equal = 0;
    each_key([&](uint32_t key, int) {
        n_above += __popc(__ballot_sync(0xFFFFFFFFu, key > found));
        n_equal += __popc(__ballot_sync(0xFFFFFFFFu, key == found));
    });
    if (lane == 0) above[warp] = n_above, equal[warp] = n_equal;
    __syncthreads();
    int at_above = 0, at_equal = 0;
    for (int w = 0; w < warp; ++w) at_above += above[w], at_equal += equal[w];
    if (blocks > 1) {
        if (tid == THREADS - 1) total[0] = at_above + n_above, total[1] = at_equal + n_equal;
        cluster_sync();
        for (int r = 0; r < rank; ++r)
            at_above += cluster_load(&total[0], r), at_equal += cluster_load(&total[1], r);
        // (no block ends while another reads its shared memory)
        asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    }
    each_key([&](uint32_t key, int k) {
        const unsigned more = __ballot_sync(0xFFFFFFFFu, key > found);
        const unsigned same = __ballot_sync(0xFFFFFFFFu, key == found);
        const unsigned lower = (1u << lane) - 1;
        const int e = at_equal + __popc(same & lower);
        if (key > found || (key == found && e < need))
            out[at_above + __popc(more & lower) + min(e, need)] = start + 32 * k + lane;
        at_above += __popc(more), at_equal += __popc(same);
    });
    if (blocks > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

template <int THREADS, bool RESIDENT>
cudaError_t launch(const Job &job, long long rows, int blocks, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(rows * blocks));
    cfg.blockDim = dim3(THREADS);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = blocks;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = blocks > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, select_kernel<THREADS, RESIDENT>, job, blocks);
}

}  // namespace

cudaError_t launch_select(const float *scores, int seqs, int heads, int columns,
                          const int32_t *lens, int unit, int first, int last, int count,
                          int32_t *index, int32_t *counts, cudaStream_t stream) {
    const Job job = {scores, lens, index, counts, heads, columns, unit, first, last, count};
    const long long rows = (long long)seqs * heads;
    if (columns <= 256 * kKeys) return launch<256, true>(job, rows, 1, stream);
    int blocks = 1;
    while (blocks < 8 && (long long)blocks * 1024 * kKeys < columns) blocks *= 2;
    return columns <= blocks * 1024 * kKeys ? launch<1024, true>(job, rows, blocks, stream)
                                            : launch<1024, false>(job, rows, blocks, stream);
}

}  // namespace w4
