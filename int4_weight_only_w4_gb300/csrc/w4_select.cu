// The best items of every row of scores, in ascending order (w4_select).
//
// A score becomes an unsigned key in the scores' order.  The count-th largest key
// is found digit by digit (11, 11 and 10 bits): a histogram of the keys that
// share the digits found so far, and a sum over its bins from the top until
// `count` is reached.  As soon as few enough keys are left in the bin where it is,
// they are listed and the other digits found among those; once very few are, they
// are compared with one another instead.  Then an item is chosen if its key is above
// that one, or equal to it and among the first of those; how many are chosen before
// it is its place in the list, so nothing is sorted.
//
// A row's keys stay in registers from beginning to end.  Long rows are shared by a
// cluster of up to 8 blocks, which add up each other's histograms, and read each
// other's listed keys, through distributed shared memory; rows of more than 262144
// items are read again by each pass.
//
// Nothing here is bound by memory (8192 of 131072 items in 16 rows are 1.3 us of it): a
// dozen steps, each a microsecond or less, wait for one another.  Measured, captured
// calls: 64 of up to 2048 items in 256 rows 5.7 us; 1024 of up to 8192 in 256 rows
// 10.3; 8192 of 131072 in 16 rows 16.2 us, of which the first histogram takes 2, adding
// those of a cluster 1.7, the listed keys 3, the places and the stores 3; 4096 of 131072
// in 4 rows 12.7.  Many long rows are the slowest beside their bytes: 4096 of 32768 in
// 256 rows 39 to 42 us (bytes 5.7), as rows that do not fit as clusters take a block of
// 1024 threads with 32 keys each, which spills (284 bytes of stores) and has an SM to
// itself: two waves.  On the way there: loads of which each waited for a comparison 44.4
// us (16 rows); all under way together, clusters that fit at a time 31.0; keys listed
// after the first digit 25.6; a constant number of items a thread, without branches
// around each, 17.0.  Blocks of 512 threads with 64 items each 40.2: fewer warps to
// wait at a time.
#include <atomic>

#include "w4_device.cuh"
#include "w4_kv.cuh"

namespace w4 {
namespace {

constexpr int kBins = 2048;
constexpr int kListed = 4096;             // keys of a block that are listed
constexpr int kFew = 256;                 // keys that are compared with one another
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

// Larger scores have larger keys, -0 and 0 the same one, NaN (of which a sum is
// 0x7FFFFFFF) the largest.  0 is no score's key.
__device__ __forceinline__ uint32_t key_of(float s) {
    const uint32_t b = __float_as_uint(s + 0.f);
    return min(b ^ ((uint32_t)((int)b >> 31) | 0x80000000u), kNan);
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
// Words of block `rank`'s shared memory, by their address in the own one.
__device__ __forceinline__ uint32_t cluster_address(const int *p, int rank) {
    uint32_t at;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_addr(p)), "r"(rank));
    return at;
}
__device__ __forceinline__ int2 cluster_load(const int *p, int rank) {
    int2 r;
    asm volatile("ld.shared::cluster.v2.u32 {%0, %1}, [%2];"
                 : "=r"(r.x), "=r"(r.y)
                 : "r"(cluster_address(p, rank))
                 : "memory");
    return r;
}

__device__ __forceinline__ int cluster_load1(const int *p, int rank) {
    int r;
    asm volatile("ld.shared::cluster.u32 %0, [%1];"
                 : "=r"(r)
                 : "r"(cluster_address(p, rank))
                 : "memory");
    return r;
}

// What lanes below this one have, and all of them.
__device__ __forceinline__ int scan(int v, int *all) {
    const int lane = threadIdx.x & 31;
    int upto = v;
#pragma unroll
    for (int x = 1; x < 32; x <<= 1) {
        const int u = __shfl_up_sync(0xFFFFFFFFu, upto, x);
        if (lane >= x) upto += u;
    }
    *all = __shfl_sync(0xFFFFFFFFu, upto, 31);
    return upto - v;
}

// KEYS items a thread, or (0) as many as it takes, which are read again by each
// pass.  blocks: of a cluster, up to 8.
template <int THREADS, int KEYS>
__global__ void __launch_bounds__(THREADS, THREADS == 512 ? 2 : 1)
select_kernel(const Job j, int blocks) {
    constexpr int WARPS = THREADS / 32, EACH = kBins / THREADS;
    constexpr bool SHARED = THREADS == 1024;                  // rows of several blocks
    __shared__ __align__(16) int hist[3][kBins];
    __shared__ int sums[WARPS], above[WARPS], equal[WARPS];
    __shared__ __align__(8) int total[2];
    __shared__ int found_bin, found_need, found_in, found_most, listed, few;
    __shared__ uint32_t list[kListed], few_keys[kFew];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    for (int i = tid; i < 3 * kBins / 4; i += THREADS)
        reinterpret_cast<int4 *>(hist)[i] = make_int4(0, 0, 0, 0);
    if (tid == 0) listed = few = 0;
    begin_after_previous();
    const bool shared = SHARED && blocks > 1;
    const int rank = shared ? cluster_rank() : 0;
    const unsigned row = shared ? blockIdx.x / blocks : blockIdx.x;
    const int b = row / j.heads, n = items_of(j, b);
    int32_t *out = j.index + (long long)row * j.count;
    if (rank == 0 && tid == 0 && row == (unsigned)b * j.heads) j.counts[b] = min(n, j.count);
    if (n <= j.count) {                                       // all of them, in every block
        for (int i = rank * THREADS + tid; i < n; i += blocks * THREADS) out[i] = i;
        return;
    }
    // a block, and a warp of it, has neighbouring items: 32 a round
    const int rounds =
        KEYS > 0 ? KEYS : (int)((((long long)n + blocks - 1) / blocks + THREADS - 1) / THREADS);
    const int start = (rank * WARPS + warp) * 32 * rounds + lane;
    const float *in = j.scores + (long long)row * j.columns;
    const auto key_at = [&](int i, float v) -> uint32_t {
        return i >= n ? 0u : i < j.first || i >= n - j.last ? kAlways : key_of(v);
    };
    // (all of a warp's items have scores that count)
    const bool inner = start - lane >= j.first && start - lane + 32 * rounds <= n - j.last;
    uint32_t keys[KEYS > 0 ? KEYS : 1];
    if constexpr (KEYS > 0) {
        float v[KEYS];                                        // all under way together
#pragma unroll
        for (int k = 0; k < KEYS; ++k) v[k] = in[min(start + 32 * k, n - 1)];
#pragma unroll
        for (int k = 0; k < KEYS; ++k) keys[k] = key_of(v[k]);
        if (!inner) {
#pragma unroll
            for (int k = 0; k < KEYS; ++k) {
                const int i = start + 32 * k;
                if (i < j.first || i >= n - j.last) keys[k] = kAlways;
                if (i >= n) keys[k] = 0u;                     // there is no item
            }
        }
    }
    // f(key) of each of the thread's items, all lanes of a warp together
    const auto each_key = [&](auto f) {
        if constexpr (KEYS > 0) {
#pragma unroll
            for (int k = 0; k < KEYS; ++k) f(keys[k], k);
        } else {
            for (int k = 0; k < rounds; ++k) {
                const int i = start + 32 * k;
                f(key_at(i, in[min(i, n - 1)]), k);
            }
        }
    };

    // ---- the count-th largest key, and how many equal to it are chosen
    constexpr int LEFT = kListed / (THREADS < 512 ? 512 : THREADS);
    uint32_t found = 0, mine_left[LEFT];                      // its upper digits
    int need = j.count, shift = 32, left = n;
    bool in_list = false;
    __syncthreads();
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
        const int bits = pass < 2 ? 11 : 10, top = shift;
        shift -= bits;
        int *h = hist[pass];
        const bool together = shared && !in_list;             // all blocks' keys
        const auto add = [&](uint32_t key, int n_same) {
            atomicAdd(&h[key >> shift & ((1u << bits) - 1)], n_same);
        };
        if (in_list) {
#pragma unroll
            for (int k = 0; k < LEFT; ++k)
                if (mine_left[k] != 0u && mine_left[k] >> top == found >> top) add(mine_left[k], 1);
        } else {
            // (a warp whose keys all fall into one bin, as where all scores are
            // equal, does not add them one after another)
            bool alike = false;
            if constexpr (KEYS > 0) {
                const uint32_t one = __shfl_sync(0xFFFFFFFFu, keys[0], 0);
                alike = __all_sync(0xFFFFFFFFu, (keys[0] ^ one) >> shift == 0u);
                if (alike) {                                  // seldom by chance
                    uint32_t other = 0u;
                    each_key([&](uint32_t key, int) { other |= key ^ one; });
                    alike = __all_sync(0xFFFFFFFFu, other >> shift == 0u);
                }
                if (alike && lane == 0 && one != 0u &&
                    (top == 32 || one >> top == found >> top))
                    add(one, 32 * KEYS);
            }
            if (alike) {
            } else if (top == 32 && inner) {
                each_key([&](uint32_t key, int) { add(key, 1); });
            } else if (top == 32) {
                each_key([&](uint32_t key, int) {
                    if (key != 0u) add(key, 1);
                });
            } else {
                each_key([&](uint32_t key, int) {
                    if (key >> top == found >> top) add(key, 1);
                });
            }
        }
        if (together)
            cluster_sync();
        else
            __syncthreads();
        // thread t: bins from the top, EACH of them
        const int bin0 = kBins - (tid + 1) * EACH;
        int in_bin[EACH], most[EACH], mine = 0, whole;        // most: of any block
        if constexpr (SHARED) {
            static_assert(!SHARED || EACH == 2, "a pair of bins a thread");
            const int2 own = *reinterpret_cast<const int2 *>(&h[bin0]);
            in_bin[0] = most[0] = own.x, in_bin[1] = most[1] = own.y;
            if (together) {
                int2 part[7];                                 // of the blocks after this one
#pragma unroll
                for (int r = 1; r < 8; ++r)
                    if (r < blocks) {
                        const int other = rank + r;
                        part[r - 1] = cluster_load(&h[bin0], other < blocks ? other : other - blocks);
                    }
#pragma unroll
                for (int r = 1; r < 8; ++r)
                    if (r < blocks) {
                        in_bin[0] += part[r - 1].x, in_bin[1] += part[r - 1].y;
                        most[0] = max(most[0], part[r - 1].x);
                        most[1] = max(most[1], part[r - 1].y);
                    }
            }
        } else {
#pragma unroll
            for (int x = 0; x < EACH; x += 4) {
                const int4 v = *reinterpret_cast<const int4 *>(&h[bin0 + x]);
                in_bin[x] = v.x, in_bin[x + 1] = v.y, in_bin[x + 2] = v.z, in_bin[x + 3] = v.w;
            }
#pragma unroll
            for (int x = 0; x < EACH; ++x) most[x] = in_bin[x];
        }
#pragma unroll
        for (int x = 0; x < EACH; ++x) mine += in_bin[x];
        int before = scan(mine, &whole);
        if (lane == 0) sums[warp] = whole;
        __syncthreads();
        int all;
        const int below = scan(lane < WARPS ? sums[lane] : 0, &all);
        before += __shfl_sync(0xFFFFFFFFu, below, warp);
        if (before < need && need <= before + mine) {
#pragma unroll
            for (int x = EACH - 1; x >= 0; --x) {
                if (before < need && need <= before + in_bin[x]) {
                    found_bin = bin0 + x, found_need = need - before;
                    found_in = in_bin[x], found_most = most[x];
                }
                before += in_bin[x];
            }
        }
        __syncthreads();
        found |= (uint32_t)found_bin << shift;
        need = found_need, left = found_in;
        if (need == left || pass == 2) break;                 // every one of the bin
        if (!in_list && left <= LEFT * THREADS && found_most <= kListed) {
            in_list = true;
            int own = 0, whole_warp;
            each_key([&](uint32_t key, int) { own += key >> shift == found >> shift; });
            own = scan(own, &whole_warp);
            int at = 0;
            if (lane == 0 && whole_warp) at = atomicAdd(&listed, whole_warp);
            at = __shfl_sync(0xFFFFFFFFu, at, 0) + own;
            if (whole_warp)
                each_key([&](uint32_t key, int) {
                    if (key >> shift == found >> shift) list[at++] = key;
                });
            if (shared)
                cluster_sync();
            else
                __syncthreads();
            // the keys of all blocks, one block's after another's
            int end[7];
            if (shared) {
                int all_of, upto = lane < blocks ? cluster_load1(&listed, lane) : 0;
                upto += scan(upto, &all_of);                  // lane r: of blocks 0 .. r
#pragma unroll
                for (int x = 0; x < 7; ++x) end[x] = __shfl_sync(0xFFFFFFFFu, upto, x);
            }
#pragma unroll
            for (int k = 0; k < LEFT; ++k) {
                const int i = tid + k * THREADS;
                mine_left[k] = 0u;
                if (i >= left) continue;
                if (!shared) {
                    mine_left[k] = list[i];
                    continue;
                }
                int r = 0, from = 0;
#pragma unroll
                for (int x = 0; x < 7; ++x)
                    if (i >= end[x]) r = x + 1, from = end[x];
                mine_left[k] =
                    (uint32_t)cluster_load1(reinterpret_cast<const int *>(&list[i - from]), r);
            }
        }
        if (in_list && left <= kFew) {
            // each of the few counts the larger and the equal ones
#pragma unroll
            for (int k = 0; k < LEFT; ++k)
                if (mine_left[k] != 0u && mine_left[k] >> shift == found >> shift)
                    few_keys[atomicAdd(&few, 1)] = mine_left[k];
            __syncthreads();
            if (tid < left) {
                const uint32_t key = few_keys[tid];
                int larger = 0, same = 0;
#pragma unroll 4
                for (int x = 0; x < left; ++x) {
                    const uint32_t other = few_keys[x];
                    larger += other > key, same += other == key;
                }
                if (larger < need && need <= larger + same)
                    found_bin = (int)key, found_need = need - larger, found_in = same;
            }
            __syncthreads();
            found = (uint32_t)found_bin, need = found_need, left = found_in;
            break;
        }
    }
    if (need == left) --found, need = 0;                      // (found is no score's 0)

    // ---- how many are above it, or equal to it, before a warp's first item
    int n_above = 0, n_equal = 0;
    each_key([&](uint32_t key, int) { n_above += key > found; });
    n_above = __reduce_add_sync(0xFFFFFFFFu, n_above);
    if (need > 0) {
        each_key([&](uint32_t key, int) { n_equal += key == found; });
        n_equal = __reduce_add_sync(0xFFFFFFFFu, n_equal);
    }
    if (lane == 0) above[warp] = n_above, equal[warp] = n_equal;
    __syncthreads();
    int all_above, all_equal;
    const int more_below = scan(lane < WARPS ? above[lane] : 0, &all_above);
    const int same_below = scan(lane < WARPS ? equal[lane] : 0, &all_equal);
    int at_above = __shfl_sync(0xFFFFFFFFu, more_below, warp);
    int at_equal = __shfl_sync(0xFFFFFFFFu, same_below, warp);
    if (shared) {
        if (tid == 0) total[0] = all_above, total[1] = all_equal;
        cluster_sync();
        if (rank > 0) {
            // lane r: block r's
            const int2 v = lane < rank ? cluster_load(total, lane) : make_int2(0, 0);
            int sum_above, sum_equal;
            scan(v.x, &sum_above), scan(v.y, &sum_equal);
            at_above += sum_above, at_equal += sum_equal;
        }
        // (no block ends while another reads its shared memory)
        asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    }
    const unsigned lower = (1u << lane) - 1;
    if (n_equal == 0 || need <= at_equal) {                   // no item here is chosen for equality
        int32_t *to = out + min(at_equal, need);
        each_key([&](uint32_t key, int k) {
            const unsigned more = __ballot_sync(0xFFFFFFFFu, key > found);
            if (key > found) to[at_above + __popc(more & lower)] = start + 32 * k;
            at_above += __popc(more);
        });
    } else {
        each_key([&](uint32_t key, int k) {
            const unsigned more = __ballot_sync(0xFFFFFFFFu, key > found);
            const unsigned same = __ballot_sync(0xFFFFFFFFu, key == found);
            const int e = at_equal + __popc(same & lower);
            if (key > found || (key == found && e < need))
                out[at_above + __popc(more & lower) + min(e, need)] = start + 32 * k;
            at_above += __popc(more), at_equal += __popc(same);
        });
    }
    if (shared) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

template <int THREADS>
cudaLaunchConfig_t config(long long rows, int blocks, cudaLaunchAttribute *attr,
                          cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(rows * blocks));
    cfg.blockDim = dim3(THREADS);
    cfg.stream = stream;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = blocks;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cfg;
}

template <int THREADS, int KEYS>
cudaError_t launch(const Job &job, long long rows, int blocks, cudaStream_t stream) {
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t cfg = config<THREADS>(rows, blocks, attr, stream);
    if (blocks == 1) cfg.attrs = attr + 1, cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, select_kernel<THREADS, KEYS>, job, blocks);
}

// Clusters of `blocks` blocks that the device runs at a time (0: it does not say),
// kept by device.
int clusters_held(int blocks) {
    static std::atomic<int> kept[64][9] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    if (dev >= 0 && dev < 64) {
        const int v = kept[dev][blocks].load(std::memory_order_relaxed);
        if (v > 0) return v;
    }
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t cfg = config<1024>(1, blocks, attr, nullptr);
    cfg.numAttrs = 1;
    int v = 0;
    if (cudaOccupancyMaxActiveClusters(&v, select_kernel<1024, 32>, &cfg) != cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    if (dev >= 0 && dev < 64) kept[dev][blocks].store(v, std::memory_order_relaxed);
    return v;
}

}  // namespace

cudaError_t launch_select(const float *scores, int seqs, int heads, int columns,
                          const int32_t *lens, int unit, int first, int last, int count,
                          int32_t *index, int32_t *counts, int num_sms, cudaStream_t stream) {
    const Job job = {scores, lens, index, counts, heads, columns, unit, first, last, count};
    const long long rows = (long long)seqs * heads;
    if (columns <= 256 * 2) return launch<256, 2>(job, rows, 1, stream);
    if (columns <= 256 * 8) return launch<256, 8>(job, rows, 1, stream);
    if (columns <= 512 * 8) return launch<512, 8>(job, rows, 1, stream);
    if (columns <= 512 * 16 && rows > num_sms) return launch<512, 16>(job, rows, 1, stream);
    // the largest cluster of which the device runs all rows' at a time, as long as a
    // block has 4096 items; or the smallest one that keeps a row in registers
    int blocks = 8;
    while (blocks > 1 && (columns <= 4096 * (blocks - 1) || rows > clusters_held(blocks))) --blocks;
    while (blocks < 8 && columns > 32 * 1024 * blocks) ++blocks;
    const int each = (columns + blocks - 1) / blocks;
    return each <= 1024 * 8    ? launch<1024, 8>(job, rows, blocks, stream)
           : each <= 1024 * 16 ? launch<1024, 16>(job, rows, blocks, stream)
           : each <= 1024 * 24 ? launch<1024, 24>(job, rows, blocks, stream)
           : each <= 1024 * 32 ? launch<1024, 32>(job, rows, blocks, stream)
                               : launch<1024, 0>(job, rows, blocks, stream);
}

}  // namespace w4
