// One step's block tables, slot mapping and sequence starts, built on the GPU from
// the requests' lengths and a stack of free blocks; and the return of finished
// sequences' blocks to that stack.
//
// What is computed (include/pa.h): with len_s tokens held and cnt_s to append,
//   new_s   = ceil((len_s + cnt_s) / 16) - ceil(len_s / 16)
//   start_s = sum_{s' < s} cnt_s',  pop_s = sum_{s' < s} new_s'
//   table[s][ceil(len_s / 16) + j] = free[num_free - 1 - (pop_s + j)]   (j < new_s)
//   slot[start_s + i] = table[s][(len_s + i) / 16] * 16 + (len_s + i) % 16
// i.e. the host block manager's append_step for sequences that share no block
// (blocks popped from a LIFO stack, sequence by sequence).
//
// What bounds it: latency.  A step of 256 sequences touches 6 KB, an admission of
// 69 thousand prompt tokens 0.6 MB (0.1 us of HBM time), so everything is one launch:
// every CTA reads all lengths and scans them itself (in shared memory; two 32-bit
// scans with saturating sums, which stay associative), and the CTAs of one cluster
// share the writing.  The cluster barrier between reading and writing is what lets
// the new lengths and the new stack height go where the old ones are (a captured
// graph replays the step in place).  Few slots: one CTA, no cluster.  Measured in a graph: 256
// sequences with a token each 4.2 us; 64 prompts with 4, 33, 66, 260 thousand slots 4.6, 6.0, 8.0,
// 20.4 us with a cluster of 8 CTAs, 4.7, 5.2, 6.1, 12.0 with 16 (16 thousand: 4.9 with either), so
// calls with more than 16 thousand take 16, a size above the portable one, where the device can
// hold it.
#include <atomic>

#include <cooperative_groups.h>

#include "pa_common.cuh"
#include "pa_launch.h"
#include "pa_step.h"

namespace pa {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kPlanThreads = 1024;
constexpr int kPlanCluster = 8;       // portable cluster size
constexpr int kPlanClusterBig = 16;   // where the device can hold one
constexpr int64_t kBigWork = 16384;   // slots or table entries: one for each of their threads
constexpr uint32_t kSat = 1u << 30;   // sums at or above it are "too many"

__device__ __forceinline__ uint32_t sat_add(uint32_t a, uint32_t b) { return min(a + b, kSat); }

__device__ __forceinline__ int blocks_of(int tokens) { return tokens / kBlockSize + (tokens % kBlockSize != 0); }

// Exclusive scans of two values per thread over the CTA; totals in every thread.
__device__ __forceinline__ void scan2(uint32_t &a, uint32_t &b, uint32_t &ta, uint32_t &tb, uint2 *warp_sums) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint32_t ia = a, ib = b;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t ya = __shfl_up_sync(kFull, ia, o), yb = __shfl_up_sync(kFull, ib, o);
        if (lane >= o) {
            ia = sat_add(ia, ya);
            ib = sat_add(ib, yb);
        }
    }
    uint32_t ea = __shfl_up_sync(kFull, ia, 1), eb = __shfl_up_sync(kFull, ib, 1);
    if (lane == 0) ea = eb = 0;
    if (lane == 31) warp_sums[warp] = make_uint2(ia, ib);
    __syncthreads();
    uint2 w = warp_sums[lane];  // kPlanThreads / 32 = 32 warps
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t ya = __shfl_up_sync(kFull, w.x, o), yb = __shfl_up_sync(kFull, w.y, o);
        if (lane >= o) {
            w.x = sat_add(w.x, ya);
            w.y = sat_add(w.y, yb);
        }
    }
    ta = __shfl_sync(kFull, w.x, 31);
    tb = __shfl_sync(kFull, w.y, 31);
    const uint32_t oa = __shfl_sync(kFull, w.x, warp > 0 ? warp - 1 : 0);
    const uint32_t ob = __shfl_sync(kFull, w.y, warp > 0 ? warp - 1 : 0);
    a = warp > 0 ? sat_add(oa, ea) : ea;
    b = warp > 0 ? sat_add(ob, eb) : eb;
}

// Largest s in [0, n) with cum[s] <= v (cum[0] = 0, cum[n] > v).
__device__ __forceinline__ int find_seq(const int *cum, int n, int v) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cum[mid] <= v) lo = mid; else hi = mid;
    }
    return lo;
}

template <bool kCluster>
__device__ __forceinline__ void reads_done() {
    if constexpr (kCluster) cooperative_groups::this_cluster().sync();
    else __syncthreads();
}

// kRelease false: the step plan; true: give the blocks of the sequences with
// counts[s] != 0 back to the stack (table entries become -1, lengths 0).
template <bool kRelease, bool kCluster>
__global__ void __launch_bounds__(kPlanThreads, 1) step_plan_kernel(const StepPlan p) {
    extern __shared__ int smem[];
    __shared__ uint2 warp_sums[kPlanThreads / 32];
    __shared__ int any_bad;
    const int S = p.num_seqs;
    int *starts = smem, *pops = smem + S + 1, *held = smem + 2 * (S + 1);
    if (threadIdx.x == 0) any_bad = 0;
    const int per = (S + kPlanThreads - 1) / kPlanThreads;
    const int beg = min(S, (int)threadIdx.x * per), end = min(S, beg + per);
    const int nfree = *p.num_free;
    uint32_t a = 0, b = 0;
    bool bad = nfree < 0 || nfree > p.free_capacity;
    // this thread's sums; lengths and block counts kept for the second pass
    for (int s = beg; s < end; ++s) {
        const int len = p.lens[s], cnt = p.counts[s];
        bool wrong = len < 0 || (int64_t)len > (int64_t)p.max_blocks * kBlockSize;
        uint32_t na = 0, nb = 0;
        if constexpr (kRelease) {
            nb = !wrong && cnt != 0 ? (uint32_t)blocks_of(len) : 0u;
        } else {
            wrong = wrong || cnt < 0 || (int64_t)len + cnt > min((int64_t)p.max_blocks * kBlockSize, (int64_t)INT32_MAX);
            if (!wrong) {
                na = min((uint32_t)cnt, kSat);
                nb = min((uint32_t)(blocks_of(len + cnt) - blocks_of(len)), kSat);
            }
        }
        bad |= wrong;
        held[s] = len;
        starts[s] = (int)na;
        pops[s] = (int)nb;
        a = sat_add(a, na);
        b = sat_add(b, nb);
    }
    uint32_t total = 0, blocks = 0;
    __syncthreads();  // any_bad is zero
    if (bad) any_bad = 1;
    scan2(a, b, total, blocks, warp_sums);
    for (int s = beg; s < end; ++s) {
        const uint32_t na = (uint32_t)starts[s], nb = (uint32_t)pops[s];
        starts[s] = (int)a;
        pops[s] = (int)b;
        a = sat_add(a, na);
        b = sat_add(b, nb);
    }
    if (threadIdx.x == 0) {
        starts[S] = (int)total;
        pops[S] = (int)blocks;
    }
    reads_done<kCluster>();  // every CTA has read the lengths and the stack height
    bool ok = any_bad == 0 && blocks < kSat;
    if constexpr (kRelease) ok = ok && (int64_t)nfree + (int)blocks <= (int64_t)p.free_capacity;
    else ok = ok && total < kSat && (int)total <= p.slot_capacity && (int)blocks <= nfree;
    const int tid = (int)(blockIdx.x * kPlanThreads + threadIdx.x), nthreads = (int)(gridDim.x * kPlanThreads);
    if (tid == 0) {
        if (!ok) flag_error(p.err, PA_DEVERR_PLAN);
        *p.new_num_free = !ok ? nfree : kRelease ? nfree + (int)blocks : nfree - (int)blocks;
    }
    if constexpr (kRelease) {
        for (int s = tid; s < S; s += nthreads) p.new_lens[s] = ok && p.counts[s] != 0 ? 0 : held[s];
        if (!ok) return;
        for (int j = tid; j < (int)blocks; j += nthreads) {
            const int s = find_seq(pops, S, j);
            int32_t *entry = p.tables + (int64_t)s * p.max_blocks + (j - pops[s]);
            const int32_t id = *entry;
            if (id < 0) flag_error(p.err, PA_DEVERR_BLOCK_ID);
            p.free_out[nfree + j] = id;
            *entry = -1;
        }
        return;
    }
    if (!ok) total = blocks = 0;
    for (int s = tid; s <= S; s += nthreads) {
        p.starts[s] = ok ? starts[s] : 0;
        if (s < S) p.new_lens[s] = held[s] + (ok ? starts[s + 1] - starts[s] : 0);
    }
    for (int j = tid; j < (int)blocks; j += nthreads) {
        const int s = find_seq(pops, S, j);
        p.tables[(int64_t)s * p.max_blocks + blocks_of(held[s]) + (j - pops[s])] = p.free_blocks[nfree - 1 - j];
    }
    // The slots, two neighbours per thread (one 16-byte store where the buffer allows
    // it).  Ids of blocks popped in this step come from the stack itself, so no thread
    // waits for a table entry written by another.
    auto slot_of = [&](int i, int s) -> long long {
        const int at = held[s] + (i - starts[s]);
        const int lb = at / kBlockSize, first = blocks_of(held[s]);
        const int id = lb >= first ? p.free_blocks[nfree - 1 - (pops[s] + lb - first)]
                                   : p.tables[(int64_t)s * p.max_blocks + lb];
        if (id < 0) {
            flag_error(p.err, PA_DEVERR_BLOCK_ID);
            return -1;
        }
        return (long long)id * kBlockSize + at % kBlockSize;
    };
    const bool pairs = (reinterpret_cast<uintptr_t>(p.slots) & 15u) == 0;
    for (int i = 2 * tid; i < p.slot_capacity; i += 2 * nthreads) {
        long long v0 = -1, v1 = -1;
        if (i < (int)total) {
            int s = find_seq(starts, S, i);
            v0 = slot_of(i, s);
            if (i + 1 < (int)total) {
                while (starts[s + 1] <= i + 1) ++s;
                v1 = slot_of(i + 1, s);
            }
        }
        if (pairs && i + 1 < p.slot_capacity) {
            *reinterpret_cast<longlong2 *>(p.slots + i) = make_longlong2(v0, v1);
        } else {
            p.slots[i] = v0;
            if (i + 1 < p.slot_capacity) p.slots[i + 1] = v1;
        }
    }
}

// Whether the device can hold a cluster of kPlanClusterBig CTAs of this kernel with its most
// shared memory (above the portable size, so it is asked; once per device).
template <bool kRelease>
bool big_cluster() {
    constexpr int kDevices = 64;
    static std::atomic<int> known[kDevices];   // 0: not asked, 1: no, 2: yes
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kDevices) return false;
    int k = known[dev].load(std::memory_order_relaxed);
    if (k == 0) {
        const auto kern = step_plan_kernel<kRelease, true>;
        const int smem = 3 * (kMaxPlanSeqs + 1) * 4;
        int clusters = 0;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(kPlanClusterBig);
        cfg.blockDim = dim3(kPlanThreads);
        cfg.dynamicSmemBytes = (size_t)smem;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = kPlanClusterBig;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        const bool yes = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess &&
                         cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) == cudaSuccess &&
                         cudaOccupancyMaxActiveClusters(&clusters, kern, &cfg) == cudaSuccess && clusters > 0;
        if (!yes) (void)cudaGetLastError();
        k = yes ? 2 : 1;
        known[dev].store(k, std::memory_order_relaxed);
    }
    return k == 2;
}

template <bool kRelease, bool kCluster>
cudaError_t launch(const StepPlan &p, int ctas, cudaStream_t stream) {
    const size_t smem = (size_t)(3 * (p.num_seqs + 1)) * 4;
    // The 48 KB that a launch may ask for anyway hold the kernel's static arrays too (272 bytes).
    if (smem > 47 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(step_plan_kernel<kRelease, kCluster>,
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   3 * (kMaxPlanSeqs + 1) * 4);
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(kPlanThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)ctas;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, step_plan_kernel<kRelease, kCluster>, p);
}

}  // namespace

cudaError_t launch_step_plan(const StepPlan &p, bool release, cudaStream_t stream) {
    // What the writers share out: slots (plan) or at most every table entry (release).
    const int64_t work = release ? (int64_t)p.num_seqs * p.max_blocks : (int64_t)p.slot_capacity;
    if (work <= 2 * kPlanThreads)
        return release ? launch<true, false>(p, 1, stream) : launch<false, false>(p, 1, stream);
    if (release) return launch<true, true>(p, work > kBigWork && big_cluster<true>() ? kPlanClusterBig : kPlanCluster, stream);
    return launch<false, true>(p, work > kBigWork && big_cluster<false>() ? kPlanClusterBig : kPlanCluster, stream);
}

}  // namespace pa
