// Causal attention over whole prompts packed without padding, grouped heads, on
// 5th-generation tensor cores.
//
// What is computed (include/pa.h): sequence s owns rows [starts[s], starts[s + 1]) of
// query, key and value; for its row i and query head hq of kv head h = hq / g
//   out_i = sum_{j <= i} softmax_j(scale * <q_i, k_j>) v_j.
//
// Rows: the g query heads of one kv head are packed into the rows of a tile (row =
// token * g + head), so a K/V tile in shared memory serves all of them.  A job is two
// such 128-row tiles of one (sequence, kv head), streams 0 and 1, that share every K/V
// tile of 128 keys (stream 0 may need one tile less):
//   S_t = Q_t K^T   tcgen05.mma, M = N = 128 -> tensor memory
//   P_t = 2^(S_t scale log2(e) - m_t), one row per thread, written back as bf16 over S_t
//   O_t += P_t V    tcgen05.mma with A = P_t read from tensor memory, B = V (MN-major)
// One stream's softmax runs while the tensor core works for the other.  The reference
// point m_t moves (and O_t is rescaled) only when a row's maximum rises by more than
// 2^8; sums are fp32, P is rounded to bf16 once (2^-8, as the operand type asks).
//
// What bounds it: per 128 x 128 tile the tensor core needs 512 clocks per product
// (d = 128), and the special-function units 1024 clocks for the 16,384 exponentials:
// as much as both products.  So a share of the exponentials (kPoly of 16 in a row) is
// computed on the FMA units instead: 2^x = 2^n 2^f with n = rint(x) and a cubic in f (least
// relative maximum error, fitted numerically: 1.0e-4, a fortieth of P's own rounding;
// its constant is exactly 1, so that a masked score still gives exactly 0).
//
// Work: plan_kernel lists the (sequence, row pair) jobs, longest first, and zeroes the
// counter from which the persistent CTAs draw (job, kv head) in that order; so the
// lengths are read on the device only and a captured graph follows them.
// Warp roles: 0-3 softmax of stream 0, 4-7 of stream 1 (tensor-memory lanes 32 (w % 4) ..),
// 8 issues the MMAs and owns the tensor memory, 9 draws jobs and loads Q and K, 10 loads
// V (11 only completes the warpgroup).  K and V have rings of their own.
// Masked places: a key behind a row is left out by position, so its score may be
// anything.  Its value meets P = 0 in the tensor core, where an infinity or a NaN would
// survive: the loader zeroes the rows of the last tile that no row of the job sees, and a
// row that comes out not finite while a value masked for it is not finite is
// computed again without tensor cores (redo_row).
// Every wait is bounded; an abort drains the copies and MMAs in flight and frees the
// tensor memory.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <climits>
#include <cstring>
#include <mutex>

#include "pa_common.cuh"
#include "pa_launch.h"
#include "pa_step.h"
#include "tcgen05.cuh"

namespace pa {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kTile = 128;           // rows of a query tile, keys of a K/V tile
constexpr int kThreads = 12 * 32;
constexpr int kMmaWarp = 8, kLoadWarp = 9, kVLoadWarp = 10;
// Registers: the launch gives 384 x 168; the softmax warpgroups take 200 (a row of S), the
// other one 96: 256 x 200 + 128 x 96 <= 384 x 168.
constexpr int kRegsSoftmax = 200, kRegsOther = 96;
static_assert(256 * kRegsSoftmax + 128 * kRegsOther <= kThreads * 168, "register split over the launch's total");
constexpr uint32_t kTmemCols = 512;  // S0, S1, O0, O1, 128 columns apart
constexpr float kRescaleLog2 = 8.f;

constexpr int kKStages = 2, kVStages = 2;
constexpr uint32_t kHalf = kTile * 128;  // 64 columns of a 128-row tile

enum Bar {
    kBarKFull = 0,                       // [kKStages] K stage landed
    kBarKEmpty = kBarKFull + kKStages,   // [kKStages] its products are done
    kBarVFull = kBarKEmpty + kKStages,   // [kVStages] V stage ready
    kBarVEmpty = kBarVFull + kVStages,   // [kVStages]
    kBarVLand = kBarVEmpty + kVStages,   // a last V tile landed (its unseen rows are zeroed next)
    kBarQFull = kBarVLand + 1,           // [2] Q_t landed
    kBarQEmpty = kBarQFull + 2,          // the job's last QKs are done
    kBarSFull = kBarQEmpty + 1,          // [2] S_t written
    kBarPFull = kBarSFull + 2,           // [2] P_t written (128 threads)
    kBarOFull = kBarPFull + 2,           // [2] the job's last PV_t is done
    kBarOFree = kBarOFull + 2,           // [2] O_t has been read (128 threads)
    kBarIdle = kBarOFree + 2,
    kNumBars = kBarIdle + 1
};

template <int D>
struct Smem {
    static constexpr int kHalves = D / 64;
    static constexpr uint32_t kTileBytes = kHalves * kHalf;
    static constexpr uint32_t kQ = 0;
    static constexpr uint32_t kK = 2 * kTileBytes;
    static constexpr uint32_t kV = kK + kKStages * kTileBytes;
    static constexpr uint32_t kBars = kV + kVStages * kTileBytes;
    static constexpr uint32_t kMisc = kBars + kNumBars * 8;              // tensor-memory address, abort flag
    static constexpr uint32_t kJobs = (kMisc + 8 + 15) / 16 * 16;        // int4 [8] records, int [8] tags
    static constexpr size_t kBytes = kJobs + 8 * 16 + 8 * 4 + 1024;      // slack to align the base
    static_assert(kTileBytes % 1024 == 0 && kBars % 8 == 0, "swizzled tiles 1024-byte aligned, barriers 8");
    static_assert(kBytes <= 232448, "shared memory of an sm_100 CTA");
};

struct Params {
    CUtensorMap qmap, kmap, vmap;
    const unsigned char *q, *k, *v;
    int64_t q_stride, k_stride, v_stride;   // bytes between tokens
    unsigned char *out;
    int32_t *err;
    const int4 *jobs;                       // (first row, tokens, row pair, 0), longest first
    int32_t *meta;                          // [0] jobs, [1] work counter
    int32_t num_q_heads, num_kv_heads;
    float scale_log2;
    unsigned long long wait_ns;
};

struct PlanParams {
    const int32_t *starts;
    int4 *jobs;
    int32_t *meta;
    int32_t *err;
    int32_t num_seqs, num_tokens, max_len, pair_tokens, max_jobs;
};

// ---------------------------------------------------------------- the job list
constexpr int kPlanThreads = 1024;
constexpr int kBuckets = 256;

__device__ __forceinline__ int block_scan(int v, int *total, int *warp_sums) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(kFull, incl, o);
        if (lane >= o) incl += y;
    }
    if (lane == 31) warp_sums[warp] = incl;
    __syncthreads();
    int w = warp_sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(kFull, w, o);
        if (lane >= o) w += y;
    }
    *total = __shfl_sync(kFull, w, 31);
    const int off = __shfl_sync(kFull, w, warp > 0 ? warp - 1 : 0);
    __syncthreads();
    return (warp > 0 ? off : 0) + incl - v;
}

// Lists every sequence's row pairs in buckets of falling key count (a counting sort; the
// order inside a bucket does not matter) and zeroes the work counter.
__global__ void __launch_bounds__(kPlanThreads, 1) packed_plan_kernel(const PlanParams p) {
    extern __shared__ int cum[];          // [num_seqs + 1] pairs before each sequence
    __shared__ int warp_sums[32], hist[kBuckets];
    grid_dep_launch();
    const int S = p.num_seqs;
    const int per = (S + kPlanThreads - 1) / kPlanThreads;
    const int beg = min(S, (int)threadIdx.x * per), end = min(S, beg + per);
    for (int i = threadIdx.x; i < kBuckets; i += kPlanThreads) hist[i] = 0;
    int sum = 0;
    bool bad = false;
    for (int s = beg; s < end; ++s) {
        const int a = __ldg(p.starts + s), b = __ldg(p.starts + s + 1);
        int pairs = 0;
        // rows outside the tensors or a sequence longer than announced: skipped and flagged
        if (a < 0 || b < a || b > p.num_tokens || b - a > p.max_len) bad = true;
        else pairs = (b - a + p.pair_tokens - 1) / p.pair_tokens;
        cum[s] = pairs;
        sum += pairs;
    }
    int total;
    int run = block_scan(sum, &total, warp_sums);
    for (int s = beg; s < end; ++s) {
        const int pairs = cum[s];
        cum[s] = run;
        run += pairs;
    }
    if (threadIdx.x == 0) cum[S] = total;
    // overlapping sequences could list more pairs than the list holds
    const bool fits = total <= p.max_jobs;
    if (bad || (!fits && threadIdx.x == 0)) flag_error(p.err, PA_DEVERR_CHUNK);
    __syncthreads();
    if (!fits) total = 0;
    const int most = (p.max_len + p.pair_tokens - 1) / p.pair_tokens;
    auto bucket_of = [&](int jp) { return kBuckets - 1 - (int)((int64_t)jp * kBuckets / max(most, 1)); };
    auto seq_of = [&](int e) {
        int lo = 0, hi = S;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (cum[mid] <= e) lo = mid; else hi = mid;
        }
        return lo;
    };
    for (int e = threadIdx.x; e < total; e += kPlanThreads) atomicAdd(&hist[bucket_of(e - cum[seq_of(e)])], 1);
    __syncthreads();
    int dummy;
    const int mine = threadIdx.x < kBuckets ? hist[threadIdx.x] : 0;
    const int before = block_scan(mine, &dummy, warp_sums);
    if (threadIdx.x < kBuckets) hist[threadIdx.x] = before;
    __syncthreads();
    for (int e = threadIdx.x; e < total; e += kPlanThreads) {
        const int s = seq_of(e), jp = e - cum[s];
        const int a = __ldg(p.starts + s), b = __ldg(p.starts + s + 1);
        p.jobs[atomicAdd(&hist[bucket_of(jp)], 1)] = make_int4(a, b - a, jp, 0);
    }
    if (threadIdx.x == 0) {
        p.meta[0] = total;
        p.meta[1] = 0;
    }
}

// ---------------------------------------------------------------- the attention
__device__ __forceinline__ bool wait_bar(uint64_t *bar, uint32_t parity, volatile int *abort, const Params &p) {
    return mbar_wait_bounded(bar, parity, abort, p.err, p.wait_ns);
}

struct Job {
    int row0;        // the sequence's first row
    int i0;          // first token of tile 0 within the sequence
    int h;
    int nrows[2];    // packed rows in use
    int ntiles[2];   // key tiles of each stream (0: the stream has no rows)
    int nkeys;       // keys the job's last row sees
};

template <int G>
__device__ __forceinline__ void make_job(int4 rec, Job &jb) {
    constexpr int kTok = kTile / G;   // tokens of a tile
    const int rows = rec.y * G - rec.z * 2 * kTile;
    jb.row0 = rec.x;
    jb.i0 = rec.z * 2 * kTok;
    jb.h = rec.w;
    jb.nrows[0] = min(kTile, rows);
    jb.nrows[1] = min(kTile, max(0, rows - kTile));
    const int k0 = min(rec.y, jb.i0 + kTok), k1 = min(rec.y, jb.i0 + 2 * kTok);
    jb.ntiles[0] = (k0 + kTile - 1) / kTile;
    jb.ntiles[1] = jb.nrows[1] > 0 ? (k1 + kTile - 1) / kTile : 0;
    jb.nkeys = jb.nrows[1] > 0 ? k1 : k0;
}

__device__ __forceinline__ float fmax3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// 2^x for two values on the FMA units (x <= 128; at or below -127: 0).  See the head of
// the file for the method and its error.
__device__ __forceinline__ float2 exp2_fma(float2 x) {
    constexpr float kMagic = 12582912.f;  // 1.5 * 2^23: adding it rounds to an integer
    x.x = fmaxf(x.x, -127.f);
    x.y = fmaxf(x.y, -127.f);
    const float2 t = __fadd2_rn(x, make_float2(kMagic, kMagic));
    const float2 n = __fadd2_rn(t, make_float2(-kMagic, -kMagic));
    const float2 f = __fadd2_rn(x, make_float2(-n.x, -n.y));
    float2 r = __ffma2_rn(f, make_float2(0.05500893294811249f, 0.05500893294811249f),
                          make_float2(0.2422109693288803f, 0.2422109693288803f));
    r = __ffma2_rn(r, f, make_float2(0.6932829022407532f, 0.6932829022407532f));
    r = __ffma2_rn(r, f, make_float2(1.f, 1.f));
    // n sits in the low bits of t: shifted into the exponent field
    r.x = __int_as_float(__float_as_int(r.x) + (__float_as_int(t.x) << 23));
    r.y = __int_as_float(__float_as_int(r.y) + (__float_as_int(t.y) << 23));
    return r;
}

constexpr int kPoly = 4;  // of 16 pairs of a row chunk, computed on the FMA units

// One output row (token i of the sequence at row0, query head hq) without tensor cores, by
// a whole warp: only keys 0 .. i are read, so nothing masked can reach it.
template <int D>
__device__ __noinline__ void redo_row(const Params &p, int row0, int i, int hq, int h, int lane) {
    constexpr int E = D / 32;
    const __nv_bfloat16 *q = reinterpret_cast<const __nv_bfloat16 *>(p.q + (int64_t)(row0 + i) * p.q_stride) + hq * D;
    float qv[E], acc[E], m = -INFINITY, l = 0.f;
    for (int e = 0; e < E; ++e) {
        qv[e] = __bfloat162float(q[lane * E + e]);
        acc[e] = 0.f;
    }
    for (int j = 0; j <= i; ++j) {
        const __nv_bfloat16 *k = reinterpret_cast<const __nv_bfloat16 *>(p.k + (int64_t)(row0 + j) * p.k_stride) + h * D;
        const __nv_bfloat16 *v = reinterpret_cast<const __nv_bfloat16 *>(p.v + (int64_t)(row0 + j) * p.v_stride) + h * D;
        float s = 0.f;
        for (int e = 0; e < E; ++e) s = fmaf(qv[e], __bfloat162float(k[lane * E + e]), s);
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(kFull, s, o);
        s *= p.scale_log2;
        const float mn = fmaxf(m, s);
        const float base = mn == -INFINITY ? 0.f : mn;
        const float a = exp2f(m - base), w = exp2f(s - base);
        m = mn;
        l = l * a + w;
        for (int e = 0; e < E; ++e) acc[e] = acc[e] * a + w * __bfloat162float(v[lane * E + e]);
        if (l != l) break;  // a visible score is not a number: so is the row
    }
    __nv_bfloat16 *out = reinterpret_cast<__nv_bfloat16 *>(p.out) + ((int64_t)(row0 + i) * p.num_q_heads + hq) * D;
    for (int e = 0; e < E; ++e) out[lane * E + e] = __float2bfloat16_rn(l != l ? l : l > 0.f ? acc[e] / l : 0.f);
}

// Does any value behind token i, up to key `end` of the sequence, hold an infinity or a NaN?
template <int D>
__device__ __noinline__ bool masked_not_finite(const Params &p, int row0, int i, int end, int h, int lane) {
    bool found = false;
    for (int j = i + 1; j < end; ++j) {
        const __nv_bfloat16 *v = reinterpret_cast<const __nv_bfloat16 *>(p.v + (int64_t)(row0 + j) * p.v_stride) + h * D;
        for (int e = lane; e < D; e += 32) found |= !isfinite(__bfloat162float(v[e]));
    }
    return __any_sync(kFull, found);
}

template <int D, int G>
__global__ void __launch_bounds__(kThreads, 1) packed_prefill_kernel(const __grid_constant__ Params p) {
    using SM = Smem<D>;
    constexpr uint32_t kTileBytes = SM::kTileBytes;
    constexpr int kTok = kTile / G;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char *smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    const uint32_t sbase = smem_u32(smem);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + SM::kBars);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + SM::kMisc);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + SM::kMisc + 4);
    // The K loader draws the CTA's jobs and publishes job k in slot k & 7 (a record without
    // tokens ends the work); the other warps read it there.
    volatile int *job_rec = reinterpret_cast<volatile int *>(smem + SM::kJobs);
    volatile int *job_tag = job_rec + 32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < 8; ++i) job_tag[i] = -1;
        for (int i = 0; i < kNumBars; ++i) {
            const bool half = (i >= kBarPFull && i < kBarPFull + 2) || (i >= kBarOFree && i < kBarOFree + 2);
            mbar_init(&bars[i], half ? 128 : 1);
        }
        *abort_flag = 0;
        mbar_init_fence();
    }
    if (warp == kLoadWarp && lane == 0) {
        tc::prefetch_map(&p.qmap);
        tc::prefetch_map(&p.kmap);
        tc::prefetch_map(&p.vmap);
    }
    if (warp == kMmaWarp) tc::alloc(tmem_slot, kTmemCols);
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tmem = *tmem_slot;

    auto read_job = [&](int k, Job &jb) -> bool {   // one thread; false: no more jobs
        const unsigned long long t0 = global_ns();
        while (job_tag[k & 7] != k) {
            if (*abort_flag || global_ns() - t0 > p.wait_ns) {
                if (!*abort_flag) flag_error(p.err, PA_DEVERR_TIMEOUT);
                *abort_flag = 1;
                return false;
            }
        }
        __threadfence_block();
        const int4 rec = make_int4(job_rec[(k & 7) * 4], job_rec[(k & 7) * 4 + 1], job_rec[(k & 7) * 4 + 2],
                                   job_rec[(k & 7) * 4 + 3]);
        if (rec.y <= 0) return false;
        make_job<G>(rec, jb);
        return true;
    };
    auto read_job_warp = [&](int k, Job &jb) -> bool {
        int ok = 0;
        if (lane == 0) {
            const unsigned long long t0 = global_ns();
            ok = 1;
            while (job_tag[k & 7] != k) {
                if (*abort_flag || global_ns() - t0 > p.wait_ns) {
                    if (!*abort_flag) flag_error(p.err, PA_DEVERR_TIMEOUT);
                    *abort_flag = 1;
                    ok = 0;
                    break;
                }
            }
            __threadfence_block();
        }
        ok = __shfl_sync(kFull, ok, 0);
        if (!ok) return false;
        const int4 rec = make_int4(job_rec[(k & 7) * 4], job_rec[(k & 7) * 4 + 1], job_rec[(k & 7) * 4 + 2],
                                   job_rec[(k & 7) * 4 + 3]);
        if (rec.y <= 0) return false;
        make_job<G>(rec, jb);
        return true;
    };

    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
        if (warp == kLoadWarp) {
            // ---------------------------------------------- jobs, Q and K tiles
            if (lane == 0) {
                grid_dep_wait();   // the job list is complete
                const int njobs = __ldcg(p.meta) * p.num_kv_heads;
                int it = 0, nq[2] = {0, 0}, nj = 0;
                bool ok = true;
                int u = (int)blockIdx.x;
                for (int k = 0; ok; ++k) {
                    int4 rec = make_int4(0, 0, 0, 0);
                    if (u < njobs) {
                        rec = __ldcg(p.jobs + u / p.num_kv_heads);
                        rec.w = u % p.num_kv_heads;
                    }
                    job_rec[(k & 7) * 4] = rec.x;
                    job_rec[(k & 7) * 4 + 1] = rec.y;
                    job_rec[(k & 7) * 4 + 2] = rec.z;
                    job_rec[(k & 7) * 4 + 3] = rec.w;
                    __threadfence_block();
                    job_tag[k & 7] = k;
                    if (rec.y <= 0) break;
                    // the next job is drawn now and needed when this one's tiles are issued
                    u = (int)gridDim.x + atomicAdd(p.meta + 1, 1);
                    Job jb;
                    make_job<G>(rec, jb);
                    if (nj > 0) ok = wait_bar(&bars[kBarQEmpty], (nj - 1) & 1, abort_flag, p);
                    for (int t = 0; ok && t < 2; ++t) {
                        if (jb.ntiles[t] == 0) continue;
                        mbar_arrive_expect_tx(&bars[kBarQFull + t], kTileBytes);
                        for (int f = 0; f < SM::kHalves; ++f)
                            tc::tma_load_3d(sbase + SM::kQ + t * kTileBytes + f * kHalf, &p.qmap, f * 64, jb.h * G,
                                            jb.row0 + jb.i0 + t * kTok, &bars[kBarQFull + t]);
                        ++nq[t];
                    }
                    const int nt = max(jb.ntiles[0], jb.ntiles[1]);
                    for (int j = 0; ok && j < nt; ++j, ++it) {
                        const int st = it % kKStages;
                        ok = it < kKStages || wait_bar(&bars[kBarKEmpty + st], ((it / kKStages) - 1) & 1, abort_flag, p);
                        if (!ok) break;
                        mbar_arrive_expect_tx(&bars[kBarKFull + st], kTileBytes);
                        for (int f = 0; f < SM::kHalves; ++f)
                            tc::tma_load_3d(sbase + SM::kK + st * kTileBytes + f * kHalf, &p.kmap, f * 64, jb.h,
                                            jb.row0 + j * kTile, &bars[kBarKFull + st]);
                    }
                    ++nj;
                }
                // nothing may land after the CTA exits
                for (int i = max(0, it - kKStages); i < it; ++i)
                    mbar_wait_drain(&bars[kBarKFull + i % kKStages], (i / kKStages) & 1);
                for (int t = 0; t < 2; ++t)
                    if (nq[t] > 0) mbar_wait_drain(&bars[kBarQFull + t], (nq[t] - 1) & 1);
            }
            __syncwarp();
        } else if (warp == kVLoadWarp) {
            // ---------------------------------------------- V tiles
            int it = 0, nland = 0;
            bool ok = true;
            Job jb;
            for (int k = 0; ok && read_job_warp(k, jb); ++k) {
                const int nt = max(jb.ntiles[0], jb.ntiles[1]);
                for (int j = 0; ok && j < nt; ++j, ++it) {
                    const int st = it % kVStages;
                    const int seen = jb.nkeys - j * kTile;   // rows of the tile that the job sees
                    const bool tail = seen < kTile;
                    if (lane == 0) {
                        ok = it < kVStages || wait_bar(&bars[kBarVEmpty + st], ((it / kVStages) - 1) & 1, abort_flag, p);
                        if (ok) {
                            uint64_t *bar = tail ? &bars[kBarVLand] : &bars[kBarVFull + st];
                            mbar_arrive_expect_tx(bar, kTileBytes);
                            for (int f = 0; f < SM::kHalves; ++f)
                                tc::tma_load_3d(sbase + SM::kV + st * kTileBytes + f * kHalf, &p.vmap, f * 64, jb.h,
                                                jb.row0 + j * kTile, bar);
                        }
                    }
                    ok = __shfl_sync(kFull, ok, 0);
                    if (!ok) break;
                    if (tail) {
                        if (lane == 0) {
                            ok = wait_bar(&bars[kBarVLand], nland & 1, abort_flag, p);
                            if (!ok) mbar_wait_drain(&bars[kBarVLand], nland & 1);
                        }
                        ok = __shfl_sync(kFull, ok, 0);
                        ++nland;
                        if (!ok) break;
                        // whole rows become zero: the swizzle moves chunks within a row only
                        for (int i = lane; i < (kTile - seen) * 8 * SM::kHalves; i += 32) {
                            const int f = i / ((kTile - seen) * 8), r = i % ((kTile - seen) * 8);
                            *reinterpret_cast<uint4 *>(smem + SM::kV + st * kTileBytes + f * kHalf + seen * 128 + r * 16) =
                                make_uint4(0, 0, 0, 0);
                        }
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&bars[kBarVFull + st]);
                    }
                }
            }
            if (lane == 0)
                for (int i = max(0, it - kVStages); i < it; ++i)
                    mbar_wait_drain(&bars[kBarVFull + i % kVStages], (i / kVStages) & 1);
            __syncwarp();
        } else if (warp == kMmaWarp) {
            // ---------------------------------------------- MMA issue
            if (lane == 0) {
                constexpr uint32_t kIdQK = tc::idesc_bf16(kTile, kTile, false), kIdPV = tc::idesc_bf16(kTile, D, true);
                int itk = 0;                     // K / V tiles of earlier jobs
                int nuse[2] = {0, 0}, npf[2] = {0, 0};
                bool ok = true;
                Job jb;
                for (int k = 0; ok && read_job(k, jb); ++k) {
                    const int nt = max(jb.ntiles[0], jb.ntiles[1]);
                    const bool two = jb.ntiles[1] > 0;
                    int pend[2] = {-1, -1};      // key tile whose PV is still to be issued
                    auto issue_pv = [&](int t, int j) -> bool {
                        if (j == 0 && nuse[t] > 0 && !wait_bar(&bars[kBarOFree + t], (nuse[t] - 1) & 1, abort_flag, p))
                            return false;        // O_t of the stream's previous job
                        const int iv = itk + j, st = iv % kVStages;
                        if (!wait_bar(&bars[kBarVFull + st], (iv / kVStages) & 1, abort_flag, p)) return false;
                        if (!wait_bar(&bars[kBarPFull + t], npf[t] & 1, abort_flag, p)) return false;
                        ++npf[t];
                        tc::fence_after();
                        const uint32_t va = sbase + SM::kV + st * kTileBytes;
                        const uint32_t tP = tmem + t * 128, tO = tmem + 256 + t * 128;
#pragma unroll
                        for (int kk = 0; kk < kTile / 16; ++kk)
                            tc::mma_ts(tO, tP + kk * 8, tc::smem_desc(va + kk * 2048, kHalf, 1024), kIdPV, j > 0 || kk > 0);
                        if (t == (two ? 1 : 0)) tc::commit(&bars[kBarVEmpty + st]);   // its last reader
                        if (j == jb.ntiles[t] - 1) tc::commit(&bars[kBarOFull + t]);
                        return true;
                    };
                    for (int j = 0; ok && j <= nt; ++j) {
                        const int ik = itk + j, st = ik % kKStages;
                        bool k_ready = false;
                        for (int t = 0; ok && t < 2; ++t) {
                            if (pend[t] >= 0) {
                                ok = issue_pv(t, pend[t]);
                                pend[t] = -1;
                            }
                            if (!ok || j >= jb.ntiles[t]) continue;
                            if (j == 0) ok = wait_bar(&bars[kBarQFull + t], nuse[t] & 1, abort_flag, p);
                            if (ok && !k_ready) {
                                ok = wait_bar(&bars[kBarKFull + st], (ik / kKStages) & 1, abort_flag, p);
                                k_ready = true;
                            }
                            if (!ok) break;
                            tc::fence_after();
                            const uint32_t qa = sbase + SM::kQ + t * kTileBytes, ka = sbase + SM::kK + st * kTileBytes;
#pragma unroll
                            for (int kk = 0; kk < D / 16; ++kk) {
                                const uint32_t off = (kk & 3) * 32 + (kk >> 2) * kHalf;
                                tc::mma_ss(tmem + t * 128, tc::smem_desc(qa + off, 16, 1024),
                                           tc::smem_desc(ka + off, 16, 1024), kIdQK, kk > 0);
                            }
                            tc::commit(&bars[kBarSFull + t]);
                            pend[t] = j;
                        }
                        if (ok && j < nt) {
                            tc::commit(&bars[kBarKEmpty + st]);
                            if (j == nt - 1) tc::commit(&bars[kBarQEmpty]);
                        }
                    }
                    itk += nt;
                    for (int t = 0; t < 2; ++t) nuse[t] += jb.ntiles[t] > 0;
                }
                // everything issued has completed once this arrives
                tc::commit(&bars[kBarIdle]);
                if (!mbar_wait_drain(&bars[kBarIdle], 0)) {
                    *abort_flag = 1;
                    flag_error(p.err, PA_DEVERR_TIMEOUT);
                }
            }
            __syncwarp();
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
        // -------------------------------------------------- softmax of stream t
        const int t = warp >> 2, qd = warp & 3;
        const int r = qd * 32 + lane;                       // the thread's row
        const uint32_t lane_off = (uint32_t)(qd * 32) << 16;
        const uint32_t tS = tmem + lane_off + t * 128, tO = tmem + lane_off + 256 + t * 128;
        // a negative scale is moved into the scores; zero becomes the smallest factor that
        // still sends a masked -inf to -inf
        const bool neg = p.scale_log2 < 0.f;
        const float sl2 = fmaxf(fabsf(p.scale_log2), 1e-37f);
        int ns = 0, nuse = 0;
        bool live = true;
        Job jb;
        for (int k = 0; live && read_job_warp(k, jb); ++k) {
            if (jb.ntiles[t] == 0) continue;
            const bool row_ok = r < jb.nrows[t];
            const int tok = jb.i0 + t * kTok + r / G;        // token within the sequence
            const int lim = row_ok ? tok : INT_MAX;          // padding rows mask nothing
            float m = -INFINITY, l = 0.f;
            for (int j = 0; j < jb.ntiles[t]; ++j) {
                live = wait_bar(&bars[kBarSFull + t], ns & 1, abort_flag, p);
                live = __all_sync(kFull, live);
                if (!live) break;
                ++ns;
                tc::fence_after();
                const int key0 = j * kTile;
                float sv[kTile];
#pragma unroll
                for (int c = 0; c < 4; ++c) tc::ld32(tS + c * 32, sv + c * 32);
                tc::wait_ld();
                if (neg) {
#pragma unroll
                    for (int i = 0; i < kTile; ++i) sv[i] = -sv[i];
                }
                if (!__all_sync(kFull, lim >= key0 + kTile - 1)) {
#pragma unroll
                    for (int i = 0; i < kTile; ++i) sv[i] = key0 + i <= lim ? sv[i] : -INFINITY;
                }
                float a0 = -INFINITY, a1 = -INFINITY, a2 = -INFINITY, a3 = -INFINITY;
#pragma unroll
                for (int i = 0; i < kTile; i += 8) {
                    a0 = fmax3(a0, sv[i], sv[i + 1]);
                    a1 = fmax3(a1, sv[i + 2], sv[i + 3]);
                    a2 = fmax3(a2, sv[i + 4], sv[i + 5]);
                    a3 = fmax3(a3, sv[i + 6], sv[i + 7]);
                }
                const float mx = fmaxf(fmaxf(a0, a1), fmaxf(a2, a3)) * sl2;
                const float m_new = fmaxf(m, mx);
                if (j == 0) {
                    m = m_new;
                } else {
                    const bool resc = row_ok && m_new > m + kRescaleLog2;
                    if (__any_sync(kFull, resc)) {
                        const float alpha = resc ? fast_exp2(m - m_new) : 1.f;
                        if (resc) m = m_new;
                        l *= alpha;
                        // O_t is idle: its last PV was issued before this S
#pragma unroll 1
                        for (int c = 0; c < D; c += 16) {
                            float ov[16];
                            tc::ld16(tO + c, ov);
                            tc::wait_ld();
                            uint32_t w[16];
#pragma unroll
                            for (int i = 0; i < 16; ++i) w[i] = __float_as_uint(ov[i] * alpha);
                            tc::st16(tO + c, w);
                        }
                    }
                }
                const float m_use = m == -INFINITY ? 0.f : m;
                const float2 sc2 = make_float2(sl2, sl2), nm2 = make_float2(-m_use, -m_use);
                float2 acc0 = make_float2(0.f, 0.f), acc1 = acc0;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t w[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const int e = c * 32 + 2 * i;
                        float2 x = __ffma2_rn(make_float2(sv[e], sv[e + 1]), sc2, nm2);
                        if ((i * kPoly) / 16 != ((i + 1) * kPoly) / 16) {
                            x = exp2_fma(x);
                        } else {
                            x.x = fast_exp2(x.x);
                            x.y = fast_exp2(x.y);
                        }
                        if (i & 1) acc1 = __fadd2_rn(acc1, x);
                        else acc0 = __fadd2_rn(acc0, x);
                        w[i] = pack_bf16x2(x.x, x.y);
                    }
                    tc::st16(tS + c * 16, w);
                }
                l += (acc0.x + acc0.y) + (acc1.x + acc1.y);
                tc::wait_st();
                tc::fence_before();
                mbar_arrive(&bars[kBarPFull + t]);
            }
            if (!live) break;
            // ---- the output rows
            live = wait_bar(&bars[kBarOFull + t], nuse & 1, abort_flag, p);
            live = __all_sync(kFull, live);
            if (!live) break;
            ++nuse;
            tc::fence_after();
            const float inv = l > 0.f ? 1.f / l : l;      // NaN stays NaN
            unsigned char *dst = p.out + ((int64_t)(jb.row0 + tok) * p.num_q_heads + jb.h * G + r % G) * (D * 2);
            bool odd = false;
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
                float o[32];
                tc::ld32(tO + c, o);
                tc::wait_ld();
                uint32_t w[16];
                float bad = 0.f;
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float x = o[2 * i] * inv, y = o[2 * i + 1] * inv;
                    bad = fmaf(x, 0.f, fmaf(y, 0.f, bad));   // NaN once anything is not finite
                    w[i] = pack_bf16x2(x, y);
                }
                odd |= bad != 0.f;
                if (row_ok) {
#pragma unroll
                    for (int i = 0; i < 16; i += 4)
                        *reinterpret_cast<uint4 *>(dst + c * 2 + i * 4) = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
                }
            }
            tc::fence_before();
            mbar_arrive(&bars[kBarOFree + t]);
            unsigned again = __ballot_sync(kFull, odd && row_ok);
            while (again) {
                const int ln = __ffs(again) - 1;
                again &= again - 1;
                const int rr = qd * 32 + ln, i = jb.i0 + t * kTok + rr / G;
                if (masked_not_finite<D>(p, jb.row0, i, min(jb.nkeys, (jb.ntiles[t]) * kTile), jb.h, lane))
                    redo_row<D>(p, jb.row0, i, jb.h * G + rr % G, jb.h, lane);
            }
        }
    }
    tc::fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc::fence_after();
        tc::dealloc(tmem, kTmemCols);
    }
}

// ---------------------------------------------------------------- host
PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
    });
    return fn;
}

// [tokens][heads][d] bf16 rows, tokens `stride` bytes apart, as {d, heads, tokens} with boxes
// {64, b1, b2} and the 128-byte swizzle; coordinates outside read zeros.
bool encode_map(CUtensorMap *m, const void *base, int d, uint64_t heads, uint64_t tokens, uint64_t stride, uint32_t b1,
                uint32_t b2) {
    auto fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)d, heads, tokens};
    const cuuint64_t strides[2] = {(cuuint64_t)d * 2, stride};
    const cuuint32_t box[3] = {64, b1, b2};
    const cuuint32_t estr[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, int G>
cudaError_t launch_attention(const Params &p, int grid, cudaStream_t stream) {
    const cudaError_t e = cudaFuncSetAttribute(packed_prefill_kernel<D, G>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (int)Smem<D>::kBytes);
    if (e != cudaSuccess) return e;
    return launch_after(packed_prefill_kernel<D, G>, dim3((unsigned)grid), dim3(kThreads), Smem<D>::kBytes, stream, p);
}

template <int D>
cudaError_t launch_group(const Params &p, int g, int grid, cudaStream_t stream) {
    switch (g) {
        case 1: return launch_attention<D, 1>(p, grid, stream);
        case 2: return launch_attention<D, 2>(p, grid, stream);
        case 4: return launch_attention<D, 4>(p, grid, stream);
        case 8: return launch_attention<D, 8>(p, grid, stream);
        default: return cudaErrorInvalidValue;
    }
}

int64_t max_jobs(int64_t num_tokens, int64_t num_seqs, int64_t g) {
    // pairs of sequence s: ceil(len g / 256) <= len g / 256 + 1
    return num_tokens * g / (2 * kTile) + num_seqs;
}

}  // namespace

size_t packed_workspace(int32_t num_tokens, int32_t num_seqs, int32_t g) {
    return 16 + (size_t)max_jobs(num_tokens, num_seqs, g) * 16;
}

cudaError_t launch_prefill_packed(const PackedPrefill &a, cudaStream_t stream) {
    const int g = a.num_q_heads / a.num_kv_heads, d = a.head_dim;
    const int64_t jobs = max_jobs(a.num_tokens, a.num_seqs, g);
    if (jobs * a.num_kv_heads > INT32_MAX / 2) return cudaErrorNotSupported;
    PlanParams pl;
    pl.starts = a.starts;
    pl.meta = static_cast<int32_t *>(a.workspace);
    pl.jobs = reinterpret_cast<int4 *>(static_cast<char *>(a.workspace) + 16);
    pl.err = a.err;
    pl.num_seqs = a.num_seqs;
    pl.num_tokens = a.num_tokens;
    pl.max_len = a.max_seq_len;
    pl.pair_tokens = 2 * kTile / g;
    pl.max_jobs = (int32_t)jobs;
    Params p;
    std::memset(&p, 0, sizeof(p));
    const uint64_t T = (uint64_t)a.num_tokens;
    if (!encode_map(&p.qmap, a.query, d, (uint64_t)a.num_q_heads, T, (uint64_t)a.q_stride * 2, (uint32_t)g, kTile / g) ||
        !encode_map(&p.kmap, a.key, d, (uint64_t)a.num_kv_heads, T, (uint64_t)a.k_stride * 2, 1, kTile) ||
        !encode_map(&p.vmap, a.value, d, (uint64_t)a.num_kv_heads, T, (uint64_t)a.v_stride * 2, 1, kTile))
        return cudaErrorInvalidValue;
    p.q = static_cast<const unsigned char *>(a.query);
    p.k = static_cast<const unsigned char *>(a.key);
    p.v = static_cast<const unsigned char *>(a.value);
    p.q_stride = a.q_stride * 2;
    p.k_stride = a.k_stride * 2;
    p.v_stride = a.v_stride * 2;
    p.out = static_cast<unsigned char *>(a.out);
    p.err = a.err;
    p.jobs = pl.jobs;
    p.meta = pl.meta;
    p.num_q_heads = a.num_q_heads;
    p.num_kv_heads = a.num_kv_heads;
    p.scale_log2 = a.scale * kLog2e;
    p.wait_ns = wait_limit_ns();
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const size_t plan_smem = (size_t)(a.num_seqs + 1) * 4;
    if ((e = cudaFuncSetAttribute(packed_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                  (kMaxPlanSeqs + 1) * 4)) != cudaSuccess)
        return e;
    packed_plan_kernel<<<1, kPlanThreads, plan_smem, stream>>>(pl);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    const int grid = (int)std::min<int64_t>(jobs * a.num_kv_heads, num_sms(dev));
    return d == 128 ? launch_group<128>(p, g, grid, stream) : launch_group<64>(p, g, grid, stream);
}

}  // namespace pa
