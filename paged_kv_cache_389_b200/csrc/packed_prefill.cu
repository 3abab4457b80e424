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
// tile (stream 0 may need one tile less):
//   S_t = Q_t K^T   tcgen05.mma, M = 128, N = keys of the tile -> tensor memory
//   P_t = 2^(S_t scale log2(e) - m_t), one row per thread -> tensor memory as bf16
//   O_t += P_t V    tcgen05.mma with A = P_t read from tensor memory, B = V (MN-major)
// P does not take S's place: S(j + 1) is computed as soon as S(j) is in registers, so the
// softmax warps find their next tile ready and the tensor core works behind them.  (With P
// over S, a stream's scores had to wait for P, PV and QK in turn: 4,100 to 4,700 clocks a
// 128-key step of both streams, 2.1 to 2.5 ms for the case below.)  The reference point m_t moves (and O_t is
// rescaled) only when a row's maximum rises by more than 2^8; sums are fp32, P is
// rounded to bf16 once (2^-8, as the operand type asks).
//
// What bounds it.  d = 128: per 80-key tile of both streams the tensor core needs 1,490
// clocks (measured alone; S with both operands in shared memory reads them at the
// bank limit), the special-function units 1,280 for the exponentials; a step takes about
// 1,850.  2 x 8192 tokens, 64/8 heads: 1.76 ms in a burst (1,225 TFLOP/s), 1.99 to 2.09 ms where
// calls follow each other for 0.15 s and the power limit takes the clock down to 1.56 GHz; 16 x 1024 tokens,
// 32/8 heads: 0.17 ms, 815 TFLOP/s, where a job has 7 tiles and its output rows (4,000 clocks) are no
// longer small beside them.
// d = 64: the products are half as long, the exponentials are not: 2,048 clocks of a step's 2,900.
// Tried and slower: output rows written by four more warps (128 registers a thread at launch:
// 184 us against 170 for 16 x 1024 tokens) or after the next job's first tile (189); jobs
// ordered by sequence instead of longest first (177).
// Within a softmax step, all slower: exponentials with the old reference point while the new
// maximum is found (16 sequences up to 2048: 213 us against 179); the next tile's first scores
// fetched between them (203); P handed over in two halves (183); the two streams taking turns
// at the exponentials (2 x 8192: 2,130 us against 2,035).  d = 64 with 64, 96, 112 keys a tile: 95,
// 92, 90 us against 85.
// A share of the exponentials on the FMA units (a cubic in the fraction) was tried at 1, 2
// and 3 of 8: no gain at d = 128, 3 to 9 % slower at d = 64, so there is none.
//
// Work: plan_kernel lists the (sequence, row pair) jobs, longest first, and zeroes the
// counter from which the persistent CTAs draw (job, kv head) in that order; so the
// lengths are read on the device only and a captured graph follows them.  A few short
// sequences (one row pair each) need no list: see launch_prefill_packed.
// Warp roles: 0-3 softmax of stream 0, 4-7 of stream 1 (tensor-memory lanes 32 (w % 4) ..),
// 8 and 11 issue the MMAs of streams 0 and 1 (8 owns the tensor memory), 9 draws jobs and
// loads Q and K, 10 loads V.  K and V tiles share a ring, each slot released by both
// streams; a stream that has no rows for a tile still waits for it and releases it, so that
// the slot's arrivals never mix phases.
// Masked places: a key behind a row is left out by position, so its score may be
// anything.  Its value meets P = 0 in the tensor core, where an infinity or a NaN would
// survive: the loader zeroes the rows of the last tile that no row of the job sees, and a
// row that comes out not finite while a value masked for it is not finite is
// computed again (redo_rows).
// Every wait is bounded (from the last step of redo_rows, if there was one); an abort drains the
// copies and MMAs in flight and frees the tensor memory.
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
constexpr int kTile = 128;           // rows of a query tile
constexpr int kThreads = 12 * 32;
constexpr int kMmaWarp = 8, kLoadWarp = 9, kVLoadWarp = 10;
// Registers: the launch gives 384 x 168; the softmax warpgroups take 200 (a row of S), the
// other one 96: 256 x 200 + 128 x 96 <= 384 x 168.
constexpr int kRegsSoftmax = 200, kRegsOther = 96;
static_assert(256 * kRegsSoftmax + 128 * kRegsOther <= kThreads * 168, "register split over the launch's total");
constexpr float kRescaleLog2 = 8.f;
constexpr int kDirectJobs = 16;
constexpr int kStages = 3;           // K/V ring
constexpr uint32_t kOutBytes = 32 * 128;   // a softmax warp's staging of output rows, 64 columns at a time

// Keys of a K/V tile, and a stream's 256 tensor-memory columns: S (fp32 scores), P (bf16
// probabilities, two to a column) and O.  P does not lie over S, so that the next tile's
// scores are computed while this tile's exponentials are: with d = 128 that leaves room
// for 80 keys.
template <int D>
struct Tiles {
    static constexpr int kKeys = D == 128 ? 80 : 128;
    static constexpr uint32_t kP = kKeys, kO = 256 - D, kStream = 256, kCols = 512;
    static_assert(kP + kKeys / 2 <= kO, "S, P and O of a stream share 256 columns");
    // Sixteens of keys whose exponentials are taken before P_t is known to be free (kept in the
    // registers that their scores held): the last PV is waited for behind them.  In the order of
    // 0, 1, 3, all: 2 x 8192 tokens 2,002, 1,961, 1,961, 1,971 us (at the power limit), 16
    // sequences up to 2048 184, 179, 178, 179 us; d = 64: 85, 85, 85, 87 us.
    static constexpr int kAhead = 3;
    static_assert(kKeys % 16 == 0, "whole k steps");
};
constexpr uint32_t kQHalf = kTile * 128;   // 64 columns of a 128-row tile in shared memory

constexpr int kJobSlots = 8;         // job records in shared memory

enum Bar {
    // A job of n key tiles uses n + 1 slots of the K/V ring; slot i holds K(i) and V(i - 1): what
    // the products between two softmax steps read, under one barrier.
    kBarFull = 0,                        // [kStages] K landed, and V ready (one arrival of each loader)
    kBarEmpty = kBarFull + kStages,      // [kStages] both streams are done with the slot
    kBarVLand = kBarEmpty + kStages,     // a last V tile landed (its unseen rows are zeroed next)
    kBarQFull = kBarVLand + 1,           // [2] Q_t landed
    kBarQEmpty = kBarQFull + 2,          // the job's last QKs are done
    kBarSFull = kBarQEmpty + 1,          // [2] S_t written
    kBarSRead = kBarSFull + 2,           // [2] S_t is in registers (128 threads)
    kBarPFull = kBarSRead + 2,           // [2] P_t written (128 threads)
    kBarPFree = kBarPFull + 2,           // [2] PV_t is done: P_t may be written, O_t rescaled
    kBarOFull = kBarPFree + 2,           // [2] the job's last PV_t is done
    kBarOFree = kBarOFull + 2,           // [2] O_t has been read (128 threads)
    kBarIdle = kBarOFree + 2,            // [2] every MMA of a stream has completed
    kBarRead = kBarIdle + 2,             // [kJobSlots] the slot's job has been read by every softmax warp
    kNumBars = kBarRead + kJobSlots
};

struct Misc {                     // in shared memory
    uint32_t tmem;                // tensor-memory address
    int abort;                    // raised by the first warp whose wait ran out
    unsigned long long step;      // when redo_rows took its last step
};

template <int D>
struct Smem {
    static constexpr int kHalves = D / 64;
    static constexpr uint32_t kQBytes = kHalves * kQHalf;
    static constexpr uint32_t kHalf = Tiles<D>::kKeys * 128;             // 64 columns of a K/V tile
    static constexpr uint32_t kTileBytes = kHalves * kHalf;
    static constexpr uint32_t kQ = 0;
    static constexpr uint32_t kK = 2 * kQBytes;
    static constexpr uint32_t kV = kK + kStages * kTileBytes;
    static constexpr uint32_t kOut = kV + kStages * kTileBytes;
    static constexpr uint32_t kBars = kOut + 8 * kOutBytes;
    static constexpr uint32_t kMisc = kBars + kNumBars * 8;              // Misc
    static constexpr uint32_t kJobs = (kMisc + sizeof(Misc) + 15) / 16 * 16;     // int4 [8] records, int [8] tags
    static constexpr size_t kBytes = kJobs + 8 * 16 + 8 * 4 + 1024;      // slack to align the base
    static_assert(kQBytes % 1024 == 0 && kHalf % 1024 == 0 && kBars % 8 == 0, "swizzled tiles 1024-byte aligned");
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
    const int32_t *starts;                  // not null: no list, one job per sequence and kv head
    int32_t num_seqs, num_tokens, max_len;
    int32_t num_q_heads, num_kv_heads;
    float scale_log2;
    unsigned long long wait_ns;
};

struct PlanParams {
    const int32_t *starts;
    int4 *jobs;
    int32_t *meta;
    int32_t *err;
    int32_t num_seqs, num_tokens, max_len, pair_tokens, max_jobs;   // 1 <= max_len <= num_tokens
};

// ---------------------------------------------------------------- the job list
constexpr int kPlanThreads = 1024;
constexpr int kBuckets = 256;

// Rows outside the tensors, or a sequence longer than announced.
__device__ __forceinline__ bool bad_sequence(int a, int b, int num_tokens, int max_len) {
    return a < 0 || b < a || b > num_tokens || b - a > max_len;
}

// Sums of pairs stop here: starts that go back and forth can name far more than 2^31 of
// them, and such a list has to read as too long, not as a short one.
constexpr int kManyPairs = INT32_MAX / 2;
__device__ __forceinline__ int add_pairs(int a, int b) { return min(a + b, kManyPairs); }

// The sum (add_pairs) of the values of the threads before this one; *total: of all.
__device__ __forceinline__ int block_scan(int v, int *total, int *warp_sums) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(kFull, incl, o);
        if (lane >= o) incl = add_pairs(incl, y);
    }
    const int excl = __shfl_up_sync(kFull, incl, 1);
    if (lane == 31) warp_sums[warp] = incl;
    __syncthreads();
    int w = warp_sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(kFull, w, o);
        if (lane >= o) w = add_pairs(w, y);
    }
    *total = __shfl_sync(kFull, w, 31);
    const int off = __shfl_sync(kFull, w, warp > 0 ? warp - 1 : 0);
    __syncthreads();
    return add_pairs(warp > 0 ? off : 0, lane > 0 ? excl : 0);
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
        if (bad_sequence(a, b, p.num_tokens, p.max_len)) bad = true;   // skipped and flagged
        else if (b > a) pairs = (b - a - 1) / p.pair_tokens + 1;
        cum[s] = pairs;
        sum = add_pairs(sum, pairs);
    }
    int total;
    int run = block_scan(sum, &total, warp_sums);
    for (int s = beg; s < end; ++s) {
        const int pairs = cum[s];
        cum[s] = run;
        run = add_pairs(run, pairs);
    }
    if (threadIdx.x == 0) cum[S] = total;
    // overlapping sequences could list more pairs than the list holds
    const bool fits = total <= p.max_jobs;
    if (bad || (!fits && threadIdx.x == 0)) flag_error(p.err, PA_DEVERR_CHUNK);
    __syncthreads();
    if (!fits) total = 0;
    const int most = (p.max_len - 1) / p.pair_tokens + 1;   // pairs of the longest sequence: jp < most
    auto bucket_of = [&](int jp) { return kBuckets - 1 - (int)((int64_t)jp * kBuckets / most); };
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
// Within a wait since t0: false when another warp gave up or the bound has passed.  It counts from
// the last step of redo_rows: that takes as long as its prompt is, and is no wait that ran out.
__device__ __forceinline__ bool may_wait(unsigned long long t0, volatile Misc *misc, const Params &p) {
    if (misc->abort) return false;
    const unsigned long long now = global_ns();
    if (now - t0 <= p.wait_ns) return true;
    const unsigned long long step = misc->step;
    if (step >= now || now - step <= p.wait_ns) return true;
    misc->abort = 1;
    flag_error(p.err, PA_DEVERR_TIMEOUT);
    return false;
}

__device__ __forceinline__ bool wait_bar(uint64_t *bar, uint32_t parity, volatile Misc *misc, const Params &p) {
    if (mbar_try_wait(bar, parity)) return true;
    const unsigned long long t0 = global_ns();
    for (uint32_t it = 1;; ++it) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((it & 7u) == 0 && !may_wait(t0, misc, p)) return false;
    }
}

struct Job {
    int row0;        // the sequence's first row
    int i0;          // first token of tile 0 within the sequence
    int h;
    int nrows[2];    // packed rows in use
    int ntiles[2];   // key tiles of each stream (0: the stream has no rows)
    int nkeys;       // keys the job's last row sees
};

template <int D, int G>
__device__ __forceinline__ void make_job(int4 rec, Job &jb) {
    constexpr int kTok = kTile / G;   // tokens of a tile
    const int rows = rec.y * G - rec.z * 2 * kTile;
    jb.row0 = rec.x;
    jb.i0 = rec.z * 2 * kTok;
    jb.h = rec.w;
    jb.nrows[0] = min(kTile, rows);
    jb.nrows[1] = min(kTile, max(0, rows - kTile));
    const int k0 = min(rec.y, jb.i0 + kTok), k1 = min(rec.y, jb.i0 + 2 * kTok);
    constexpr int kKeys = Tiles<D>::kKeys;
    jb.ntiles[0] = (k0 + kKeys - 1) / kKeys;
    jb.ntiles[1] = jb.nrows[1] > 0 ? (k1 + kKeys - 1) / kKeys : 0;
    jb.nkeys = jb.nrows[1] > 0 ? k1 : k0;
}

__device__ __forceinline__ float fmax3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// The last key of [from, end) whose value holds an infinity or a NaN; -1 if none does.
template <int D>
__device__ __forceinline__ int last_not_finite(const Params &p, int row0, int from, int end, int h, int lane, volatile Misc *misc) {
    for (int j = end - 1; j >= from; --j) {
        const uint16_t *v = reinterpret_cast<const uint16_t *>(p.v + (int64_t)(row0 + j) * p.v_stride) + h * D;
        bool found = false;
        for (int e = lane; e < D; e += 32) found |= (v[e] & 0x7fffu) >= 0x7f80u;
        if (__any_sync(kFull, found)) return j;
        if (lane == 0) misc->step = global_ns();
    }
    return -1;
}

// Eight rows of a tile again, those whose bit is set in `want`, by a whole warp: row x is token
// tok0 + x / G of the sequence at row0, query head h G + x % G.  A value meets only the rows that
// see it (a row's sum skips the others), so nothing masked can reach one.
// Scores eight keys at a time on 16 x 8 tiles, whose lower half is empty (lane 4 g + t: row g, dims
// D / 4 t .. of queries, keys, values and sums, keys 2 t and 2 t + 1 of the scores); the sums in
// fp32 fused multiply-adds.  A prompt of 16,384 tokens, 32/8 heads, head_dim 128, whose last value
// is not finite: 37 ms (1.7 without; one row after the other, a key at a time, 307).  Sixteen rows at a
// time left the softmax warps fewer registers: 24 short prompts 12.4 us instead of 11.6.
template <int D, int G>
__device__ __forceinline__ void redo_eight(const Params &p, int row0, int tok0, int h, unsigned want, int lane,
                                           volatile Misc *misc) {
    constexpr int E = D / 4;
    const int g = lane >> 2, t = lane & 3;
    const int tok = tok0 + g / G, hq = h * G + g % G;
    const bool mine = (want >> g & 1u) != 0;
    const int last = tok0 + (31 - __clz(want)) / G;      // the last key that one of the rows sees
    uint32_t qa[D / 16][2];
    const unsigned char *qr = p.q + (int64_t)(row0 + tok) * p.q_stride + (hq * D + E * t) * 2;
#pragma unroll
    for (int i = 0; i < E / 8; ++i) {
        uint4 x = make_uint4(0, 0, 0, 0);
        if (mine) x = __ldg(reinterpret_cast<const uint4 *>(qr) + i);
        qa[2 * i][0] = x.x;
        qa[2 * i][1] = x.y;
        qa[2 * i + 1][0] = x.z;
        qa[2 * i + 1][1] = x.w;
    }
    float acc[E], m = -INFINITY, l = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
#pragma unroll 1
    for (int kb = 0; kb <= last; kb += 8) {
        const unsigned char *kr = p.k + (int64_t)(row0 + kb + g) * p.k_stride + (h * D + E * t) * 2;
        float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < E / 8; ++i) {
            uint4 x = make_uint4(0, 0, 0, 0);
            if (kb + g <= last) x = __ldg(reinterpret_cast<const uint4 *>(kr) + i);
            const uint32_t a0[4] = {qa[2 * i][0], 0u, qa[2 * i][1], 0u}, a1[4] = {qa[2 * i + 1][0], 0u, qa[2 * i + 1][1], 0u};
            mma_bf16_16816(s, a0, x.x, x.y);
            mma_bf16_16816(s, a1, x.z, x.w);
        }
        const bool see0 = kb + 2 * t <= tok, see1 = kb + 2 * t + 1 <= tok;
        const float s0 = s[0] * p.scale_log2, s1 = s[1] * p.scale_log2;
        float mn = m;
        if (see0) mn = fmaxf(mn, s0);
        if (see1) mn = fmaxf(mn, s1);
        mn = fmaxf(mn, __shfl_xor_sync(kFull, mn, 1));
        mn = fmaxf(mn, __shfl_xor_sync(kFull, mn, 2));
        const float base = mn == -INFINITY ? 0.f : mn, a = exp2f(m - base);
        m = mn;
        const float p0 = see0 ? exp2f(s0 - base) : 0.f, p1 = see1 ? exp2f(s1 - base) : 0.f;
        l = l * a + (p0 + p1);
        if (a != 1.f) {
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] *= a;
        }
        const int keys = min(8, last + 1 - kb);
#pragma unroll 1
        for (int c = 0; c < keys; ++c) {
            const float w = __shfl_sync(kFull, c & 1 ? p1 : p0, (lane & 28) | (c >> 1));
            const uint4 *vr = reinterpret_cast<const uint4 *>(p.v + (int64_t)(row0 + kb + c) * p.v_stride + (h * D + E * t) * 2);
            uint4 x[E / 8];
#pragma unroll
            for (int i = 0; i < E / 8; ++i) x[i] = __ldg(vr + i);
            if (kb + c > tok) continue;
#pragma unroll
            for (int i = 0; i < E / 8; ++i) {
                const uint32_t v2[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    const float2 v = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&v2[y]));
                    acc[8 * i + 2 * y] = fmaf(w, v.x, acc[8 * i + 2 * y]);
                    acc[8 * i + 2 * y + 1] = fmaf(w, v.y, acc[8 * i + 2 * y + 1]);
                }
            }
        }
        if (lane == 0) misc->step = global_ns();
        if ((kb & 127) == 0) {
            // a sum that is NaN stays NaN: nothing to add where all are
            bool done = true;
#pragma unroll
            for (int e = 0; e < E; ++e) done &= !mine || acc[e] != acc[e];
            if (__all_sync(kFull, done)) break;
            if (__any_sync(kFull, misc->abort != 0)) return;
        }
    }
    l += __shfl_xor_sync(kFull, l, 1);
    l += __shfl_xor_sync(kFull, l, 2);
    if (!mine) return;
    uint4 *dst = reinterpret_cast<uint4 *>(p.out + (((int64_t)(row0 + tok) * p.num_q_heads + hq) * D + E * t) * 2);
    const float f = l > 0.f ? 1.f / l : l;               // NaN stays NaN
#pragma unroll
    for (int i = 0; i < E / 8; ++i) {
        uint32_t w[4];
#pragma unroll
        for (int y = 0; y < 4; ++y) w[y] = pack_bf16x2(acc[8 * i + 2 * y] * f, acc[8 * i + 2 * y + 1] * f);
        dst[i] = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// Of a softmax warp's 32 rows, the first of them token tok0, those whose bit is set in `odd` came out
// not finite: where a value masked for them is not finite, among the keys below `end` that their
// tiles held, they are computed again.  (A row that sees the last such value is what it should be.)
template <int D, int G>
__device__ __noinline__ void redo_rows(const Params &p, int row0, int tok0, int h, int end, unsigned odd, volatile Misc *misc) {
    const int lane = threadIdx.x & 31;
    const int worst = last_not_finite<D>(p, row0, tok0 + 1, end, h, lane, misc);
    odd &= __ballot_sync(kFull, tok0 + lane / G < worst);
#pragma unroll 1
    for (int x = 0; x < 32; x += 8)
        if (odd >> x & 0xffu) redo_eight<D, G>(p, row0, tok0 + x / G, h, odd >> x & 0xffu, lane, misc);
}

template <int D, int G>
__global__ void __launch_bounds__(kThreads, 1) packed_prefill_kernel(const __grid_constant__ Params p) {
    using SM = Smem<D>;
    using TL = Tiles<D>;
    constexpr uint32_t kTileBytes = SM::kTileBytes, kHalf = SM::kHalf;
    constexpr int kKeys = TL::kKeys;
    constexpr int kTok = kTile / G;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char *smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    const uint32_t sbase = smem_u32(smem);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + SM::kBars);
    volatile Misc *misc = reinterpret_cast<volatile Misc *>(smem + SM::kMisc);
    // The K loader draws the CTA's jobs and publishes job k in slot k & 7 (a record without
    // tokens ends the work); the other warps read it there.
    volatile int *job_rec = reinterpret_cast<volatile int *>(smem + SM::kJobs);
    volatile int *job_tag = job_rec + 32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < 8; ++i) job_tag[i] = -1;
        for (int i = 0; i < kNumBars; ++i) {
            const bool rows = (i >= kBarSRead && i < kBarSRead + 2) || (i >= kBarPFull && i < kBarPFull + 2) ||
                              (i >= kBarOFree && i < kBarOFree + 2);
            const bool both = i < kBarVLand || i == kBarQEmpty;
            mbar_init(&bars[i], rows ? 128 : i >= kBarRead ? 8 : both ? 2 : 1);
        }
        misc->abort = 0;
        misc->step = 0;
        mbar_init_fence();
    }
    if (warp == kLoadWarp && lane == 0) {
        tc::prefetch_map(&p.qmap);
        tc::prefetch_map(&p.kmap);
        tc::prefetch_map(&p.vmap);
    }
    if (warp == kMmaWarp) tc::alloc(const_cast<uint32_t *>(&misc->tmem), TL::kCols);
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tmem = misc->tmem;

    auto read_job_warp = [&](int k, Job &jb) -> bool {
        int ok = 0;
        if (lane == 0) {
            const unsigned long long t0 = global_ns();
            ok = 1;
            while (ok && job_tag[k & 7] != k) ok = may_wait(t0, misc, p);
            __threadfence_block();
        }
        ok = __shfl_sync(kFull, ok, 0);
        if (!ok) return false;
        const int4 rec = make_int4(job_rec[(k & 7) * 4], job_rec[(k & 7) * 4 + 1], job_rec[(k & 7) * 4 + 2],
                                   job_rec[(k & 7) * 4 + 3]);
        if (rec.y <= 0) return false;
        make_job<D, G>(rec, jb);
        return true;
    };

    // Nothing may land after the CTA exits: a loader waits for the slots it filled last (their
    // loads land together; after an abort, when the other loader has left its half out, until
    // the bound).
    auto drain_slots = [&](int it) {
        for (int i = max(0, it - kStages); i < it; ++i)
            mbar_wait_drain(&bars[kBarFull + i % kStages], (i / kStages) & 1);
    };

    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
        if (warp == kLoadWarp) {
            // ---------------------------------------------- jobs, Q and K tiles
            if (lane == 0) {
                grid_dep_wait();   // the job list is complete
                const int njobs = (p.starts ? p.num_seqs : __ldcg(p.meta)) * p.num_kv_heads;
                int it = 0, nq[2] = {0, 0}, nj = 0;
                bool ok = true;
                int u = (int)blockIdx.x;
                for (int k = 0; ok; ++k) {
                    int4 rec = make_int4(0, 0, 0, 0);
                    for (; u < njobs; u += (int)gridDim.x) {
                        const int e = u / p.num_kv_heads, h = u % p.num_kv_heads;
                        if (!p.starts) {
                            rec = __ldcg(p.jobs + e);
                            rec.w = h;
                            break;
                        }
                        const int a = __ldg(p.starts + e), b = __ldg(p.starts + e + 1);
                        if (bad_sequence(a, b, p.num_tokens, p.max_len)) {
                            if (h == 0) flag_error(p.err, PA_DEVERR_CHUNK);
                        } else if (b > a) {
                            rec = make_int4(a, b - a, 0, h);
                            break;
                        }
                    }
                    // A stream without rows in a job does not hold the others up, so a softmax warp
                    // may be jobs behind: its record has to stay until it has read it.
                    if (k >= kJobSlots) ok = wait_bar(&bars[kBarRead + (k & 7)], ((k >> 3) - 1) & 1, misc, p);
                    if (!ok) break;
                    job_rec[(k & 7) * 4] = rec.x;
                    job_rec[(k & 7) * 4 + 1] = rec.y;
                    job_rec[(k & 7) * 4 + 2] = rec.z;
                    job_rec[(k & 7) * 4 + 3] = rec.w;
                    __threadfence_block();
                    job_tag[k & 7] = k;
                    if (rec.y <= 0) break;
                    // the next job is drawn now and needed when this one's tiles are issued
                    u = p.starts ? u + (int)gridDim.x : (int)gridDim.x + atomicAdd(p.meta + 1, 1);
                    Job jb;
                    make_job<D, G>(rec, jb);
                    if (nj > 0) ok = wait_bar(&bars[kBarQEmpty], (nj - 1) & 1, misc, p);
                    for (int t = 0; ok && t < 2; ++t) {
                        if (jb.ntiles[t] == 0) continue;
                        mbar_arrive_expect_tx(&bars[kBarQFull + t], SM::kQBytes);
                        for (int f = 0; f < SM::kHalves; ++f)
                            tc::tma_load_3d(sbase + SM::kQ + t * SM::kQBytes + f * kQHalf, &p.qmap, f * 64, jb.h * G,
                                            jb.row0 + jb.i0 + t * kTok, &bars[kBarQFull + t]);
                        ++nq[t];
                    }
                    const int nt = max(jb.ntiles[0], jb.ntiles[1]);
                    for (int i = 0; ok && i <= nt; ++i, ++it) {
                        const int st = it % kStages;
                        ok = it < kStages || wait_bar(&bars[kBarEmpty + st], ((it / kStages) - 1) & 1, misc, p);
                        if (!ok) break;
                        if (i == nt) {           // the last slot holds V only
                            mbar_arrive(&bars[kBarFull + st]);
                            continue;
                        }
                        mbar_arrive_expect_tx(&bars[kBarFull + st], kTileBytes);
                        for (int f = 0; f < SM::kHalves; ++f)
                            tc::tma_load_3d(sbase + SM::kK + st * kTileBytes + f * kHalf, &p.kmap, f * 64, jb.h,
                                            jb.row0 + i * kKeys, &bars[kBarFull + st]);
                    }
                    ++nj;
                }
                // nothing may land after the CTA exits
                drain_slots(it);
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
                for (int i = 0; ok && i <= nt; ++i, ++it) {
                    const int st = it % kStages;
                    const int seen = jb.nkeys - (i - 1) * kKeys;   // rows of V(i - 1) that the job sees
                    const bool tail = i > 0 && seen < kKeys;
                    if (lane == 0) {
                        ok = it < kStages || wait_bar(&bars[kBarEmpty + st], ((it / kStages) - 1) & 1, misc, p);
                        if (ok && i == 0) mbar_arrive(&bars[kBarFull + st]);   // the first slot holds K only
                        if (ok && i > 0) {
                            uint64_t *bar = tail ? &bars[kBarVLand] : &bars[kBarFull + st];
                            mbar_arrive_expect_tx(bar, kTileBytes);
                            for (int f = 0; f < SM::kHalves; ++f)
                                tc::tma_load_3d(sbase + SM::kV + st * kTileBytes + f * kHalf, &p.vmap, f * 64, jb.h,
                                                jb.row0 + (i - 1) * kKeys, bar);
                            if (tail) {
                                ok = wait_bar(bar, nland & 1, misc, p);
                                if (!ok) mbar_wait_drain(bar, nland & 1);
                            }
                        }
                    }
                    ok = __shfl_sync(kFull, ok, 0);
                    if (!ok) break;
                    if (tail) {
                        ++nland;
                        // whole rows become zero: the swizzle moves chunks within a row only
                        const int bytes = (kKeys - seen) * 128;
#pragma unroll
                        for (int f = 0; f < SM::kHalves; ++f) {
                            unsigned char *rows = smem + SM::kV + st * kTileBytes + f * kHalf + seen * 128;
                            for (int x = lane * 16; x < bytes; x += 512)
                                *reinterpret_cast<uint4 *>(rows + x) = make_uint4(0, 0, 0, 0);
                        }
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&bars[kBarFull + st]);
                    }
                }
            }
            if (lane == 0) drain_slots(it);
            __syncwarp();
        } else {
            // ---------------------------------------------- MMA issue of stream t (the whole
            // warp, converged; one elected lane issues).  A warp per stream, because issuing
            // blocks at the tensor core's own pace and a wait costs 70 to 200 clocks even
            // when its phase is long over: one stream's waits pass while the other's
            // products run.
            const int t = warp == kMmaWarp ? 0 : 1;
            constexpr uint32_t kIdQK = tc::idesc_bf16(kTile, kKeys, false), kIdPV = tc::idesc_bf16(kTile, D, true);
            const uint64_t qd = tc::smem_desc(sbase + SM::kQ + t * SM::kQBytes, 16, 1024);
            const uint64_t k_desc = tc::smem_desc(sbase + SM::kK, 16, 1024);
            const uint64_t v_desc = tc::smem_desc(sbase + SM::kV, kHalf, 1024);
            const uint32_t tS = tmem + t * TL::kStream, tP = tS + TL::kP, tO = tS + TL::kO;
            auto wait_all = [&](int bar, uint32_t parity) -> bool {
                return __all_sync(kFull, wait_bar(&bars[bar], parity, misc, p));
            };
            int it = 0;                          // slots of the K/V ring so far
            int nuse = 0, nqk = 0, npv = 0;      // this stream's jobs, QKs and PVs
            bool ok = true;
            Job jb;
            for (int k = 0; ok && read_job_warp(k, jb); ++k) {
                const int nt = max(jb.ntiles[0], jb.ntiles[1]), mine = jb.ntiles[t];
                if (mine > 0) ok = wait_all(kBarQFull + t, nuse & 1);
                // slot i: QK(i) once S(i - 1) is in registers, then PV(i - 1) once P(i - 1) is written
                for (int i = 0; ok && i <= nt; ++i, ++it) {
                    const int st = it % kStages;
                    const bool qk = i < mine, pv = i > 0 && i <= mine;
                    ok = wait_all(kBarFull + st, (it / kStages) & 1);
                    if (qk) {
                        if (ok && nqk > 0) ok = wait_all(kBarSRead + t, (nqk - 1) & 1);
                        if (!ok) break;
                        ++nqk;
                        tc::fence_after();
                        if (tc::elect_one()) {
                            const uint64_t kd = k_desc + (uint32_t)st * (kTileBytes >> 4);
#pragma unroll
                            for (int kk = 0; kk < D / 16; ++kk)
                                tc::mma_ss(tS, qd + (((kk & 3) * 32 + (kk >> 2) * kQHalf) >> 4),
                                           kd + (((kk & 3) * 32 + (kk >> 2) * kHalf) >> 4), kIdQK, kk > 0);
                            tc::commit(&bars[kBarSFull + t]);
                        }
                        __syncwarp();
                    }
                    if (pv) {
                        if (ok && i == 1 && nuse > 0)
                            ok = wait_all(kBarOFree + t, (nuse - 1) & 1);   // O_t of the stream's previous job
                        if (ok) ok = wait_all(kBarPFull + t, npv & 1);
                        if (!ok) break;
                        ++npv;
                        tc::fence_after();
                    }
                    if (!ok) break;
                    if (tc::elect_one()) {
                        if (pv) {
                            const uint64_t vd = v_desc + (uint32_t)st * (kTileBytes >> 4);
#pragma unroll
                            for (int kk = 0; kk < kKeys / 16; ++kk)
                                tc::mma_ts(tO, tP + kk * 8, vd + kk * (2048 >> 4), kIdPV, i > 1 || kk > 0);
                            tc::commit(&bars[kBarPFree + t]);
                            if (i == mine) tc::commit(&bars[kBarOFull + t]);
                        }
                        tc::commit(&bars[kBarEmpty + st]);
                        if (i == nt - 1) tc::commit(&bars[kBarQEmpty]);
                    }
                    __syncwarp();
                }
                nuse += mine > 0;
            }
            // everything issued has completed once this arrives
            if (tc::elect_one()) tc::commit(&bars[kBarIdle + t]);
            __syncwarp();
            if (lane == 0 && !mbar_wait_drain(&bars[kBarIdle + t], 0)) {
                misc->abort = 1;
                flag_error(p.err, PA_DEVERR_TIMEOUT);
            }
            __syncwarp();
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
        // -------------------------------------------------- softmax of stream t
        const int t = warp >> 2, qd = warp & 3;
        const int r = qd * 32 + lane;                       // the thread's row
        const uint32_t lane_off = (uint32_t)(qd * 32) << 16;
        const uint32_t tS = tmem + lane_off + t * TL::kStream, tP = tS + TL::kP, tO = tS + TL::kO;
        // a negative scale is moved into the scores; zero becomes the smallest factor that
        // still sends a masked -inf to -inf
        const bool neg = p.scale_log2 < 0.f;
        const float sl2 = fmaxf(fabsf(p.scale_log2), 1e-37f);
        int ns = 0, nuse = 0;   // tiles and jobs of this stream so far
        bool live = true;
        Job jb;
        for (int k = 0; live && read_job_warp(k, jb); ++k) {
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[kBarRead + (k & 7)]);
            if (jb.ntiles[t] == 0) continue;
            const bool row_ok = r < jb.nrows[t];
            const int tok = jb.i0 + t * kTok + r / G;        // token within the sequence
            const int lim = row_ok ? tok : INT_MAX;          // padding rows mask nothing
            float m = -INFINITY, l = 0.f;
            for (int j = 0; j < jb.ntiles[t]; ++j) {
                live = wait_bar(&bars[kBarSFull + t], ns & 1, misc, p);
                live = __all_sync(kFull, live);
                if (!live) break;
                tc::fence_after();
                const int key0 = j * kKeys;
                float sv[kKeys];
#pragma unroll
                for (int c = 0; c < kKeys; c += 16) tc::ld16(tS + c, sv + c);
                tc::wait_ld();
                tc::fence_before();
                mbar_arrive(&bars[kBarSRead + t]);
                if (neg) {
#pragma unroll
                    for (int i = 0; i < kKeys; ++i) sv[i] = -sv[i];
                }
                if (!__all_sync(kFull, lim >= key0 + kKeys - 1)) {
#pragma unroll
                    for (int i = 0; i < kKeys; ++i) sv[i] = key0 + i <= lim ? sv[i] : -INFINITY;
                }
                float a0 = -INFINITY, a1 = -INFINITY, a2 = -INFINITY, a3 = -INFINITY;
#pragma unroll
                for (int i = 0; i < kKeys; i += 8) {
                    a0 = fmax3(a0, sv[i], sv[i + 1]);
                    a1 = fmax3(a1, sv[i + 2], sv[i + 3]);
                    a2 = fmax3(a2, sv[i + 4], sv[i + 5]);
                    a3 = fmax3(a3, sv[i + 6], sv[i + 7]);
                }
                const float m_new = fmaxf(m, fmaxf(fmax3(a0, a1, a2), a3) * sl2);
                const bool move = j > 0 && row_ok && m_new > m + kRescaleLog2;
                const bool any_move = __any_sync(kFull, move);
                const float m_old = m;
                if (j == 0 || move) m = m_new;
                // P_t may be written, and O_t rescaled, once the stream's last PV is done
                auto own_p = [&]() {
                    if (ns > 0) {
                        live = wait_bar(&bars[kBarPFree + t], (ns - 1) & 1, misc, p);
                        live = __all_sync(kFull, live);
                        if (!live) return;
                        tc::fence_after();
                    }
                    ++ns;
                    if (!any_move) return;
                    const float alpha = move ? fast_exp2(m_old - m) : 1.f;
                    l *= alpha;
#pragma unroll 1
                    for (int c = 0; c < D; c += 16) {
                        float ov[16];
                        tc::ld16(tO + c, ov);
                        tc::wait_ld();
                        uint32_t x[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) x[i] = __float_as_uint(ov[i] * alpha);
                        tc::st16(tO + c, x);
                    }
                };
                const float ref = m == -INFINITY ? 0.f : m;
                const float2 sc2 = make_float2(sl2, sl2), nm2 = make_float2(-ref, -ref);
                float2 acc0 = make_float2(0.f, 0.f), acc1 = acc0;
                uint32_t w[kKeys / 16][8];
#pragma unroll
                for (int c = 0; c < kKeys / 16; ++c) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        float2 x = __ffma2_rn(make_float2(sv[16 * c + 2 * i], sv[16 * c + 2 * i + 1]), sc2, nm2);
                        x.x = fast_exp2(x.x);
                        x.y = fast_exp2(x.y);
                        if (i & 1) acc1 = __fadd2_rn(acc1, x);
                        else acc0 = __fadd2_rn(acc0, x);
                        w[c][i] = pack_bf16x2(x.x, x.y);
                    }
                    if (c + 1 == TL::kAhead) {
                        own_p();
#pragma unroll
                        for (int e = 0; e < c; ++e) tc::st8(tP + e * 8, w[e]);
                    }
                    if (c + 1 >= TL::kAhead) tc::st8(tP + c * 8, w[c]);
                }
                if (!live) break;
                l += (acc0.x + acc0.y) + (acc1.x + acc1.y);
                tc::wait_st();
                tc::fence_before();
                mbar_arrive(&bars[kBarPFull + t]);
            }
            if (!live) break;
            // ---- the output rows
            live = wait_bar(&bars[kBarOFull + t], nuse & 1, misc, p);
            live = __all_sync(kFull, live);
            if (!live) break;
            ++nuse;
            tc::fence_after();
            const float inv = l > 0.f ? 1.f / l : l;      // NaN stays NaN
            // Through shared memory, so that a store covers whole 128-byte lines (a row per
            // thread and store would touch 32 of them).
            unsigned char *stage = smem + SM::kOut + warp * kOutBytes;
            const uint32_t head_bytes = D * 2, tok_bytes = (uint32_t)p.num_q_heads * head_bytes;
            unsigned char *out0 = p.out + (int64_t)(jb.row0 + jb.i0 + t * kTok) * tok_bytes + jb.h * G * head_bytes +
                                  (lane & 7) * 16;
            const float2 inv2 = make_float2(inv, inv), zero2 = make_float2(0.f, 0.f);
            float2 bad0 = zero2, bad1 = zero2;           // NaN once anything is not finite
#pragma unroll
            for (int c = 0; c < D; c += 64) {
                float o[64];
#pragma unroll
                for (int x = 0; x < 64; x += 16) tc::ld16(tO + c + x, o + x);
                tc::wait_ld();
#pragma unroll
                for (int x = 0; x < 8; ++x) {
                    uint32_t w[4];
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        const float2 v = __fmul2_rn(make_float2(o[8 * x + 2 * y], o[8 * x + 2 * y + 1]), inv2);
                        if (y & 1) bad1 = __ffma2_rn(v, zero2, bad1);
                        else bad0 = __ffma2_rn(v, zero2, bad0);
                        w[y] = pack_bf16x2(v.x, v.y);
                    }
                    *reinterpret_cast<uint4 *>(stage + lane * 128 + ((x ^ (lane & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
                }
                if (c + 64 >= D) {       // O_t has been read
                    tc::fence_before();
                    mbar_arrive(&bars[kBarOFree + t]);
                }
                __syncwarp();
                uint4 w[8];
#pragma unroll
                for (int x = 0; x < 8; ++x) {
                    const int rl = 4 * x + (lane >> 3);                      // row of the warp
                    w[x] = *reinterpret_cast<const uint4 *>(stage + rl * 128 + (((lane & 7) ^ (rl & 7)) << 4));
                }
#pragma unroll
                for (int x = 0; x < 8; ++x) {
                    const int rr = qd * 32 + 4 * x + (lane >> 3);            // row of the tile
                    if (rr < jb.nrows[t])
                        *reinterpret_cast<uint4 *>(out0 + ((uint32_t)(rr / G) * tok_bytes + (rr % G) * head_bytes) + c * 2) = w[x];
                }
                __syncwarp();
            }
            const bool odd = (bad0.x + bad0.y) + (bad1.x + bad1.y) != 0.f;
            const unsigned again = __ballot_sync(kFull, odd && r < jb.nrows[t]);
            if (again)
                redo_rows<D, G>(p, jb.row0, jb.i0 + t * kTok + qd * 32 / G, jb.h, min(jb.nkeys, jb.ntiles[t] * kKeys), again,
                                misc);
        }
    }
    tc::fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc::fence_after();
        tc::dealloc(tmem, TL::kCols);
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
    // no sequence has more tokens than there are rows, whatever the caller's upper bound is
    const int32_t max_len = std::min(a.max_seq_len, a.num_tokens);
    if (jobs * a.num_kv_heads >= kManyPairs) return cudaErrorNotSupported;
    PlanParams pl;
    pl.starts = a.starts;
    pl.meta = static_cast<int32_t *>(a.workspace);
    pl.jobs = reinterpret_cast<int4 *>(static_cast<char *>(a.workspace) + 16);
    pl.err = a.err;
    pl.num_seqs = a.num_seqs;
    pl.num_tokens = a.num_tokens;
    pl.max_len = max_len;
    pl.pair_tokens = 2 * kTile / g;
    pl.max_jobs = (int32_t)jobs;
    Params p;
    std::memset(&p, 0, sizeof(p));
    const uint64_t T = (uint64_t)a.num_tokens;
    const uint32_t keys = d == 128 ? Tiles<128>::kKeys : Tiles<64>::kKeys;
    if (!encode_map(&p.qmap, a.query, d, (uint64_t)a.num_q_heads, T, (uint64_t)a.q_stride * 2, (uint32_t)g, kTile / g) ||
        !encode_map(&p.kmap, a.key, d, (uint64_t)a.num_kv_heads, T, (uint64_t)a.k_stride * 2, 1, keys) ||
        !encode_map(&p.vmap, a.value, d, (uint64_t)a.num_kv_heads, T, (uint64_t)a.v_stride * 2, 1, keys))
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
    p.num_seqs = a.num_seqs;
    p.num_tokens = a.num_tokens;
    p.max_len = max_len;
    p.wait_ns = wait_limit_ns();
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    // Where no sequence has more than one pair of row tiles, and a CTA at most kDirectJobs jobs,
    // the CTAs take (sequence, kv head) in turn and no list is made: without the first kernel 24
    // prompts of up to 64 tokens take 11.6 us instead of 14.8, 40 of 200 to 256 tokens 26.1 instead of 29.2
    // (1.3 and 2.2 jobs a CTA); with more jobs handing them out evens the CTAs (22 a CTA: 87 us
    // with the list, 89 without; 108: 392 and 416).
    const int64_t direct = (int64_t)a.num_seqs * a.num_kv_heads;
    if (max_len <= pl.pair_tokens && direct <= (int64_t)kDirectJobs * num_sms(dev)) {
        p.starts = a.starts;
        const int grid = (int)std::min<int64_t>(direct, num_sms(dev));
        return d == 128 ? launch_group<128>(p, g, grid, stream) : launch_group<64>(p, g, grid, stream);
    }
    const size_t plan_smem = (size_t)(a.num_seqs + 1) * 4;
    if (plan_smem > 46 * 1024) {   // with its static arrays above what a launch may ask for anyway
        e = cudaFuncSetAttribute(packed_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (kMaxPlanSeqs + 1) * 4);
        if (e != cudaSuccess) return e;
    }
    packed_plan_kernel<<<1, kPlanThreads, plan_smem, stream>>>(pl);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    const int grid = (int)std::min<int64_t>(jobs * a.num_kv_heads, num_sms(dev));
    return d == 128 ? launch_group<128>(p, g, grid, stream) : launch_group<64>(p, g, grid, stream);
}

}  // namespace pa
