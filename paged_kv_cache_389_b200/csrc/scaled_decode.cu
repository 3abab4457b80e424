// Decode attention (one query token per sequence) over an 8-bit KV cache with one
// scale per (block, kv head).
//
// What is computed (include/pa.h), for query head hq of kv head h = hq / g:
//   s_t = scale * sigma_k(b, h) * <q, kcode_t>,   b = table[t / 16]
//   out = sum_t softmax_t(s) sigma_v(b, h) vcode_t
// online, in units of log2: with a reference point m of the scores and a second one,
// mo, of the scores plus log2(sigma_v), each token adds p = 2^(s - m) to l and
// w = p * sigma_v * 2^(m - mo) times its codes to O, so that the size of a block's values
// neither overflows the 16-bit operands of the tensor cores nor costs it bits: what counts is
// w beside the row's largest.  out = O / l * 2^(mo - m).  Both points move only when a p or a
// w has grown by 2^8 (a vote per block), so the reductions over lanes are rare.
// Where sigma_v 2^(m - mo) is so large that a p of zero may belong to a w that is
// not, w is computed as 2^(s + log2(sigma_v) - mo) instead.  Sums, maxima and O are fp32; w is
// rounded to f16 for the product with V (relative 2^-11; a w below 2^-21 of the row's
// largest is off by up to 2^-32 of that one); codes are exact in f16; the query is scaled per
// head by a power of two into the middle of f16's range, which keeps every bf16 bit of its elements
// down to 2^-24 of the head's largest (smaller ones are off by at most 2^-32 of it).
//
// What bounds it: HBM, 2 * L * Hkv * d bytes (in a graph: 256 lognormal contexts, 32/8 heads, e4m3, 1.08
// GB: 190 us, 5.7 TB/s; 64 contexts, 32/32 heads, int8, 0.58 GB: 102 us; 8 x 32768 tokens, 64/8
// heads, 0.54 GB: 100 us).  So:
//  * Work is cut evenly whatever the lengths are: the blocks of all (sequence, kv head)
//    segments form one line (each segment followed by one empty item that stands for
//    its fixed cost), and warp w of the grid takes items [w n, (w + 1) n).  No unit is
//    longer than another, few long contexts fill the GPU as many short ones do, and the
//    cut is computed on the device from the lengths (a captured graph follows them).
//  * A warp streams its blocks through a ring of its own (16-byte cp.async, the next
//    blocks and their scales in flight while one is computed): 12 warps with 8 KB each
//    are 96 KB in flight per SM; nothing is shared between warps while they stream.  (16 warps of
//    128 registers or a third stage only lengthened the queue to memory: 200 and 201 us
//    against 193 for 256 lognormal contexts, 1.08 GB.)
//  * A segment that lies within one warp's items is written out at once.  Parts of
//    segments at the ends of a warp's items meet in shared memory when the CTA's warps
//    are done, and only parts at the ends of a CTA's items go through the workspace (two
//    per CTA, whatever the context) to a second kernel.  Where all contexts are short, CTAs
//    take whole segments and there is no second kernel.
//  * What is left (figures of the 1.08 GB case): the median warp is done after 159 us, at
//    6.9 TB/s, the last after 183: the same 28 SMs in every run get 8 % less of the memory than
//    the others, and an even cut waits for them.  Drawing the last eighth of the line in units from a
//    counter brought the ends together (163 to 178 us) but cost more, in moving between units, in the
//    counter's zeroing and in joining the units' parts: 195 us against 190.
//  * QK^T as S^T = K Q^T and PV as O^T = V^T W^T on m16n8k16 f16 tiles with the
//    block's 16 tokens (or 16 head dims) in M and the g heads in N: each thread reads
//    whole 16-byte pieces of the code rows and widens them in registers.
#include <algorithm>
#include <cfloat>
#include <climits>
#include <cstring>

#include "pa_common.cuh"
#include "pa_launch.h"
#include "pa_step.h"

namespace pa {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kWarps = 12;
constexpr int kThreads = kWarps * 32;
// The reference points lie 2^kHead below the largest p and w when they move, and move again when one has
// grown by 2^8: p and w reach 2^15, inside f16's range, and w loses bits (below f16's normal numbers, 2^-14)
// only where it is less than 2^-21 of the row's largest.
constexpr float kHead = 7.f, kLazy = 32768.f;
constexpr float kFactor = 0x1p100f;   // p below 2^-126 is zero: with a factor up to this, so is its w for f16
constexpr int kMaxCum = 8192;         // prefix-sum entries in shared memory (every k-th sequence beyond)
constexpr int kWholeItems = 33;       // longest segments that stay within a CTA
constexpr int kMergeThreads = 256;

template <int D, int G>
struct Lay {
    static constexpr int kSlab = kBlockSize * D;              // codes of one (block, kv head)
    static constexpr int kStage = 2 * kSlab + 16;             // K, V, the two scales
    static constexpr int kStages = D == 128 ? 2 : 4;
    static constexpr int kPiece = G * D * 4 + G * 12 + (16 - (G * 12) % 16) % 16;  // O, then (m, l, mo) per head
    static constexpr size_t kRing = (size_t)kWarps * kStages * kStage;
    static constexpr size_t kOffA = kRing;                    // first parts
    static constexpr size_t kOffB = 0;                        // last parts: over the ring, once it is idle
    static constexpr size_t kOffSeg = kOffA + (size_t)kWarps * kPiece;   // int [2 * kWarps] twice: segments, order
    static constexpr size_t kOffScratch = kOffSeg + 4 * kWarps * 4;      // uint [kWarps + 2]
    static constexpr size_t kOffCum = kOffScratch + 96;
    static constexpr size_t bytes(int cum) { return kOffCum + (size_t)cum * 4; }
    static_assert((size_t)kWarps * kPiece <= kRing, "the last parts fit the ring");
    static_assert(kStage % 16 == 0 && kPiece % 16 == 0 && kOffA % 16 == 0 && kOffSeg % 16 == 0, "aligned fields");
    static_assert(kOffCum + (kMaxCum + 1) * 4 <= 232448, "shared memory of an sm_100 CTA");
};

struct Params {
    const unsigned char *q, *kc, *vc;
    const float *ks, *vs;
    const int32_t *tables, *lens;
    unsigned char *out;
    unsigned char *parts;    // workspace: [ctas][2] parts
    int4 *tails;             // workspace: [ctas] (segment, last CTA of it, 0, 0) of the last, unfinished segment
    int32_t *err;
    int32_t max_blocks, max_context, num_seqs, num_q_heads, num_kv_heads, num_blocks;
    int32_t cum_step;        // sequences per prefix-sum entry
    bool whole;              // CTAs take whole segments: nothing to join afterwards
    float scale_log2;
};

__device__ __forceinline__ int checked_len(const Params &p, int s) {
    const int L = __ldg(p.lens + s);
    return L < 0 || L > p.max_context || (int64_t)L > (int64_t)p.max_blocks * kBlockSize ? -1 : L;
}
__device__ __forceinline__ int blocks_of(int tokens) { return tokens > 0 ? (tokens - 1) / kBlockSize + 1 : 0; }

// Four codes -> two f16x2 (bytes 0, 1 and bytes 2, 3).
template <bool kInt8>
__device__ __forceinline__ void widen4(uint32_t w, uint32_t &lo, uint32_t &hi) {
    if constexpr (kInt8) {
        // 0x64uu is the f16 number 1024 + uu: with uu = code + 128, minus 1152 (exact)
        const uint32_t u = w ^ 0x80808080u;
        lo = __byte_perm(u, 0x64646464u, 0x4140);
        hi = __byte_perm(u, 0x64646464u, 0x4342);
        asm("sub.f16x2 %0, %0, %1;" : "+r"(lo) : "r"(0x64806480u));
        asm("sub.f16x2 %0, %0, %1;" : "+r"(hi) : "r"(0x64806480u));
    } else {
        asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
            "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
            : "=r"(lo), "=r"(hi)
            : "r"(w));
    }
}

// 16-byte chunk c of row r of a slab sits at chunk position c ^ swz(r): conflict-free
// reads of one chunk column over rows.
template <int D>
__device__ __forceinline__ int swz(int r) {
    return D == 128 ? (r & 7) : ((r >> 1) & 3);
}

__device__ __forceinline__ void cp_async4(uint32_t dst_smem, const void *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst_smem), "l"(src) : "memory");
}

// A warp's running state.  Columns (heads) 2t and 2t + 1 of lane 4 g + t; m, mo are
// uniform over the 8 lanes of a column pair, l is this thread's share of the sum.
template <int D>
struct State {
    float m[2], mo[2], l[2];
    float gf[2];             // 2^(m - mo)
    float c[2];              // score units: log2(e) * scale * (the query head's power of two)
    float o[D / 16][4];      // rows d0 + 2 mt and d0 + 2 mt + 1 with d0 = g * D / 8; columns 2t, 2t + 1
    uint32_t q[D / 16][2];
};

template <int D>
__device__ __forceinline__ void reset(State<D> &st) {
    st.m[0] = st.m[1] = st.mo[0] = st.mo[1] = -INFINITY;
    st.l[0] = st.l[1] = 0.f;
    st.gf[0] = st.gf[1] = 0.f;
#pragma unroll
    for (int i = 0; i < D / 16; ++i) st.o[i][0] = st.o[i][1] = st.o[i][2] = st.o[i][3] = 0.f;
}

// The query heads of a segment as f16 operand fragments: thread (g, t) holds dims
// (D/4) t + 16 j + 4 i + {0, 1} and + {2, 3} of head g for k step 4 j + i.
template <int D, int G>
__device__ __forceinline__ void load_q(const Params &p, int s, int h, State<D> &st, int lane) {
    const int gr = lane >> 2, t = lane & 3;
    uint2 w[D / 16];
    float big = 0.f;
    const unsigned char *src =
        p.q + (((int64_t)s * p.num_q_heads + (int64_t)h * G + gr) * D + (D / 4) * t) * 2;
#pragma unroll
    for (int i = 0; i < D / 16; i += 2) {
        uint4 x = make_uint4(0, 0, 0, 0);
        if (gr < G) x = __ldg(reinterpret_cast<const uint4 *>(src + i * 8));
        w[i] = make_uint2(x.x, x.y);
        w[i + 1] = make_uint2(x.z, x.w);
    }
    float2 a[D / 16][2];
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
        a[i][0] = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&w[i].x));
        a[i][1] = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&w[i].y));
        big = fmaxf(fmaxf(big, fmaxf(fabsf(a[i][0].x), fabsf(a[i][0].y))), fmaxf(fabsf(a[i][1].x), fabsf(a[i][1].y)));
    }
    big = fmaxf(big, __shfl_xor_sync(kFull, big, 1));
    big = fmaxf(big, __shfl_xor_sync(kFull, big, 2));
    // a power of two that brings the head's largest element to [2^7, 2^8)
    int e = (__float_as_int(big) >> 23) - 127 - 7;
    e = max(-126, min(e, 126));
    if (big == 0.f) e = 0;
    const float down = __int_as_float((127 - e) << 23);
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
        st.q[i][0] = pack_f16x2(a[i][0].x * down, a[i][0].y * down);
        st.q[i][1] = pack_f16x2(a[i][1].x * down, a[i][1].y * down);
    }
    // the power of two back into the scores, for this thread's two columns
    const float up = __int_as_float((127 + e) << 23);
#pragma unroll
    for (int k = 0; k < 2; ++k) st.c[k] = p.scale_log2 * __shfl_sync(kFull, up, (2 * t + k) * 4);
}

__device__ __forceinline__ float fmax3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// One 16-token block; kTail: only ntok (1 .. 15) of them are in the context.
template <int D, bool kInt8, bool kTail>
__device__ __forceinline__ void block_step(unsigned char *stage, const float2 sc, int ntok, State<D> &st, int lane) {
    constexpr int kSlab = kBlockSize * D;
    constexpr int kVBytes = D / 8;   // bytes of a V row per thread
    const int g = lane >> 2, t = lane & 3;
    float sx[4][4] = {};   // four chains of k steps
#pragma unroll
    for (int j = 0; j < D / 64; ++j) {
        const int ch = (D / 64) * t + j;
        // swz(g + 8) == swz(g)
        const unsigned char *row = stage + g * D + ((ch ^ swz<D>(g)) << 4);
        const uint4 lo = *reinterpret_cast<const uint4 *>(row);
        const uint4 hi = *reinterpret_cast<const uint4 *>(row + 8 * D);
        const uint32_t wl[4] = {lo.x, lo.y, lo.z, lo.w}, wh[4] = {hi.x, hi.y, hi.z, hi.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int kk = 4 * j + i;
            uint32_t a[4];
            widen4<kInt8>(wl[i], a[0], a[2]);
            widen4<kInt8>(wh[i], a[1], a[3]);
            mma_f16_16816(sx[kk & 3], a, st.q[kk][0], st.q[kk][1]);
        }
    }
    float s[4], pr[4], w[4];
    const float c0 = st.c[0] * sc.x, c1 = st.c[1] * sc.x;
#pragma unroll
    for (int i = 0; i < 4; ++i) s[i] = (sx[0][i] + sx[1][i]) + (sx[2][i] + sx[3][i]);
    if constexpr (kTail) {
        // a masked score is -inf whatever the sign of the factor
        const float n0 = c0 < 0.f ? INFINITY : -INFINITY, n1 = c1 < 0.f ? INFINITY : -INFINITY;
        if (g >= ntok) s[0] = n0, s[1] = n1;
        if (g + 8 >= ntok) s[2] = n0, s[3] = n1;
    }
    auto probabilities = [&]() {
#pragma unroll
        for (int i = 0; i < 4; ++i) pr[i] = fast_exp2(fmaf(s[i], i & 1 ? c1 : c0, -st.m[i & 1]));
        if constexpr (kTail) {   // a factor of zero would make the masked ones NaN
            if (g >= ntok) pr[0] = pr[1] = 0.f;
            if (g + 8 >= ntok) pr[2] = pr[3] = 0.f;
        }
    };
    probabilities();
    const float f0 = sc.y * st.gf[0], f1 = sc.y * st.gf[1];
    w[0] = pr[0] * f0;
    w[1] = pr[1] * f1;
    w[2] = pr[2] * f0;
    w[3] = pr[3] * f1;
    // Where the factor is above kFactor (block scales that far apart), a p of zero may stand for a w
    // that is not: those blocks take the branch below, where w has an exponential of its own.
    const float a = fmax3(fmax3(pr[0], pr[1], pr[2]), pr[3], w[0]);
    const float b = fmax3(w[1], w[2], w[3]);
    // m is -inf until the first block: the exponentials are then infinite or NaN
    const bool fine = fmax3(a, b, fmaxf(f0, f1) * (kLazy / kFactor)) <= kLazy && st.m[0] != -INFINITY;
    if (!__all_sync(kFull, fine)) {
        // move the reference points: the largest score so far, and the largest score plus log2(sigma_v)
        float x0 = -INFINITY, x1 = -INFINITY;
        if (!kTail || g < ntok) {
            x0 = s[0] * c0;
            x1 = s[1] * c1;
        }
        if (!kTail || g + 8 < ntok) {
            x0 = fmaxf(x0, s[2] * c0);
            x1 = fmaxf(x1, s[3] * c1);
        }
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) {
            x0 = fmaxf(x0, __shfl_xor_sync(kFull, x0, off));
            x1 = fmaxf(x1, __shfl_xor_sync(kFull, x1, off));
        }
        const float log_v = __log2f(sc.y), lv = fmaxf(log_v, -100.f);   // m - mo is at most 100
        const float x[2] = {x0, x1};
        float ao[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const float m = fmaxf(st.m[k], x[k] - kHead), mo = fmaxf(st.mo[k], x[k] + lv - kHead);
            const float al = st.m[k] == -INFINITY ? 0.f : fast_exp2(st.m[k] - m);
            ao[k] = st.mo[k] == -INFINITY ? 0.f : fast_exp2(st.mo[k] - mo);
            // no finite score yet: any finite reference will do
            st.m[k] = m == -INFINITY ? -FLT_MAX : m;
            st.mo[k] = m == -INFINITY ? -FLT_MAX : mo;
            st.gf[k] = fast_exp2(st.m[k] - st.mo[k]);
            st.l[k] *= al;
        }
#pragma unroll
        for (int mt = 0; mt < D / 16; ++mt) {
            st.o[mt][0] *= ao[0];
            st.o[mt][1] *= ao[1];
            st.o[mt][2] *= ao[0];
            st.o[mt][3] *= ao[1];
        }
        probabilities();
        const float v0 = log_v - st.mo[0], v1 = log_v - st.mo[1];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = fast_exp2(fmaf(s[i], i & 1 ? c1 : c0, i & 1 ? v1 : v0));
        if constexpr (kTail) {
            if (g >= ntok) w[0] = w[1] = 0.f;
            if (g + 8 >= ntok) w[2] = w[3] = 0.f;
        }
    }
    st.l[0] += pr[0] + pr[2];
    st.l[1] += pr[1] + pr[3];
    const uint32_t pb0 = movmatrix_trans(pack_f16x2(w[0], w[1]));
    const uint32_t pb1 = movmatrix_trans(pack_f16x2(w[2], w[3]));
    unsigned char *vb = stage + kSlab;
    if constexpr (kTail) {
        // codes past the context may stand for NaN: zero those rows
        for (int i = lane; i < (kBlockSize - ntok) * (D / 16); i += 32)
            *reinterpret_cast<uint4 *>(vb + (ntok + i / (D / 16)) * D + (i % (D / 16)) * 16) = make_uint4(0, 0, 0, 0);
        __syncwarp();
    }
    uint32_t r[4][kVBytes / 4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int row = 2 * t + (k & 1) + 8 * (k >> 1);
        if constexpr (D == 128) {
            const uint4 v = *reinterpret_cast<const uint4 *>(vb + row * D + ((g ^ swz<D>(row)) << 4));
            r[k][0] = v.x; r[k][1] = v.y; r[k][2] = v.z; r[k][3] = v.w;
        } else {
            const uint2 v = *reinterpret_cast<const uint2 *>(vb + row * D + (((g >> 1) ^ swz<D>(row)) << 4) + (g & 1) * 8);
            r[k][0] = v.x; r[k][1] = v.y;
        }
    }
#pragma unroll
    for (int i = 0; i < kVBytes / 4; ++i) {
        // token pairs (2t, 2t+1) and (2t+8, 2t+9) of dims 4i + {0, 1}, then 4i + {2, 3}
        uint32_t a[4];
        widen4<kInt8>(__byte_perm(r[0][i], r[1][i], 0x5140), a[0], a[1]);
        widen4<kInt8>(__byte_perm(r[2][i], r[3][i], 0x5140), a[2], a[3]);
        mma_f16_16816(st.o[2 * i], a, pb0, pb1);
        widen4<kInt8>(__byte_perm(r[0][i], r[1][i], 0x7362), a[0], a[1]);
        widen4<kInt8>(__byte_perm(r[2][i], r[3][i], 0x7362), a[2], a[3]);
        mma_f16_16816(st.o[2 * i + 1], a, pb0, pb1);
    }
}

// Sum of l over the 8 lanes of each column.
template <int D>
__device__ __forceinline__ void sum_l(State<D> &st) {
#pragma unroll
    for (int off = 4; off < 32; off <<= 1) {
        st.l[0] += __shfl_xor_sync(kFull, st.l[0], off);
        st.l[1] += __shfl_xor_sync(kFull, st.l[1], off);
    }
}

// A finished segment's output rows, straight from the registers.
template <int D, int G>
__device__ __forceinline__ void write_out(const Params &p, int seg, State<D> &st, int lane) {
    sum_l(st);
    const int g = lane >> 2, t = lane & 3;
    const int s = seg / p.num_kv_heads, h = seg - s * p.num_kv_heads;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int head = 2 * t + k;
        if (head >= G) continue;
        const float f = st.l[k] == 0.f ? 0.f : fast_exp2(st.mo[k] - st.m[k]) / st.l[k];
        unsigned char *dst = p.out + (((int64_t)s * p.num_q_heads + (int64_t)h * G + head) * D + g * (D / 8)) * 2;
#pragma unroll
        for (int mt = 0; mt < D / 16; mt += 4) {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = pack_bf16x2(st.o[mt + i][k] * f, st.o[mt + i][2 + k] * f);
            *reinterpret_cast<uint4 *>(dst + mt * 4) = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
}

// A part of a segment: O [G][D], then (m, l, mo) of each head.
template <int D, int G>
__device__ __forceinline__ void write_part(unsigned char *dst, State<D> &st, int lane) {
    sum_l(st);
    const int g = lane >> 2, t = lane & 3;
    float *o = reinterpret_cast<float *>(dst), *ml = o + G * D;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int head = 2 * t + k;
        if (head >= G) continue;
        float *row = o + head * D + g * (D / 8);
#pragma unroll
        for (int mt = 0; mt < D / 16; mt += 2)
            *reinterpret_cast<float4 *>(row + 2 * mt) =
                make_float4(st.o[mt][k], st.o[mt][2 + k], st.o[mt + 1][k], st.o[mt + 1][2 + k]);
        if (g == 0) {
            ml[3 * head] = st.m[k];
            ml[3 * head + 1] = st.l[k];
            ml[3 * head + 2] = st.mo[k];
        }
    }
}

// The parts part(0) .. part(n - 1) of one segment, head `head`, joined by one warp: lane i
// gets dims (D/32) i .. of the unnormalised sum, and the joint (m, l, mo).
template <int D, int G, typename Part>
__device__ __forceinline__ void join(const Part &part, int n, int head, int lane, float (&acc)[D / 32], float &m,
                                     float &l, float &mo) {
    m = mo = -INFINITY;
    for (int i = lane; i < n; i += 32) {
        const float *ml = part(i) + G * D + 3 * head;
        m = fmaxf(m, ml[0]);
        mo = fmaxf(mo, ml[2]);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
        mo = fmaxf(mo, __shfl_xor_sync(kFull, mo, o));
    }
    l = 0.f;
#pragma unroll
    for (int k = 0; k < D / 32; ++k) acc[k] = 0.f;
    if (m == -INFINITY) return;  // no token at all
#pragma unroll 4
    for (int i = 0; i < n; ++i) {
        const float *o = part(i), *ml = o + G * D + 3 * head;
        const float mi = ml[0], li = ml[1], moi = ml[2];
        const float fl = mi == -INFINITY ? 0.f : fast_exp2(mi - m), fo = moi == -INFINITY ? 0.f : fast_exp2(moi - mo);
        l = fmaf(li, fl, l);
        const float *x = o + head * D + lane * (D / 32);
        if constexpr (D == 128) {
            const float4 v = *reinterpret_cast<const float4 *>(x);
            acc[0] = fmaf(v.x, fo, acc[0]); acc[1] = fmaf(v.y, fo, acc[1]);
            acc[2] = fmaf(v.z, fo, acc[2]); acc[3] = fmaf(v.w, fo, acc[3]);
        } else {
            const float2 v = *reinterpret_cast<const float2 *>(x);
            acc[0] = fmaf(v.x, fo, acc[0]); acc[1] = fmaf(v.y, fo, acc[1]);
        }
    }
}

template <int D, int G>
__device__ __forceinline__ void store_joined(const Params &p, int seg, int head, int lane, const float (&acc)[D / 32],
                                             float m, float l, float mo) {
    const int s = seg / p.num_kv_heads, h = seg - s * p.num_kv_heads;
    const float f = l == 0.f ? 0.f : fast_exp2(mo - m) / l;
    unsigned char *dst = p.out + (((int64_t)s * p.num_q_heads + (int64_t)h * G + head) * D + lane * (D / 32)) * 2;
    if constexpr (D == 128)
        *reinterpret_cast<uint2 *>(dst) = make_uint2(pack_bf16x2(acc[0] * f, acc[1] * f), pack_bf16x2(acc[2] * f, acc[3] * f));
    else
        *reinterpret_cast<uint32_t *>(dst) = pack_bf16x2(acc[0] * f, acc[1] * f);
}

// ---- the line of items --------------------------------------------------------------
// Sequence s owns hkv * (blocks(s) + 1) items: per kv head its blocks, then one empty item.
struct Place {
    int s, h, b, nb;   // sequence, kv head, block (nb: the empty item), the sequence's blocks
};

// cum[i]: sum over sequences s' < i * step of blocks(s') + 1
__device__ __forceinline__ Place place_of(const Params &p, const uint32_t *cum, int ncum, int64_t item) {
    const int hkv = p.num_kv_heads;
    const uint32_t v = (uint32_t)(item / hkv);
    int lo = 0, hi = ncum;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cum[mid] <= v) lo = mid; else hi = mid;
    }
    Place pl;
    pl.s = lo * p.cum_step;
    uint32_t base = cum[lo];
    pl.nb = blocks_of(checked_len(p, pl.s));
    while (v - base > (uint32_t)pl.nb) {  // every step-th sequence has an entry: walk to the one
        base += (uint32_t)pl.nb + 1;
        ++pl.s;
        pl.nb = blocks_of(checked_len(p, pl.s));
    }
    const int64_t r = item - (int64_t)base * hkv;
    pl.h = (int)(r / (pl.nb + 1));
    pl.b = (int)(r - (int64_t)pl.h * (pl.nb + 1));
    return pl;
}

// The next segment.
__device__ __forceinline__ void advance(const Params &p, Place &pl) {
    pl.b = 0;
    if (++pl.h < p.num_kv_heads) return;
    pl.h = 0;
    ++pl.s;
    pl.nb = pl.s < p.num_seqs ? blocks_of(checked_len(p, pl.s)) : 0;
}

template <int D, int G, bool kInt8>
__global__ void __launch_bounds__(kThreads, 1) decode_scaled_kernel(const __grid_constant__ Params p) {
    using L = Lay<D, G>;
    extern __shared__ __align__(128) unsigned char smem[];
    uint32_t *cum = reinterpret_cast<uint32_t *>(smem + L::kOffCum);
    uint32_t *scratch = reinterpret_cast<uint32_t *>(smem + L::kOffScratch);
    int *segs = reinterpret_cast<int *>(smem + L::kOffSeg);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int S = p.num_seqs, hkv = p.num_kv_heads, step = p.cum_step;
    const int ncum = (S + step - 1) / step;
    if (!p.whole) grid_dep_launch();  // the join may be set up; it waits for this grid
    // prefix sums of blocks + 1, one chunk of entries per thread
    {
        const int per = (ncum + kThreads - 1) / kThreads;
        const int beg = min(ncum, (int)threadIdx.x * per), end = min(ncum, beg + per);
        uint32_t sum = 0;
        bool bad = false;
        for (int i = beg; i < end; ++i) {
            uint32_t here = 0;
            for (int s = i * step; s < min(S, (i + 1) * step); ++s) {
                const int len = checked_len(p, s);
                bad |= len < 0;
                here += (uint32_t)blocks_of(len) + 1;
            }
            cum[i] = here;
            sum += here;
        }
        if (bad && blockIdx.x == 0) flag_error(p.err, PA_DEVERR_CONTEXT_LEN);
        uint32_t incl = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t y = __shfl_up_sync(kFull, incl, o);
            if (lane >= o) incl += y;
        }
        if (lane == 31) scratch[warp] = incl;
        __syncthreads();
        uint32_t run = incl - sum;
        for (int w = 0; w < warp; ++w) run += scratch[w];
        for (int i = beg; i < end; ++i) {
            const uint32_t here = cum[i];
            cum[i] = run;
            run += here;
        }
        if (threadIdx.x == kThreads - 1) cum[ncum] = run;
        __syncthreads();
    }
    const int64_t total = (int64_t)cum[ncum] * hkv;
    const int64_t workers = (int64_t)gridDim.x * kWarps;
    // down to one item a warp: four sequences of 17 to 100 tokens take 7.7 us (in a graph), with at
    // least 2, 4, 8 items 9.0, 9.9, 12.1
    const int64_t per = (total + workers - 1) / workers;
    int64_t cta0 = min(total, (int64_t)blockIdx.x * kWarps * per), cta1 = min(total, cta0 + kWarps * per);
    int64_t warp_items = per;
    if (p.whole) {   // both ends move up to where a segment begins
        auto up = [&](int64_t x) -> int64_t {
            if (x >= total) return total;
            const Place pl = place_of(p, cum, ncum, x);
            return pl.b == 0 ? x : x - pl.b + pl.nb + 1;
        };
        cta0 = up(cta0);
        cta1 = up(cta1);
        warp_items = (cta1 - cta0 + kWarps - 1) / kWarps;
    }
    if (cta0 >= cta1) {
        if (threadIdx.x == 0 && !p.whole) p.tails[blockIdx.x] = make_int4(-1, 0, 0, 0);
        return;
    }
    const int64_t w0 = min(cta1, cta0 + warp * warp_items), w1 = min(cta1, w0 + warp_items);
    int seg_a = -1, seg_b = -1;  // segments of this warp's first and last parts
    unsigned char *part_a = smem + L::kOffA + (size_t)warp * L::kPiece;
    State<D> st;
    reset(st);
    if (w0 < w1) {
        unsigned char *ring = smem + (size_t)warp * L::kStages * L::kStage;
        const uint32_t ring_s = smem_u32(ring);
        constexpr int kPerRow = D / 16;   // 16-byte chunks of a row
        const uint32_t lane_off = (uint32_t)((lane / kPerRow) * D + (((lane % kPerRow) ^ swz<D>(lane / kPerRow)) << 4));
        // The fetch cursor: item by item over the warp's blocks.  Lane i of `ent` holds the
        // table entry of block eb + i of its segment; `nxt` those of the 32 after them, or of
        // the next segment's first 32.
        Place fp = place_of(p, cum, ncum, w0);
        int64_t fi = w0;                 // item of the cursor
        const Place first = fp;
        auto entries = [&](int s, int b, int nb) -> int {
            const int j = b + lane;
            return s < S && j < nb ? __ldg(p.tables + (int64_t)s * p.max_blocks + j) : -1;
        };
        int eb = fp.b;
        int ent = entries(fp.s, fp.b, fp.nb);
        Place np = fp;                   // where `nxt` was taken
        auto take_next = [&]() -> int {
            // entries after those of `ent`
            if (eb + 32 < fp.nb) {
                np = fp;
                np.b = eb + 32;
            } else {
                np = fp;
                advance(p, np);
            }
            return entries(np.s, np.b, np.nb);
        };
        int nxt = take_next();
        int n_iss = 0, n_cmp = 0;
        uint32_t okmask = 0;
        // fetch the cursor's block, if any is left; skips the empty items
        auto fetch_one = [&]() -> bool {
            while (fi < w1) {
                if (fp.b >= fp.nb) {     // the empty item: on to the next segment
                    ++fi;
                    if (fi >= w1) return false;
                    fp = np;
                    eb = 0;
                    ent = nxt;
                    nxt = take_next();
                    continue;
                }
                if (fp.b - eb >= 32) {
                    eb += 32;
                    ent = nxt;
                    nxt = take_next();
                }
                const int blk = __shfl_sync(kFull, ent, fp.b - eb);
                const int stage = n_iss % L::kStages;
                const bool ok = blk >= 0 && blk < p.num_blocks;
                if (ok) {
                    const int64_t bh = (int64_t)blk * hkv + fp.h;
                    const unsigned char *ks = p.kc + bh * L::kSlab + lane * 16, *vs = p.vc + bh * L::kSlab + lane * 16;
                    const uint32_t dst = ring_s + stage * L::kStage;
#pragma unroll
                    for (int i = 0; i < L::kSlab / 512; ++i) {
                        // chunk 32 i + lane is in row i * (512 / D) + lane / (D / 16): the row's part of the
                        // swizzle that i sets is bit 2 (d = 128) or none (d = 64)
                        const uint32_t at = dst + i * 512 + (D == 128 && (i & 1) ? lane_off ^ 64u : lane_off);
                        cp_async16(at, ks + i * 512);
                        cp_async16(at + L::kSlab, vs + i * 512);
                    }
                    if (lane < 2) cp_async4(dst + 2 * L::kSlab + lane * 4, (lane == 0 ? p.ks : p.vs) + bh);
                } else if (lane == 0) {
                    flag_error(p.err, PA_DEVERR_BLOCK_ID);
                }
                cp_async_commit();
                okmask = (okmask & ~(1u << stage)) | ((ok ? 1u : 0u) << stage);
                ++fp.b;
                ++fi;
                ++n_iss;
                return true;
            }
            return false;
        };
#pragma unroll 1
        for (int i = 0; i < L::kStages; ++i) fetch_one();
        // the compute cursor
        Place cp = first;
        int64_t ci = w0;
        while (ci < w1) {
            const int seg = cp.s * hkv + cp.h;
            const int len = max(checked_len(p, cp.s), 0);
            const int b_end = (int)min((int64_t)cp.nb, cp.b + (w1 - ci));   // blocks [cp.b, b_end) are this warp's
            const bool ends = cp.nb - cp.b < w1 - ci;                       // the empty item too
            const bool whole = cp.b == 0 && ends;
            if (b_end > cp.b) load_q<D, G>(p, cp.s, cp.h, st, lane);
            const int b_tail = len % kBlockSize != 0 ? cp.nb - 1 : INT_MAX;   // the partly filled block
            for (int b = cp.b; b < b_end; ++b) {
                cp_async_wait_dyn(n_iss - n_cmp - 1);
                __syncwarp();
                const int stage = n_cmp % L::kStages;
                if (okmask >> stage & 1u) {
                    unsigned char *at = ring + stage * L::kStage;
                    const float2 sc = *reinterpret_cast<const float2 *>(at + 2 * L::kSlab);
                    if (b != b_tail) block_step<D, kInt8, false>(at, sc, kBlockSize, st, lane);
                    else block_step<D, kInt8, true>(at, sc, len - b * kBlockSize, st, lane);
                }
                __syncwarp();
                ++n_cmp;
                fetch_one();
            }
            ci += (b_end - cp.b) + (ends ? 1 : 0);
            if (whole) {
                write_out<D, G>(p, seg, st, lane);
                reset(st);
            } else if (ci < w1) {
                seg_a = seg;   // a first part: segments follow
                write_part<D, G>(part_a, st, lane);
                reset(st);
            } else {
                seg_b = seg;   // the last one: kept until the ring is idle
            }
            advance(p, cp);
        }
    }
    if (lane == 0) {
        segs[2 * warp] = seg_a;
        segs[2 * warp + 1] = seg_b;
    }
    __syncthreads();  // no ring in use any more
    if (seg_b >= 0) write_part<D, G>(smem + L::kOffB + (size_t)warp * L::kPiece, st, lane);
    __syncthreads();
    // ---- the CTA's parts: runs of one segment, joined; those that reach beyond the
    // CTA's items go to the workspace
    const int mine = lane < 2 * kWarps ? segs[lane] : -1;   // parts in item order
    static_assert(2 * kWarps <= 32, "one lane per part");
    const unsigned have = __ballot_sync(kFull, mine >= 0);
    const unsigned before = have & ((1u << lane) - 1u);
    const int prev = __shfl_sync(kFull, mine, before ? 31 - __clz(before) : lane);
    unsigned starts = __ballot_sync(kFull, mine >= 0 && (!before || prev != mine));
    // order[i]: the i-th part (every warp writes the same list)
    int *order = segs + 2 * kWarps;
    if (mine >= 0) order[__popc(before)] = lane;
    __syncwarp();
    const int ngroups = __popc(starts);
    bool tail = false;
    for (int task = warp, group = 0; task < ngroups * G; task += kWarps) {
        const int head = task % G;
        for (; group < task / G; ++group) starts &= starts - 1;   // the group's first part is the lowest bit
        const int lo = __ffs(starts) - 1;
        const unsigned later = starts & (starts - 1);
        const int r0 = __popc(have & ((1u << lo) - 1u));
        const int r1 = later ? __popc(have & ((1u << (__ffs(later) - 1)) - 1u)) : __popc(have);
        const int seg = __shfl_sync(kFull, mine, lo);
        auto part = [&](int i) -> const float * {
            const int at = order[r0 + i];
            return reinterpret_cast<const float *>(smem + ((at & 1) ? L::kOffB : L::kOffA) + (size_t)(at >> 1) * L::kPiece);
        };
        float acc[D / 32], m, l, mo;
        join<D, G>(part, r1 - r0, head, lane, acc, m, l, mo);
        // the segment's items
        const int s = seg / hkv, h = seg - s * hkv;
        uint32_t base = cum[s / step];
        for (int x = s / step * step; x < s; ++x) base += (uint32_t)blocks_of(checked_len(p, x)) + 1;
        const int64_t n1 = blocks_of(checked_len(p, s)) + 1;
        const int64_t i0 = (int64_t)base * hkv + h * n1, i1 = i0 + n1;
        if (i0 >= cta0 && i1 <= cta1) {
            store_joined<D, G>(p, seg, head, lane, acc, m, l, mo);
        } else {
            const int slot = i0 < cta0 ? 0 : 1;
            float *dst = reinterpret_cast<float *>(p.parts + ((size_t)blockIdx.x * 2 + slot) * L::kPiece);
            if constexpr (D == 128)
                *reinterpret_cast<float4 *>(dst + head * D + lane * 4) = make_float4(acc[0], acc[1], acc[2], acc[3]);
            else
                *reinterpret_cast<float2 *>(dst + head * D + lane * 2) = make_float2(acc[0], acc[1]);
            if (lane == 0) {
                dst[G * D + 3 * head] = m;
                dst[G * D + 3 * head + 1] = l;
                dst[G * D + 3 * head + 2] = mo;
            }
            if (slot == 1 && head == 0) {
                tail = true;
                if (lane == 0)
                    p.tails[blockIdx.x] = make_int4(seg, (int)((i1 - 1) / (kWarps * per)), 0, 0);
            }
        }
    }
    if (p.whole) return;
    // exactly one warp writes the CTA's tail record
    if (!__syncthreads_or(tail) && threadIdx.x == 0) p.tails[blockIdx.x] = make_int4(-1, 0, 0, 0);
}

// Segments that span CTAs: block c joins the one that begins in CTA c and ends beyond it.
template <int D, int G>
__global__ void __launch_bounds__(kMergeThreads) join_scaled_kernel(const __grid_constant__ Params p) {
    using L = Lay<D, G>;
    grid_dep_wait();
    const int4 t = p.tails[blockIdx.x];
    if (t.x < 0) return;
    const int lane = threadIdx.x & 31, first = (int)blockIdx.x;
    auto part = [&](int i) -> const float * {
        return reinterpret_cast<const float *>(p.parts + ((size_t)(first + i) * 2 + (i == 0 ? 1 : 0)) * L::kPiece);
    };
    for (int head = threadIdx.x >> 5; head < G; head += kMergeThreads / 32) {
        float acc[D / 32], m, l, mo;
        join<D, G>(part, t.y - first + 1, head, lane, acc, m, l, mo);
        store_joined<D, G>(p, t.x, head, lane, acc, m, l, mo);
    }
}

// Workspace bytes for a grid of `ctas`: tail records, then two parts per CTA.
size_t workspace_bytes(int ctas, int g, int d) {
    const size_t piece = (size_t)g * d * 4 + ((size_t)g * 12 + 15) / 16 * 16;
    return (size_t)ctas * 16 + (size_t)ctas * 2 * piece;
}

template <int D, int G, bool kInt8>
cudaError_t launch(Params &p, void *workspace, int ctas, cudaStream_t stream) {
    using L = Lay<D, G>;
    p.tails = static_cast<int4 *>(workspace);
    p.parts = static_cast<unsigned char *>(workspace) + (size_t)ctas * 16;
    p.cum_step = (p.num_seqs + kMaxCum - 1) / kMaxCum;
    const int ncum = (p.num_seqs + p.cum_step - 1) / p.cum_step;
    cudaError_t e = cudaFuncSetAttribute(decode_scaled_kernel<D, G, kInt8>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)L::bytes(kMaxCum + 1));
    if (e != cudaSuccess) return e;
    // Segments of at most kWholeItems items (contexts of up to 511 tokens) stay within a CTA, which costs a CTA
    // at most one segment more than its share and saves the second kernel (four
    // sequences of 17 to 100 tokens: 9.1 us against 9.6 in a graph, at two items a warp).
    p.whole = p.max_context / kBlockSize + 2 <= kWholeItems;
    decode_scaled_kernel<D, G, kInt8><<<(unsigned)ctas, kThreads, L::bytes(ncum + 1), stream>>>(p);
    if ((e = cudaGetLastError()) != cudaSuccess || p.whole) return e;
    return launch_after(join_scaled_kernel<D, G>, dim3((unsigned)ctas), dim3(kMergeThreads), 0, stream,
                        static_cast<const Params &>(p));
}

template <int D, int G>
cudaError_t launch_code(Params &p, bool int8, void *workspace, int ctas, cudaStream_t stream) {
    return int8 ? launch<D, G, true>(p, workspace, ctas, stream) : launch<D, G, false>(p, workspace, ctas, stream);
}

template <int D>
cudaError_t launch_group(Params &p, bool int8, void *workspace, int ctas, cudaStream_t stream) {
    switch (p.num_q_heads / p.num_kv_heads) {
        case 1: return launch_code<D, 1>(p, int8, workspace, ctas, stream);
        case 2: return launch_code<D, 2>(p, int8, workspace, ctas, stream);
        case 4: return launch_code<D, 4>(p, int8, workspace, ctas, stream);
        case 8: return launch_code<D, 8>(p, int8, workspace, ctas, stream);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace

// Two parts per SM of the largest device this code is built for; a device with more
// SMs runs a grid of this many CTAs.
constexpr int kMaxCtas = 160;

size_t scaled_decode_workspace(int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim) {
    return workspace_bytes(kMaxCtas, num_q_heads / num_kv_heads, head_dim);
}

cudaError_t launch_decode_scaled(const ScaledDecode &a, cudaStream_t stream) {
    Params p;
    std::memset(&p, 0, sizeof(p));
    p.q = static_cast<const unsigned char *>(a.query);
    p.kc = static_cast<const unsigned char *>(a.pool.kc);
    p.vc = static_cast<const unsigned char *>(a.pool.vc);
    p.ks = a.pool.ks;
    p.vs = a.pool.vs;
    p.tables = a.tables;
    p.lens = a.lens;
    p.out = static_cast<unsigned char *>(a.out);
    p.err = a.err;
    p.max_blocks = a.max_blocks;
    p.max_context = a.max_context;
    p.num_seqs = a.num_seqs;
    p.num_q_heads = a.num_q_heads;
    p.num_kv_heads = a.pool.num_kv_heads;
    p.num_blocks = a.pool.num_blocks;
    p.scale_log2 = a.scale * kLog2e;
    int dev = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const int ctas = std::min(num_sms(dev), kMaxCtas);
    return a.pool.head_dim == 128 ? launch_group<128>(p, a.pool.int8, a.workspace, ctas, stream)
                                  : launch_group<64>(p, a.pool.int8, a.workspace, ctas, stream);
}

}  // namespace pa
