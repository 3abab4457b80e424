// Append into, and block copy of, an 8-bit KV cache with one scale per (block, kv
// head): codes are e4m3 or int8, a value is code * scale.
//
// What is computed (include/pa.h): for the tokens of one call that go to block b
// (kv head h), A = max |x| over their finite elements and
//   need  = the smallest power of two with A <= need * Q   (Q = 448 or 127; >= 2^-64)
//   sigma = max(sigma_old, need)       (sigma_old = 0 when slot 0 of b is written:
//                                       the block starts a new life)
//   new codes = round(x / sigma), nearest even; codes of earlier tokens of the block
//   become round(code * sigma_old / sigma) when sigma has grown.
// Why powers of two: x / sigma and the change of scale are then exact before their one
// rounding, so the codes do not depend on the arithmetic, writing the same tokens again
// changes nothing, and for e4m3 (a floating format) a coarser scale costs no relative
// precision at all: an earlier code only loses bits where it becomes subnormal.  For
// int8 the step is at most twice the finest possible one.
//
// What bounds it: HBM for prompts (2 * 2 bytes read and 2 written per element pair),
// latency for a decode step.  One warp takes all tokens of one run (consecutive tokens
// of one block; 16 or fewer as appends produce them) for one kv head of K or of V: the
// rows are loaded once, kept in registers through the maximum and the rounding, and
// stored as codes, so there is one pass over the data, one launch and no atomics.
#include <type_traits>

#include <cuda_fp8.h>

#include "pa_common.cuh"
#include "pa_step.h"

namespace pa {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kWriteWarps = 4, kWriteCtas = 8;
constexpr int kMinExp = -64;   // scales below 2^-64 would only keep values below 1e-16

constexpr uint32_t kInfBits = 0x7f80;   // bf16 |x| bits from here on: infinities and NaN

// Largest |x| (bf16 bits, sign off) of the two halves of w and m.
__device__ __forceinline__ uint32_t amax2(uint32_t m, uint32_t w) { return __vmaxu2(m, w & 0x7fff7fffu); }

// The same with infinities and NaN left out.
__device__ __forceinline__ uint32_t amax2_finite(uint32_t m, uint32_t w) {
    uint32_t a = w & 0x7fff7fffu;
    if ((a & 0xffffu) >= kInfBits) a &= 0xffff0000u;
    if ((a >> 16) >= kInfBits) a &= 0x0000ffffu;
    return __vmaxu2(m, a);
}

// Exponent of the smallest power of two s with amax <= s * Q; amax as bf16 bits, finite.
template <bool kInt8>
__device__ __forceinline__ int scale_exp(uint32_t amax_bits) {
    // amax = 1.M * 2^(E - 127); Q = 448 = 1.75 * 2^8 (M <= 0x60) or 127 = 1.984375 * 2^6 (M <= 0x7e).
    // Zero and subnormal amax (E = 0) end at the floor.
    const int E = (int)(amax_bits >> 7), M = (int)(amax_bits & 0x7f);
    const int e = kInt8 ? E - 133 + (M > 0x7e) : E - 135 + (M > 0x60);
    return max(e, kMinExp);
}

__device__ __forceinline__ float exp2_int(int e) { return __int_as_float((e + 127) << 23); }  // |e| < 127

// Four values (already divided by the scale) -> four codes.
template <bool kInt8>
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d) {
    if constexpr (kInt8) {
        // nearest even; infinities saturate, NaN becomes 0
        auto q = [](float x) { return (uint32_t)(min(max(__float2int_rn(x), -127), 127)) & 0xffu; };
        return q(a) | (q(b) << 8) | (q(c) << 16) | (q(d) << 24);
    } else {
        const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
        const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
        return lo | (hi << 16);
    }
}

// Four bf16 values -> four codes.  kFinite: no infinity or NaN among them, so that |x * inv| is
// at most the largest code; int8 then rounds by adding 1.5 * 2^23 (x * inv is exact, so this is
// the one rounding, to nearest even) and takes the low byte: the conversion instruction
// runs at a quarter of that rate.
template <bool kInt8, bool kFinite>
__device__ __forceinline__ uint32_t encode_bf16x4(uint32_t w0, uint32_t w1, float inv) {
    const float2 a = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&w0));
    const float2 b = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&w1));
    const float2 i2 = make_float2(inv, inv);
    if constexpr (kInt8 && kFinite) {
        const float2 magic = make_float2(12582912.f, 12582912.f);
        const float2 x = __ffma2_rn(a, i2, magic), y = __ffma2_rn(b, i2, magic);
        const uint32_t lo = __byte_perm(__float_as_uint(x.x), __float_as_uint(x.y), 0x0040);
        const uint32_t hi = __byte_perm(__float_as_uint(y.x), __float_as_uint(y.y), 0x0040);
        return __byte_perm(lo, hi, 0x5410);
    }
    const float2 x = __fmul2_rn(a, i2), y = __fmul2_rn(b, i2);
    return encode4<kInt8>(x.x, x.y, y.x, y.y);
}

// Four codes re-expressed under a larger scale: round(code * ratio).
template <bool kInt8>
__device__ __forceinline__ uint32_t recode4(uint32_t w, float ratio) {
    float v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t c = (w >> (8 * i)) & 0xffu;
        if constexpr (kInt8) {
            v[i] = (float)(int8_t)c * ratio;
        } else {
            __nv_fp8_e4m3 f;
            f.__x = (unsigned char)c;
            v[i] = (float)f * ratio;
        }
    }
    return encode4<kInt8>(v[0], v[1], v[2], v[3]);
}

// D: head_dim.  A warp covers kRows rows of D elements per load, 16 bytes a lane.
// window: tokens whose runs one warp looks after.
// Eight CTAs to an SM: 32 warps, each with 4 KB of rows in flight, at 64 registers (what
// spills belongs to the rare paths).  102 MB of prompts: 19.0 us, 5.4 TB/s (floor 15.5); with 7
// CTAs 19.6, with 9 (rows spill) 21.7.  256 tokens: 3.95 us, the latency of one warp's chain of
// loads.  The instructions count as much as the bytes (issue slots 71 % taken with a path for
// every order of slots: 21.3 and 4.8 us), so runs of ascending slots have one of their own, and
// earlier tokens are re-expressed last, when the rows' registers are free (19.4 before).
template <int D, bool kInt8>
__global__ void __launch_bounds__(kWriteWarps * 32, kWriteCtas) cache_write_scaled_kernel(const __grid_constant__ ScaledWrite p,
                                                                              int window) {
    constexpr int kLanes = D / 8, kRows = 32 / kLanes, kPasses = kBlockSize / kRows;
    const int lane = threadIdx.x & 31;
    const int64_t wid = (int64_t)blockIdx.x * kWriteWarps + (threadIdx.x >> 5);
    const int hkv = p.pool.num_kv_heads;
    const int64_t per = 2 * (int64_t)hkv;
    const int64_t win = wid / per;
    const int rem = (int)(wid - win * per);
    const bool is_v = rem >= hkv;
    const int h = is_v ? rem - hkv : rem;
    const int T = p.num_tokens;
    if (win * window >= T) return;
    const int w0 = (int)(win * window);
    const int64_t num_slots = (int64_t)p.pool.num_blocks * kBlockSize;
    // block of token i, or -1 for padding and slots outside the pool
    auto block_of = [&](int i, int &off) -> int {
        off = 0;
        if (i < 0 || i >= T) return -1;
        const int64_t slot = p.slots[i];
        if (slot < 0 || slot >= num_slots) return -1;
        off = (int)(slot % kBlockSize);
        return (int)(slot / kBlockSize);
    };
    // lane l: token w0 - 1 + l; a run starts where the block differs from the token before
    int off;
    const int mine = block_of(w0 - 1 + lane, off);
    const int before = __shfl_up_sync(kFull, mine, 1);
    if (rem == 0 && lane >= 1 && lane <= window && w0 - 1 + lane < T && p.slots[w0 - 1 + lane] >= num_slots)
        flag_error(p.err, PA_DEVERR_SLOT);
    unsigned leaders = __ballot_sync(kFull, lane >= 1 && lane <= window && mine >= 0 && mine != before);

    const unsigned char *src = static_cast<const unsigned char *>(is_v ? p.value : p.key);
    const int64_t stride = (is_v ? p.value_stride : p.key_stride) * 2;
    unsigned char *pool = static_cast<unsigned char *>(is_v ? p.pool.vc : p.pool.kc);
    float *scales = is_v ? p.pool.vs : p.pool.ks;
    const int c = lane % kLanes, r0 = lane / kLanes;
    const unsigned char *base = src + (int64_t)h * D * 2 + c * 16;

    while (leaders) {
        const int l = __ffs(leaders) - 1;
        leaders &= leaders - 1;
        const int i0 = w0 - 1 + l;
        const int blk = __shfl_sync(kFull, mine, l);
        const int64_t bh = (int64_t)blk * hkv + h;
        const float old_scale = scales[bh];
        // The run's length and the slots it writes, from the entries this warp holds (16
        // tokens from any leader on); a run that reaches the last of them (more than 16 tokens:
        // slots named twice) is followed through the mapping.
        const unsigned same = __ballot_sync(kFull, mine == blk) >> l;
        int n = ~same == 0u ? 32 : __ffs(~same) - 1;
        uint32_t written = __reduce_or_sync(kFull, lane >= l && lane < l + n ? 1u << off : 0u);
        bool more = l + n >= 32;
        while (more) {
            int o;
            const bool go = block_of(i0 + n + lane, o) == blk;
            const unsigned m = __ballot_sync(kFull, go);
            const int k = m == kFull ? 32 : __ffs(~m) - 1;
            written |= __reduce_or_sync(kFull, lane < k ? 1u << o : 0u);
            n += k;
            more = k == 32;
        }
        unsigned char *block = pool + bh * (kBlockSize * D) + c * 8;
        // |x| bits of a row's piece into the running maximum
        auto maximum = [&](uint32_t m, const uint4 &x) { return amax2(amax2(amax2(amax2(m, x.x), x.y), x.z), x.w); };
        auto maximum_finite = [&](uint32_t m, const uint4 &x) {
            return amax2_finite(amax2_finite(amax2_finite(amax2_finite(m, x.x), x.y), x.z), x.w);
        };
        auto over_warp = [&](uint32_t m) { return __reduce_max_sync(kFull, max(m & 0xffffu, m >> 16)); };
        // The scale for a run of maximum a16 that writes the slots of `written`, stored.
        bool grown = false;
        auto settle = [&](uint32_t a16, uint32_t written) -> float {
            // a stored scale that is no finite positive number counts as none
            const bool has_old = (written & 1u) == 0u && old_scale > 0.f && old_scale < INFINITY;
            float sigma = exp2_int(scale_exp<kInt8>(a16));
            if (has_old && old_scale > sigma) sigma = old_scale;
            if (lane == 0 && !(has_old && sigma == old_scale)) scales[bh] = sigma;
            grown = has_old && sigma > old_scale;
            return sigma;
        };
        // Earlier tokens of the block under a scale that has grown.
        auto regrow = [&](float sigma, uint32_t written) {
            if (grown) {
                const float ratio = old_scale / sigma;
                const uint32_t below = (2u << (31 - __clz(written))) - 1u;
                const uint32_t keep = below & ~written;
                uint2 held[kPasses];
#pragma unroll
                for (int k = 0; k < kPasses; ++k) {
                    const int o = k * kRows + r0;
                    if (keep >> o & 1u) held[k] = *reinterpret_cast<const uint2 *>(block + o * D);
                }
#pragma unroll
                for (int k = 0; k < kPasses; ++k) {
                    const int o = k * kRows + r0;
                    if (keep >> o & 1u)
                        *reinterpret_cast<uint2 *>(block + o * D) =
                            make_uint2(recode4<kInt8>(held[k].x, ratio), recode4<kInt8>(held[k].y, ratio));
                }
            }
        };
        auto codes = [&](auto all_finite, const uint4 &x, float inv) {
            constexpr bool kFin = decltype(all_finite)::value;
            return make_uint2(encode_bf16x4<kInt8, kFin>(x.x, x.y, inv), encode_bf16x4<kInt8, kFin>(x.z, x.w, inv));
        };
        uint4 row[kPasses];
        const int o0 = __shfl_sync(kFull, off, l);
        const bool in_order = __all_sync(kFull, lane < l || lane >= l + n || off == o0 + (lane - l));
        if (in_order && n <= kBlockSize) {
            // ascending slots, as appends produce them: the rows stay in registers
            const int64_t row_bytes = kRows * stride;
            const unsigned char *at = base + (int64_t)(i0 + r0) * stride;
            uint32_t am = 0;
#pragma unroll
            for (int k = 0; k < kPasses; ++k) {
                row[k] = make_uint4(0, 0, 0, 0);
                if (k * kRows + r0 < n) row[k] = __ldg(reinterpret_cast<const uint4 *>(at + k * row_bytes));
            }
#pragma unroll
            for (int k = 0; k < kPasses; ++k) am = maximum(am, row[k]);
            uint32_t a16 = over_warp(am);
            const bool finite = a16 < kInfBits;
            if (!finite) {   // once more without the infinities and NaN
                am = 0;
#pragma unroll
                for (int k = 0; k < kPasses; ++k) am = maximum_finite(am, row[k]);
                a16 = over_warp(am);
            }
            const uint32_t wr = ((1u << n) - 1u) << o0;
            const float sigma = settle(a16, wr), inv = 1.f / sigma;
            unsigned char *dst = block + (o0 + r0) * D;
            auto store = [&](auto fin) {
#pragma unroll
                for (int k = 0; k < kPasses; ++k)
                    if (k * kRows + r0 < n) *reinterpret_cast<uint2 *>(dst + k * kRows * D) = codes(fin, row[k], inv);
            };
            if (finite) store(std::true_type{});
            else store(std::false_type{});
            regrow(sigma, wr);
        } else {
            // any order, and slots named more than once: 16 rows at a time, fetched for each pass
            uint32_t am = 0;
            auto load = [&](int first) {
#pragma unroll
                for (int k = 0; k < kPasses; ++k) {
                    const int t = first + k * kRows + r0;
                    row[k] = make_uint4(0, 0, 0, 0);
                    if (t < n) row[k] = __ldg(reinterpret_cast<const uint4 *>(base + (int64_t)(i0 + t) * stride));
                }
            };
#pragma unroll 1
            for (int first = 0; first < n; first += kBlockSize) {
                load(first);
#pragma unroll
                for (int k = 0; k < kPasses; ++k) am = maximum_finite(am, row[k]);
            }
            const float sigma = settle(over_warp(am), written), inv = 1.f / sigma;
            regrow(sigma, written);
#pragma unroll 1
            for (int first = 0; first < n; first += kBlockSize) {
                load(first);
#pragma unroll
                for (int k = 0; k < kPasses; ++k) {
                    const int t = first + k * kRows + r0;
                    if (t < n)
                        *reinterpret_cast<uint2 *>(block + (int)(p.slots[i0 + t] % kBlockSize) * D) =
                            codes(std::false_type{}, row[k], inv);
                }
            }
        }
        __syncwarp();
    }
}

// Block copies (copy on write) with their scales.  grid = (pairs, chunks, 2): z selects K or V.
constexpr int kCopyUnroll = 4;

__global__ void __launch_bounds__(256) copy_blocks_scaled_kernel(const __grid_constant__ ScaledPool p,
                                                                 const int32_t *__restrict__ pairs,
                                                                 int64_t chunks_per_block, int32_t *err) {
    const int32_t src = pairs[2 * (int64_t)blockIdx.x], dst = pairs[2 * (int64_t)blockIdx.x + 1];
    if (src < 0 || src >= p.num_blocks || dst < 0 || dst >= p.num_blocks) {
        if (blockIdx.y == 0 && blockIdx.z == 0 && threadIdx.x == 0) flag_error(err, PA_DEVERR_PAIR);
        return;
    }
    uint4 *cache = static_cast<uint4 *>(blockIdx.z == 0 ? p.kc : p.vc);
    float *scales = blockIdx.z == 0 ? p.ks : p.vs;
    const uint4 *s = cache + (int64_t)src * chunks_per_block;
    uint4 *d = cache + (int64_t)dst * chunks_per_block;
    const int64_t base = (int64_t)blockIdx.y * blockDim.x * kCopyUnroll + threadIdx.x;
    uint4 buf[kCopyUnroll];
#pragma unroll
    for (int k = 0; k < kCopyUnroll; ++k) {
        const int64_t c = base + (int64_t)k * blockDim.x;
        if (c < chunks_per_block) buf[k] = s[c];
    }
    if (blockIdx.y == 0) {
        for (int h = threadIdx.x; h < p.num_kv_heads; h += blockDim.x)
            scales[(int64_t)dst * p.num_kv_heads + h] = scales[(int64_t)src * p.num_kv_heads + h];
    }
#pragma unroll
    for (int k = 0; k < kCopyUnroll; ++k) {
        const int64_t c = base + (int64_t)k * blockDim.x;
        if (c < chunks_per_block) d[c] = buf[k];
    }
}

}  // namespace

cudaError_t launch_cache_write_scaled(const ScaledWrite &w, cudaStream_t stream) {
    // One token per warp while that fills the GPU's warps but a few times over (a decode
    // step: every token has a block of its own); 16 tokens per warp for more, where
    // most tokens are not the first of their run and their warps would only exit.
    const int64_t rows = (int64_t)w.num_tokens * w.pool.num_kv_heads * 2;
    const int window = rows > 32768 ? kBlockSize : 1;
    const int64_t warps = ((int64_t)w.num_tokens + window - 1) / window * w.pool.num_kv_heads * 2;
    const int64_t blocks = (warps + kWriteWarps - 1) / kWriteWarps;
    if (blocks > INT32_MAX) return cudaErrorNotSupported;
    const dim3 grid((unsigned)blocks), block(kWriteWarps * 32);
    if (w.pool.head_dim == 128) {
        if (w.pool.int8) cache_write_scaled_kernel<128, true><<<grid, block, 0, stream>>>(w, window);
        else cache_write_scaled_kernel<128, false><<<grid, block, 0, stream>>>(w, window);
    } else {
        if (w.pool.int8) cache_write_scaled_kernel<64, true><<<grid, block, 0, stream>>>(w, window);
        else cache_write_scaled_kernel<64, false><<<grid, block, 0, stream>>>(w, window);
    }
    return cudaGetLastError();
}

cudaError_t launch_copy_blocks_scaled(const ScaledPool &pool, const int32_t *pairs, int32_t num_pairs, int32_t *err,
                                      cudaStream_t stream) {
    const int64_t chunks = (int64_t)pool.num_kv_heads * kBlockSize * pool.head_dim / 16;
    const int64_t per_cta = 256 * kCopyUnroll;
    const dim3 grid((unsigned)num_pairs, (unsigned)((chunks + per_cta - 1) / per_cta), 2);
    copy_blocks_scaled_kernel<<<grid, 256, 0, stream>>>(pool, pairs, chunks, err);
    return cudaGetLastError();
}

}  // namespace pa
