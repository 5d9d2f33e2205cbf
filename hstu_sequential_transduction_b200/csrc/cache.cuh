// What the kernels of the 8-bit key/value cache share: the pool's view, the
// checks of a sequence, E4M3 conversions and block scales.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "common.cuh"
#include "internal.h"

namespace hstu {

constexpr int kPage = HSTU_CACHE_PAGE;

// Codes of one (page, head) start here, keys [64][D] and values [D][64] alike.
template <int D>
__device__ __forceinline__ int64_t block_offset(int page, int H, int h)
{
    return ((int64_t)page * H + h) * (kPage * D);
}

// One sequence of a call on the cache, with the bits of what is wrong with it
// (0: nothing; any other value drops it).
struct CacheSeq {
    int64_t s0;  // first row of the call's tokens
    int n;       // the call's tokens, `hist` of them history
    int hist;
    int len;     // cached tokens
    int pos;     // position of the next token
    int bits;
};

__device__ __forceinline__ CacheSeq cache_seq(const CacheCall &c, int b)
{
    CacheSeq s;
    s.s0 = c.seq_offsets ? c.seq_offsets[b] : 0;
    const int64_t end = c.seq_offsets ? c.seq_offsets[b + 1] : 0;
    const int nt = c.num_targets ? c.num_targets[b] : 0;
    s.len = c.cache_lens[b];
    s.pos = c.seq_pos ? c.seq_pos[b] : s.len;
    s.bits = 0;
    if (s.s0 < 0 || end < s.s0 || end > c.T)
        s.bits |= FLAG_SEQ_RANGE;
    else if (end - s.s0 > c.max_seq_len)
        s.bits |= FLAG_SEQ_TOO_LONG;
    else if (nt < 0 || nt > end - s.s0)
        s.bits |= FLAG_TARGETS;
    if (s.len < 0 || s.len > c.max_cache_len || s.len > (int64_t)c.max_pages * kPage)
        s.bits |= FLAG_CACHE_LEN;
    s.n = s.bits ? 0 : (int)(end - s.s0);
    s.hist = s.n - (s.bits ? 0 : nt);
    if (s.bits)
        s.len = 0;
    return s;
}

// What is wrong with the offsets as a whole, for the thread that reports sequence b.
__device__ __forceinline__ int cache_offset_bits(const CacheCall &c, int b)
{
    return (b == 0 && c.seq_offsets[0] != 0 ? FLAG_OFFSET0 : 0) |
           (b == c.B - 1 && c.seq_offsets[c.B] != c.T ? FLAG_TOTAL : 0);
}

// Page p of sequence b, or -1 where the table names none of the pool.
__device__ __forceinline__ int table_page(const int32_t *table, const CacheCall &c, int b, int p)
{
    const int page = table[(int64_t)b * c.max_pages + p];
    return page >= 0 && page < c.num_pages ? page : -1;
}

// weights_out of cached tokens j .. j + 3 of sequence b (j a multiple of 4): what they
// had plus their planes, in order.  After a wait that ran out planes are missing: nothing is
// written, for weights that go on from call to call would never lose the damage.
__device__ __forceinline__ void cache_join_weights(const CacheAttnArgs &a, int b, int j)
{
    const CacheCall &c = a.c;
    // the kernel before has ended; read here and looked at last, it costs no time of its own
    const bool whole = !(__ldcg(&c.hdr->flag) & FLAG_TIMEOUT);
    const CacheSeq s = cache_seq(c, b);
    if (j >= s.len)
        return;
    const int page = table_page(c.table, c, b, j / kPage);
    if (page < 0)
        return;
    const int planes = (s.n + a.plan.plane_rows - 1) / a.plan.plane_rows * c.H;
    const int64_t at = (int64_t)page * kPage + j % kPage, step = (int64_t)c.B * a.plan.lcap;
    const float *w = a.part_w + b * a.plan.lcap + j;
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int p = 0; p < planes; p++) {
        const float4 y = *reinterpret_cast<const float4 *>(w + p * step);
        sum.x += y.x, sum.y += y.y, sum.z += y.z, sum.w += y.w;
    }
    const float add[4] = {sum.x, sum.y, sum.z, sum.w}, scale = fabsf(a.inv_n);
#pragma unroll
    for (int e = 0; e < 4; e++)
        if (whole && j + e < s.len)
            a.weights_out[at + e] = fmaf(scale, add[e], c.weights ? c.weights[at + e] : 0.f);
}

// ---- E4M3 ---------------------------------------------------------------------

// two codes (low 16 bits) to two f16: exact
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t codes)
{
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((unsigned short)codes));
    return h;
}

__device__ __forceinline__ float2 e4m3x2_to_f32x2(uint32_t codes)
{
    const uint32_t h = e4m3x2_to_f16x2(codes);
    return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}

// two floats to codes, nearest even, lo in the low byte
__device__ __forceinline__ uint32_t f32x2_to_e4m3x2(float lo, float hi)
{
    return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}

// Scale of a block whose largest magnitude has these float bits: the smallest
// 2^e (e >= -126) with amax <= 448 * 2^e = 1.75 * 2^(e+8).  Magnitudes compare as
// integers, infinities and NaN above every finite one.
__device__ __forceinline__ float block_scale(uint32_t amax_bits)
{
    if (amax_bits == 0)
        return 0.f;
    if (amax_bits >= 0x7f800000u)
        return __int_as_float(0x7fffffff);
    const int e = (int)(amax_bits >> 23) - 127 - 8 + ((amax_bits & 0x7fffffu) > 0x600000u);
    return __int_as_float((max(e, -126) + 127) << 23);
}

// 1 / scale for encoding: exact for the powers of two; 0 (every code 0) for an
// empty or a NaN block.
__device__ __forceinline__ float scale_inverse(float scale)
{
    const int e = (int)(__float_as_uint(scale) >> 23);
    return scale > 0.f && e < 255 ? __int_as_float((254 - e) << 23) : 0.f;
}

// The larger of two block scales; NaN where one is.
__device__ __forceinline__ float larger_scale(float a, float b)
{
    return __uint_as_float(max(__float_as_uint(a) & 0x7fffffffu, __float_as_uint(b) & 0x7fffffffu));
}

}  // namespace hstu
