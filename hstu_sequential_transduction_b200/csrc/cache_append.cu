// Append to the 8-bit key/value cache: quantise a call's history tokens into
// their sequences' pages.
//
// Per block (page, head) of 64 tokens: amax over the block's new tokens, scale
// 2^e with amax <= 448 2^e, code = E4M3(x 2^-e); a partly filled block keeps the
// larger of its old scale and the new one, and its older codes are shifted to it.
//
// Bound by HBM: each k and v element is read once and its code written once (98,000
// tokens of 4 heads, d = 128: 64 us, 4.8 TB/s, with four CTAs an SM, for bf16; 68 with
// three, which float32's registers allow; 86 with two, 127 with the rows widened to
// floats before the reduction).  Issue slots are next, 70 % busy.
// One CTA per (sequence, block, head), 2 D threads: a thread takes 4 tokens x 8
// dims of K and of V, all eight 16-byte (bf16) loads in flight before the one
// reduction.  Keys leave as 8 bytes per token (16 lanes fill a 128-byte row).
// Values are stored transposed: a thread packs its 4 tokens of each dim into a
// word, the words cross through shared memory (columns XORed with the dim group
// and odd groups one dim out of step, so the 32 words of a store fall into 32
// banks) and leave as 16-byte pieces of 64-byte rows.
#include <algorithm>

#include "cache.cuh"

namespace hstu {

namespace {

// eight elements as they lie in memory
struct Eight16 {
    uint4 w;
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) { w = *reinterpret_cast<const uint4 *>(p); }
    __device__ __forceinline__ void zero() { w = make_uint4(0u, 0u, 0u, 0u); }
    __device__ __forceinline__ float get(int e) const
    {
        const uint32_t x = e < 2 ? w.x : e < 4 ? w.y : e < 6 ? w.z : w.w;
        return __uint_as_float(e & 1 ? x & 0xffff0000u : x << 16);
    }
    // the larger of m and this one's magnitudes, each parity's: NaN wins
    using Max = __nv_bfloat162;
    static __device__ __forceinline__ Max none() { return __nv_bfloat162(__ushort_as_bfloat16(0), __ushort_as_bfloat16(0)); }
    static __device__ __forceinline__ Max two(Max m, uint32_t x)
    {
        return __hmax2_nan(m, __habs2(*reinterpret_cast<const __nv_bfloat162 *>(&x)));
    }
    __device__ __forceinline__ Max max(Max m) const { return two(two(two(two(m, w.x), w.y), w.z), w.w); }
    static __device__ __forceinline__ uint32_t bits(Max m)  // as a float's
    {
        return (uint32_t)__bfloat16_as_ushort(__hmax_nan(m.x, m.y)) << 16;
    }
};

struct Eight32 {
    float4 a, b;
    __device__ __forceinline__ void load(const float *p)
    {
        a = reinterpret_cast<const float4 *>(p)[0];
        b = reinterpret_cast<const float4 *>(p)[1];
    }
    __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ __forceinline__ float get(int e) const
    {
        const float4 &f = e < 4 ? a : b;
        return (e & 3) == 0 ? f.x : (e & 3) == 1 ? f.y : (e & 3) == 2 ? f.z : f.w;
    }
    using Max = uint32_t;
    static __device__ __forceinline__ Max none() { return 0; }
    __device__ __forceinline__ Max max(Max m) const
    {
#pragma unroll
        for (int e = 0; e < 8; e++)
            m = ::max(m, __float_as_uint(get(e)) & 0x7fffffffu);
        return m;
    }
    static __device__ __forceinline__ uint32_t bits(Max m) { return m; }
};

template <typename T> struct EightOf { using type = Eight32; };
template <> struct EightOf<__nv_bfloat16> { using type = Eight16; };

// four codes re-rounded after a change of scale (ratio = old scale / new scale)
__device__ __forceinline__ uint32_t rescale4(uint32_t codes, float ratio)
{
    const float2 lo = e4m3x2_to_f32x2(codes), hi = e4m3x2_to_f32x2(codes >> 16);
    return f32x2_to_e4m3x2(lo.x * ratio, lo.y * ratio) | (f32x2_to_e4m3x2(hi.x * ratio, hi.y * ratio) << 16);
}

template <typename T, int D>
__global__ void __launch_bounds__(2 * D, (sizeof(T) == 2 ? 1024 : 768) / (2 * D))
cache_append_kernel(const CacheCall c, const T *__restrict__ k, int64_t ldk, const T *__restrict__ v, int64_t ldv,
                    int32_t *__restrict__ new_lens, int32_t *__restrict__ new_pos, int blocks)
{
    __shared__ uint32_t sv[D * 16];
    __shared__ uint32_t smax[2][D / 16];
    const int h = (int)(blockIdx.x % (unsigned)c.H);
    const int j = (int)(blockIdx.x / (unsigned)c.H % (unsigned)blocks);
    const int b = (int)(blockIdx.x / ((unsigned)c.H * (unsigned)blocks));
    CacheSeq s = cache_seq(c, b);
    if (!s.bits && (int64_t)s.len + s.hist > (int64_t)c.max_pages * kPage)
        s.bits = FLAG_CACHE_LEN;
    const int count = s.bits ? 0 : s.hist;
    if (j == 0 && h == 0 && threadIdx.x == 0) {
        new_lens[b] = c.cache_lens[b] + count;
        if (new_pos)
            new_pos[b] = s.pos + count;
        const int bits = s.bits | cache_offset_bits(c, b);
        if (bits)
            atomicOr(&c.hdr->flag, bits);
    }
    const int blk = s.len / kPage + j;                   // block of the sequence
    const int a = j == 0 ? s.len - blk * kPage : 0;      // first new slot of the block
    const int end = min(s.len + count - blk * kPage, kPage);
    if (a >= end)
        return;
    const int part = threadIdx.x % (D / 8), quad = threadIdx.x / (D / 8);
    const int t0 = 4 * quad;
    // row of slot t: the sequence's token blk * 64 + t - len
    const int64_t row0 = s.s0 + (int64_t)blk * kPage - s.len;

    using Eight = typename EightOf<T>::type;
    Eight x[4], y[4];
#pragma unroll
    for (int t = 0; t < 4; t++) {
        if (t0 + t >= a && t0 + t < end) {
            x[t].load(k + (row0 + t0 + t) * ldk + (int64_t)h * D + 8 * part);
            y[t].load(v + (row0 + t0 + t) * ldv + (int64_t)h * D + 8 * part);
        } else {
            x[t].zero();
            y[t].zero();
        }
    }
    const int page = table_page(c.table, c, b, blk);  // while the rows are on their way
    if (page < 0) {
        if (h == 0 && threadIdx.x == 0)
            atomicOr(&c.hdr->flag, FLAG_CACHE_PAGE);
        return;
    }
    const int64_t si = (int64_t)page * c.H + h;
    const float kold = a > 0 ? c.k_scale[si] : 0.f, vold = a > 0 ? c.v_scale[si] : 0.f;
    typename Eight::Max tk = Eight::none(), tv = Eight::none();
#pragma unroll
    for (int t = 0; t < 4; t++) {
        tk = x[t].max(tk);
        tv = y[t].max(tv);
    }
    uint32_t mk = __reduce_max_sync(0xffffffffu, Eight::bits(tk)), mv = __reduce_max_sync(0xffffffffu, Eight::bits(tv));
    if ((threadIdx.x & 31) == 0) {
        smax[0][threadIdx.x >> 5] = mk;
        smax[1][threadIdx.x >> 5] = mv;
    }
    __syncthreads();
    mk = mv = 0;
#pragma unroll
    for (int w = 0; w < D / 16; w++) {
        mk = max(mk, smax[0][w]);
        mv = max(mv, smax[1][w]);
    }
    const float ks = larger_scale(block_scale(mk), kold), vs = larger_scale(block_scale(mv), vold);
    const float ki = scale_inverse(ks), vi = scale_inverse(vs);
    if (threadIdx.x == 0) {  // after the barrier: every thread has read the old scales
        c.k_scale[si] = ks;
        c.v_scale[si] = vs;
    }
    uint8_t *kc = c.k_codes + block_offset<D>(page, c.H, h);
    uint8_t *vc = c.v_codes + block_offset<D>(page, c.H, h);
    const float kratio = kold * ki, vratio = vold * vi;
#pragma unroll
    for (int t = 0; t < 4; t++) {
        uint2 *dst = reinterpret_cast<uint2 *>(kc + (t0 + t) * D + 8 * part);
        if (t0 + t >= a && t0 + t < end) {
            uint2 w;
            w.x = f32x2_to_e4m3x2(x[t].get(0) * ki, x[t].get(1) * ki) | (f32x2_to_e4m3x2(x[t].get(2) * ki, x[t].get(3) * ki) << 16);
            w.y = f32x2_to_e4m3x2(x[t].get(4) * ki, x[t].get(5) * ki) | (f32x2_to_e4m3x2(x[t].get(6) * ki, x[t].get(7) * ki) << 16);
            *dst = w;
        } else if (t0 + t < a && kratio != 1.f) {
            const uint2 w = *dst;
            *dst = make_uint2(rescale4(w.x, kratio), rescale4(w.y, kratio));
        }
    }
#pragma unroll
    for (int ee = 0; ee < 8; ee++) {
        const int e = ee ^ (part & 1), d = 8 * part + e;
        // select y[.][e] without a dynamic index
        float y4[4];
#pragma unroll
        for (int t = 0; t < 4; t++)
            y4[t] = (part & 1) ? y[t].get(ee ^ 1) : y[t].get(ee);
        uint32_t w = f32x2_to_e4m3x2(y4[0] * vi, y4[1] * vi) | (f32x2_to_e4m3x2(y4[2] * vi, y4[3] * vi) << 16);
        if (t0 < a || t0 + 4 > end) {  // some of these slots are not new: shifted if older, kept if behind the end
            const uint32_t was = *reinterpret_cast<const uint32_t *>(vc + d * kPage + t0);
            const uint32_t moved = vratio != 1.f ? rescale4(was, vratio) : was;
            uint32_t mix = 0;
#pragma unroll
            for (int t = 0; t < 4; t++) {
                const uint32_t m = 0xffu << (8 * t);
                mix |= m & (t0 + t < a ? moved : (t0 + t < end ? w : was));
            }
            w = mix;
        }
        sv[d * 16 + (quad ^ (part & 15))] = w;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < D * 4; i += 2 * D) {
        const int d = i >> 2, q = (i & 3) * 4, z = (d >> 3) & 15;
        *reinterpret_cast<uint4 *>(vc + d * kPage + 4 * q) =
            make_uint4(sv[d * 16 + (q ^ z)], sv[d * 16 + ((q + 1) ^ z)], sv[d * 16 + ((q + 2) ^ z)],
                       sv[d * 16 + ((q + 3) ^ z)]);
    }
    if (h == 0) {
        for (int t = threadIdx.x; t < kPage; t += 2 * D) {
            if (t < a || t >= end)
                continue;
            const int64_t at = (int64_t)page * kPage + t;
            const int i = blk * kPage + t - s.len;
            c.timestamps[at] = c.ts[s.s0 + i];
            c.positions[at] = s.pos + i;
            if (c.weights)
                c.weights[at] = 0.f;
        }
    }
}

template <typename T, int D>
cudaError_t append(const CacheCall &c, const void *k, int64_t ldk, const void *v, int64_t ldv, int32_t *new_lens,
                   int32_t *new_pos, int blocks, cudaStream_t stream)
{
    const int64_t grid = (int64_t)c.B * blocks * c.H;
    cache_append_kernel<T, D><<<(unsigned)grid, 2 * D, 0, stream>>>(c, static_cast<const T *>(k), ldk,
                                                                    static_cast<const T *>(v), ldv, new_lens, new_pos,
                                                                    blocks);
    return cudaGetLastError();
}

}  // namespace

// blocks a sequence's new tokens may touch: they start anywhere in the first
int cache_append_blocks(int max_seq_len) { return std::max(1, (int)(((int64_t)max_seq_len + 2 * kPage - 2) / kPage)); }

cudaError_t launch_cache_append(const CacheCall &c, bool bf16, const void *k, int64_t ldk, const void *v, int64_t ldv,
                                int32_t *new_lens, int32_t *new_pos, cudaStream_t stream)
{
    if (c.B == 0)
        return launch_cache_no_sequences(c, stream);
    const int blocks = cache_append_blocks(c.max_seq_len);
    if (bf16)
        return c.d == 64 ? append<__nv_bfloat16, 64>(c, k, ldk, v, ldv, new_lens, new_pos, blocks, stream)
                         : append<__nv_bfloat16, 128>(c, k, ldk, v, ldv, new_lens, new_pos, blocks, stream);
    return c.d == 32 ? append<float, 32>(c, k, ldk, v, ldv, new_lens, new_pos, blocks, stream)
                     : append<float, 64>(c, k, ldk, v, ldv, new_lens, new_pos, blocks, stream);
}

}  // namespace hstu
