// Eviction from the 8-bit key/value cache by accumulated attention weight.
//
// Select (one CTA per sequence): weights become integers that compare as the
// weights do (NaN 0); four 8-bit histogram passes find the m-th largest of the
// unprotected tokens; two ordered passes, in which a thread owns a run of
// consecutive tokens, count and write the kept indices, ties at the threshold to
// the lowest index.  Bound by latency: a few passes over 4 L bytes that stay in L2.
//
// Move (one CTA per new block and head): keys are gathered as rows; values are
// stored transposed, so the source pages the block draws on are staged in shared
// memory whole (rows padded to 17 words: the threads of a warp read one byte each
// of 32 rows without a bank conflict) and the kept columns picked out.  The block
// gets its own scale from the largest decoded magnitude.  Bound by HBM: the kept
// keys and the source pages of the values are read once, the new block written.
#include <algorithm>

#include "cache.cuh"

namespace hstu {

namespace {

constexpr int kSelThreads = 1024;

__device__ __forceinline__ uint32_t weight_key(float w)
{
    if (w != w)
        return 0u;
    const uint32_t u = __float_as_uint(w == 0.f ? 0.f : w);  // -0 ties with 0
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// exclusive sum over the block's threads; *total the sum
__device__ __forceinline__ int block_scan(int x, int *warp_sums, int *total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int inc = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o)
            inc += y;
    }
    __syncthreads();
    if (lane == 31)
        warp_sums[warp] = inc;
    __syncthreads();
    if (warp == 0) {
        int w = warp_sums[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, w, o);
            if (lane >= o)
                w += y;
        }
        warp_sums[lane] = w;
    }
    __syncthreads();
    *total = warp_sums[31];
    return inc - x + (warp ? warp_sums[warp - 1] : 0);
}

__global__ void __launch_bounds__(kSelThreads)
cache_select_kernel(const CacheCall c, int keep, int first, int recent, const int32_t *__restrict__ new_pages,
                    int32_t *__restrict__ new_table, int32_t *__restrict__ new_lens, int32_t *__restrict__ kept,
                    uint32_t *__restrict__ keys, int64_t cap)
{
    __shared__ int hist[256];
    __shared__ int warp_sums[32];
    __shared__ int found[2];
    const int b = blockIdx.x, tid = threadIdx.x;
    const CacheSeq s = cache_seq(c, b);
    const int L = s.len;
    const bool moves = L > keep;
    if (tid == 0) {
        new_lens[b] = s.bits ? c.cache_lens[b] : min(L, keep);
        if (s.bits)
            atomicOr(&c.hdr->flag, s.bits);
    }
    const int32_t *row = moves ? new_pages : c.table;
    for (int p = tid; p < c.max_pages; p += kSelThreads)
        new_table[(int64_t)b * c.max_pages + p] = row[(int64_t)b * c.max_pages + p];
    int32_t *out = kept + (int64_t)b * keep;
    if (!moves) {
        for (int i = tid; i < keep; i += kSelThreads)
            out[i] = i < L ? i : -1;
        return;
    }
    const int late = min(keep, recent), early = min(min(keep - late, first), L - late);
    const int m = keep - late - early;  // of the tokens [early, L - late)
    uint32_t *key = keys + (int64_t)b * cap;
    bool bad = false;
    for (int j = tid; j < L; j += kSelThreads) {
        const int page = table_page(c.table, c, b, j / kPage);
        bad |= page < 0;
        key[j] = page < 0 ? 0u : weight_key(c.weights[(int64_t)page * kPage + j % kPage]);
    }
    if (bad)
        atomicOr(&c.hdr->flag, FLAG_CACHE_PAGE);
    __syncthreads();
    // the m-th largest key: `prefix` after four passes; `left` of the tokens equal to it are kept
    uint32_t prefix = 0, mask = 0;
    int left = m;
    for (int shift = 24; shift >= 0 && m > 0; shift -= 8) {
        for (int i = tid; i < 256; i += kSelThreads)
            hist[i] = 0;
        __syncthreads();
        for (int j = early + tid; j < L - late; j += kSelThreads) {
            const uint32_t u = key[j];
            if ((u & mask) == prefix)
                atomicAdd(&hist[(u >> shift) & 255], 1);
        }
        __syncthreads();
        if (tid < 32) {
            // lane: bins 255 - 8 lane downwards; the bin in which the running count reaches `left`
            int n[8], sum = 0;
#pragma unroll
            for (int e = 0; e < 8; e++) {
                n[e] = hist[255 - 8 * tid - e];
                sum += n[e];
            }
            int inc = sum;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, inc, o);
                if (tid >= o)
                    inc += y;
            }
            int run = inc - sum;
#pragma unroll
            for (int e = 0; e < 8; e++) {
                if (run < left && run + n[e] >= left) {
                    found[0] = 255 - 8 * tid - e;
                    found[1] = left - run;
                }
                run += n[e];
            }
        }
        __syncthreads();
        prefix |= (uint32_t)found[0] << shift;
        mask |= 255u << shift;
        left = found[1];
        __syncthreads();
    }
    // ordered: thread t owns [t * run, (t + 1) * run)
    const int run = (L + kSelThreads - 1) / kSelThreads;
    const int j0 = min(tid * run, L), j1 = min(j0 + run, L);
    int eq = 0, gt = 0;
    for (int j = j0; j < j1; j++) {
        const bool safe = j < early || j >= L - late;
        const uint32_t u = key[j];
        gt += safe || (m > 0 && u > prefix);
        eq += !safe && m > 0 && u == prefix;
    }
    int total;
    const int eq0 = block_scan(eq, warp_sums, &total);
    // of this thread's ties, those among the first `left` of all
    const int mine = max(0, min(eq, left - eq0));
    int at = block_scan(gt + mine, warp_sums, &total);
    int ties = mine;
    for (int j = j0; j < j1; j++) {
        const bool safe = j < early || j >= L - late;
        const uint32_t u = key[j];
        bool take = safe || (m > 0 && u > prefix);
        if (!take && m > 0 && u == prefix && ties > 0) {
            take = true;
            ties--;
        }
        if (take)
            out[at++] = j;
    }
}

template <int D>
__global__ void __launch_bounds__(2 * D)
cache_move_kernel(const CacheCall c, int keep, int blocks, const int32_t *__restrict__ new_pages,
                  const int32_t *__restrict__ kept)
{
    constexpr int NT = 2 * D, LD = 68;  // bytes of a padded row
    __shared__ __align__(16) uint8_t src[D * LD], dst[D * LD];
    __shared__ int tok_page[kPage], tok_slot[kPage];
    __shared__ float tok_ks[kPage], tok_vs[kPage];
    __shared__ uint32_t smax[2][D / 16];
    const int h = (int)(blockIdx.x % (unsigned)c.H);
    const int j = (int)(blockIdx.x / (unsigned)c.H % (unsigned)blocks);
    const int b = (int)(blockIdx.x / ((unsigned)c.H * (unsigned)blocks));
    const CacheSeq s = cache_seq(c, b);
    if (s.len <= keep)
        return;
    const int tid = threadIdx.x;
    const int count = min(keep - j * kPage, kPage);
    const int to = table_page(new_pages, c, b, j);
    if (to < 0) {
        if (h == 0 && tid == 0)
            atomicOr(&c.hdr->flag, FLAG_CACHE_PAGE);
        return;
    }
    if (tid < kPage) {
        int page = -1, slot = 0;
        if (tid < count) {
            const int i = kept[(int64_t)b * keep + j * kPage + tid];
            page = table_page(c.table, c, b, i / kPage);
            slot = i % kPage;
        }
        tok_page[tid] = page;
        tok_slot[tid] = slot;
        tok_ks[tid] = page < 0 ? 0.f : c.k_scale[(int64_t)page * c.H + h];
        tok_vs[tid] = page < 0 ? 0.f : c.v_scale[(int64_t)page * c.H + h];
        if (h == 0 && tid < count && page >= 0) {
            const int64_t from = (int64_t)page * kPage + slot, at = (int64_t)to * kPage + tid;
            c.timestamps[at] = c.timestamps[from];
            c.positions[at] = c.positions[from];
            c.weights[at] = c.weights[from];
        }
    }
    __syncthreads();
    // keys of this thread's 4 tokens x 8 dims
    const int part = tid % (D / 8), quad = tid / (D / 8), t0 = 4 * quad;
    uint2 kw[4];
#pragma unroll
    for (int t = 0; t < 4; t++) {
        const int page = tok_page[t0 + t];
        kw[t] = page < 0 ? make_uint2(0u, 0u)
                         : *reinterpret_cast<const uint2 *>(c.k_codes + block_offset<D>(page, c.H, h) +
                                                            tok_slot[t0 + t] * D + 8 * part);
    }
    // values: the tokens of one source page are neighbours (kept is ascending)
    for (int t = 0; t < count;) {
        const int page = tok_page[t];
        int t1 = t + 1;
        while (t1 < count && tok_page[t1] == page)
            t1++;
        if (page >= 0) {
            const uint8_t *vb = c.v_codes + block_offset<D>(page, c.H, h);
            for (int i = tid; i < D * 4; i += NT) {
                const uint4 w = *reinterpret_cast<const uint4 *>(vb + 16 * i);
                uint32_t *p = reinterpret_cast<uint32_t *>(src + (i >> 2) * LD + (i & 3) * 16);
                p[0] = w.x, p[1] = w.y, p[2] = w.z, p[3] = w.w;
            }
        }
        __syncthreads();
        const int d = tid % D;
        for (int u = t + tid / D; u < t1; u += 2)
            dst[d * LD + u] = page < 0 ? 0 : src[d * LD + tok_slot[u]];
        __syncthreads();
        t = t1;
    }
    for (int u = count + tid / D; u < kPage; u += 2)
        dst[(tid % D) * LD + u] = 0;
    __syncthreads();
    uint32_t vw[8], mk = 0, mv = 0;
#pragma unroll
    for (int e = 0; e < 8; e++)
        vw[e] = *reinterpret_cast<const uint32_t *>(dst + (8 * part + e) * LD + t0);
    float ksc[4], vsc[4];
#pragma unroll
    for (int t = 0; t < 4; t++) {
        ksc[t] = tok_ks[t0 + t];
        vsc[t] = tok_vs[t0 + t];
    }
    auto mag = [](float x) { return __float_as_uint(x) & 0x7fffffffu; };
#pragma unroll
    for (int t = 0; t < 4; t++)
#pragma unroll
        for (int e = 0; e < 4; e++) {
            const float2 f = e4m3x2_to_f32x2((e < 2 ? kw[t].x : kw[t].y) >> (16 * (e & 1)));
            mk = max(mk, max(mag(f.x * ksc[t]), mag(f.y * ksc[t])));
        }
#pragma unroll
    for (int e = 0; e < 8; e++) {
        const float2 lo = e4m3x2_to_f32x2(vw[e]), hi = e4m3x2_to_f32x2(vw[e] >> 16);
        mv = max(mv, max(max(mag(lo.x * vsc[0]), mag(lo.y * vsc[1])), max(mag(hi.x * vsc[2]), mag(hi.y * vsc[3]))));
    }
    mk = __reduce_max_sync(0xffffffffu, mk);
    mv = __reduce_max_sync(0xffffffffu, mv);
    if ((tid & 31) == 0) {
        smax[0][tid >> 5] = mk;
        smax[1][tid >> 5] = mv;
    }
    __syncthreads();
    mk = mv = 0;
#pragma unroll
    for (int w = 0; w < D / 16; w++) {
        mk = max(mk, smax[0][w]);
        mv = max(mv, smax[1][w]);
    }
    const float ks = block_scale(mk), vs = block_scale(mv);
    const float ki = scale_inverse(ks), vi = scale_inverse(vs);
    if (tid == 0) {
        c.k_scale[(int64_t)to * c.H + h] = ks;
        c.v_scale[(int64_t)to * c.H + h] = vs;
    }
    uint8_t *kc = c.k_codes + block_offset<D>(to, c.H, h);
    uint8_t *vc = c.v_codes + block_offset<D>(to, c.H, h);
    // re-rounded at the new scale: two exact products, so one rounding
    auto put2 = [](uint32_t codes, float r0, float r1) {
        const float2 f = e4m3x2_to_f32x2(codes);
        return f32x2_to_e4m3x2(f.x * r0, f.y * r1);
    };
#pragma unroll
    for (int t = 0; t < 4; t++) {
        if (t0 + t >= count)
            continue;
        const float r = ksc[t] * ki;
        *reinterpret_cast<uint2 *>(kc + (t0 + t) * D + 8 * part) =
            make_uint2(put2(kw[t].x, r, r) | (put2(kw[t].x >> 16, r, r) << 16),
                       put2(kw[t].y, r, r) | (put2(kw[t].y >> 16, r, r) << 16));
    }
#pragma unroll
    for (int e = 0; e < 8; e++) {
        const float r0 = vsc[0] * vi, r1 = vsc[1] * vi, r2 = vsc[2] * vi, r3 = vsc[3] * vi;
        *reinterpret_cast<uint32_t *>(dst + (8 * part + e) * LD + t0) =
            put2(vw[e], r0, r1) | (put2(vw[e] >> 16, r2, r3) << 16);
    }
    __syncthreads();
    for (int i = tid; i < D * 4; i += NT) {
        const int d = i >> 2, q = (i & 3) * 16;
        const uint32_t *p = reinterpret_cast<const uint32_t *>(dst + d * LD + q);
        uint4 w = make_uint4(p[0], p[1], p[2], p[3]);
        uint4 *g = reinterpret_cast<uint4 *>(vc + d * kPage + q);
        if (q + 16 > count) {  // slots behind the last token keep their bytes
            const uint4 was = *g;
            auto mix = [&](uint32_t a, uint32_t o, int base) {
                const int n = count - base;
                const uint32_t m = n >= 4 ? 0xffffffffu : n <= 0 ? 0u : (1u << (8 * n)) - 1u;
                return (a & m) | (o & ~m);
            };
            w = make_uint4(mix(w.x, was.x, q), mix(w.y, was.y, q + 4), mix(w.z, was.z, q + 8), mix(w.w, was.w, q + 12));
        }
        *g = w;
    }
}

template <int D>
void move(const CacheCall &c, int keep, int blocks, const int32_t *new_pages, const int32_t *kept, cudaStream_t stream)
{
    cache_move_kernel<D><<<(unsigned)((int64_t)c.B * blocks * c.H), 2 * D, 0, stream>>>(c, keep, blocks, new_pages,
                                                                                       kept);
}

}  // namespace

cudaError_t launch_cache_evict(const CacheCall &c, int keep, int first, int recent, const int32_t *new_pages,
                               int32_t *new_table, int32_t *new_lens, int32_t *kept, uint32_t *keys, int64_t cap,
                               cudaStream_t stream)
{
    if (c.B == 0)
        return cudaSuccess;
    cache_select_kernel<<<c.B, kSelThreads, 0, stream>>>(c, keep, first, recent, new_pages, new_table, new_lens, kept,
                                                         keys, cap);
    if (c.max_cache_len > keep) {
        const int blocks = std::min((keep + kPage - 1) / kPage, c.max_pages);
        switch (c.d) {
        case 32: move<32>(c, keep, blocks, new_pages, kept, stream); break;
        case 64: move<64>(c, keep, blocks, new_pages, kept, stream); break;
        default: move<128>(c, keep, blocks, new_pages, kept, stream); break;
        }
    }
    return cudaGetLastError();
}

}  // namespace hstu
