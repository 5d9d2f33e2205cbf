// Attention over the 8-bit key/value cache: the float32 kernel (CUDA cores), the join
// of the parts that the key axis is cut into, and the choice of kernel.
//
//   O_i = inv_n sum_j SiLU(q_i . k_j + bias_ij) v_j,   a_j += |inv_n| sum_ih |SiLU|
//
// One CTA takes 16 query rows of one (sequence, head) and a run of pages.  Scores:
// a thread owns a key (its codes decoded to registers) and half of the rows.
// Sums: a thread owns a dim and reads that dim's 64 codes of the transposed value
// page.  The pointwise SiLU needs no running maximum, so the parts of the key axis
// simply add; the join adds them in a fixed order.
#include <algorithm>

#include "cache.cuh"

namespace hstu {

namespace {

constexpr int kRows = 16;   // query rows of a CTA
constexpr int kThreads = 128;

__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }

// sixteen codes to floats
__device__ __forceinline__ void decode16(const uint4 w, float *x)
{
    const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int e = 0; e < 4; e++) {
        const float2 lo = e4m3x2_to_f32x2(ww[e]), hi = e4m3x2_to_f32x2(ww[e] >> 16);
        x[4 * e] = lo.x, x[4 * e + 1] = lo.y, x[4 * e + 2] = hi.x, x[4 * e + 3] = hi.y;
    }
}

template <int D>
__global__ void __launch_bounds__(kThreads)
cache_attn_f32_kernel(const CacheAttnArgs a)
{
    constexpr int RG = kThreads / D;       // row groups of the value product
    constexpr int NR = kRows / RG;
    __shared__ __align__(16) float sq[kRows][D], sp[kRows][kPage];
    __shared__ float sw[kPage];
    const CacheCall &c = a.c;
    int x = blockIdx.x;
    const int part = x % a.plan.nsplit;
    x /= a.plan.nsplit;
    const int h = x % c.H;
    x /= c.H;
    const int tile = x % a.plan.qtiles, b = x / a.plan.qtiles;
    const int tid = threadIdx.x;
    const CacheSeq s = cache_seq(c, b);
    const int r0 = tile * kRows, rows = min(s.n - r0, kRows);
    const int p0 = part * a.plan.split_pages, p1 = min((s.len + kPage - 1) / kPage, p0 + a.plan.split_pages);
    if (rows <= 0 || p0 >= p1)
        return;
    const float *q = static_cast<const float *>(a.q);
    for (int i = tid; i < kRows * D; i += kThreads)
        sq[i / D][i % D] = i / D < rows ? (q[(s.s0 + r0 + i / D) * a.ldq + (int64_t)h * D + i % D]) : 0.f;
    const float *rp = a.rab_pos + h * a.pos_hstride, *rt = a.rab_time + h * a.time_hstride;
    const int key = tid % kPage, half = tid / kPage;
    const int dim = tid % D, rg = tid / D;
    float o[NR];
#pragma unroll
    for (int r = 0; r < NR; r++)
        o[r] = 0.f;
    for (int p = p0; p < p1; p++) {
        const int page = table_page(c.table, c, b, p);
        const int count = min(s.len - p * kPage, kPage);
        float *wplane = a.part_w ? a.part_w + ((int64_t)(tile * c.H + h) * c.B + b) * a.plan.lcap + p * kPage : nullptr;
        if (page < 0) {
            if (h == 0 && tile == 0 && tid == 0)
                atomicOr(&c.hdr->flag, FLAG_CACHE_PAGE);
            if (wplane && tid < count)
                wplane[tid] = 0.f;
            continue;
        }
        __syncthreads();
        const bool live = key < count;
        float w = 0.f;
        float k[D];
        const uint8_t *kc = c.k_codes + block_offset<D>(page, c.H, h) + key * D;
#pragma unroll
        for (int e = 0; e < D; e += 16)
            decode16(*reinterpret_cast<const uint4 *>(kc + e), k + e);
        const float ks = c.k_scale[(int64_t)page * c.H + h], vs = c.v_scale[(int64_t)page * c.H + h];
        const int pj = c.positions[(int64_t)page * kPage + key];
        const int64_t tj = c.timestamps[(int64_t)page * kPage + key];
        for (int r = half; r < kRows; r += 2) {
            float pv = 0.f;
            if (r < rows && live) {
                float y = 0.f;
#pragma unroll
                for (int e = 0; e < D; e += 4) {
                    const float4 f = *reinterpret_cast<const float4 *>(&sq[r][e]);
                    y = fmaf(f.x, k[e], fmaf(f.y, k[e + 1], fmaf(f.z, k[e + 2], fmaf(f.w, k[e + 3], y))));
                }
                const int i = r0 + r;
                const int pi = s.pos + token_pos(i, s.hist, a.cand_own);
                y = fmaf(y, ks, rp[pos_index(pi, pj, a.pos_lo, a.pos_hi)] + rt[time_bucket(c.ts[s.s0 + i], tj, a.nb)]);
                pv = silu_precise(y);
                w += fabsf(pv);
            }
            sp[r][key] = pv * vs;
        }
        if (half == 1)
            sw[key] = w;
        __syncthreads();
        if (wplane && half == 0 && live)
            wplane[key] = w + sw[key];
        const uint8_t *vc = c.v_codes + block_offset<D>(page, c.H, h) + dim * kPage;
        for (int j = 0; j < count; j += 16) {
            float v[16];
            decode16(*reinterpret_cast<const uint4 *>(vc + j), v);
#pragma unroll
            for (int e = 0; e < 16; e++)  // slots behind the last token may hold anything
                v[e] = j + e < count ? v[e] : 0.f;
#pragma unroll
            for (int r = 0; r < NR; r++)
#pragma unroll
                for (int e = 0; e < 16; e++)
                    o[r] = fmaf(sp[rg * NR + r][j + e], v[e], o[r]);
        }
    }
#pragma unroll
    for (int r = 0; r < NR; r++) {
        const int i = rg * NR + r;
        if (i < rows)
            a.part_o[(((int64_t)part * c.T + s.s0 + r0 + i) * c.H + h) * D + dim] = o[r];
    }
}

__device__ __forceinline__ void put4(float *p, const float *y)
{
    *reinterpret_cast<float4 *>(p) = make_float4(y[0], y[1], y[2], y[3]);
}

__device__ __forceinline__ void put4(__nv_bfloat16 *p, const float *y)
{
    *reinterpret_cast<uint2 *>(p) = make_uint2(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]));
}

// Adds the parts: blocks [0, row_blocks * B) the output's rows, the others the weights.
template <typename T>
__global__ void __launch_bounds__(256)
cache_join_kernel(const CacheAttnArgs a, int row_blocks, int w_blocks)
{
    const CacheCall &c = a.c;
    const int64_t width = (int64_t)c.H * c.d;
    if ((int64_t)blockIdx.x < (int64_t)row_blocks * c.B) {
        const int b = blockIdx.x / row_blocks, chunk = blockIdx.x % row_blocks;
        const CacheSeq s = cache_seq(c, b);
        if (chunk == 0 && threadIdx.x == 0) {
            const int bits = s.bits | cache_offset_bits(c, b);
            if (bits)
                atomicOr(&c.hdr->flag, bits);
        }
        const int nsp = ((s.len + kPage - 1) / kPage + a.plan.split_pages - 1) / a.plan.split_pages;
        const int64_t e = ((int64_t)chunk * 256 + threadIdx.x) * 4;  // four elements of a row
        if (e >= (int64_t)s.n * width)
            return;
        const int64_t i = s.s0 * width + e;
        float y[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
        for (int p = 0; p < nsp; p++) {
            const float4 v = *reinterpret_cast<const float4 *>(a.part_o + p * c.T * width + i);
            y[0] += v.x, y[1] += v.y, y[2] += v.z, y[3] += v.w;
        }
        T *out = static_cast<T *>(a.out) + i;
        const T *add = static_cast<const T *>(a.addend);
#pragma unroll
        for (int k = 0; k < 4; k++)
            y[k] = y[k] * a.inv_n + (add ? to_float(add[i + k]) : 0.f);
        put4(out, y);
        return;
    }
    const int x = blockIdx.x - row_blocks * c.B;
    cache_join_weights(a, x / w_blocks, ((x % w_blocks) * 256 + threadIdx.x) * 4);
}

// A call without sequences: its offsets are one number, and every row is uncovered.
__global__ void cache_no_sequences_kernel(const int64_t *seq_offsets, int64_t T, WsHeader *hdr)
{
    hdr->flag = (seq_offsets[0] != 0 ? FLAG_OFFSET0 : 0) | (seq_offsets[0] != T ? FLAG_TOTAL : 0);
}

int row_blocks(const CacheCall &c)  // one at least: it reports a sequence that was dropped
{
    return (int)std::max<int64_t>(1, ((int64_t)c.max_seq_len * c.H * c.d + 1023) / 1024);
}

template <typename T>
cudaError_t join(const CacheAttnArgs &a, cudaStream_t stream)
{
    const CacheCall &c = a.c;
    const int rows = row_blocks(c), w_blocks = a.weights_out ? (c.max_cache_len + 1023) / 1024 : 0;
    cache_join_kernel<T><<<(unsigned)((rows + w_blocks) * c.B), 256, 0, stream>>>(a, rows, w_blocks);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_cache_no_sequences(const CacheCall &c, cudaStream_t stream)
{
    cache_no_sequences_kernel<<<1, 1, 0, stream>>>(c.seq_offsets, c.T, c.hdr);
    return cudaGetLastError();
}

CacheAttnPlan cache_attn_plan(const CacheCall &c, bool bf16, bool with_weights)
{
    CacheAttnPlan p{};
    const int64_t pages = (c.max_cache_len + kPage - 1) / kPage;
    const int64_t sms = device_info().sms;
    p.kernel = !bf16 ? CACHE_F32 : c.max_seq_len <= kCacheRows ? CACHE_ROWS : CACHE_TC;
    const int tile_rows = p.kernel == CACHE_TC ? kTcTile : kRows;
    p.qtiles = (c.max_seq_len + tile_rows - 1) / tile_rows;
    p.plane_rows = p.kernel == CACHE_TC ? 64 : kRows;
    const int64_t planes = (int64_t)(c.max_seq_len + p.plane_rows - 1) / p.plane_rows * c.H;
    p.lcap = pages * kPage;
    const int64_t units = (int64_t)c.B * c.H * p.qtiles;
    if (units > 0 && pages > 0 && p.kernel == CACHE_TC) {
        p.ctas = (int)std::min<int64_t>(sms, units * ((pages + 1) / 2));
        p.part_o_bytes = align256(sizeof(float) * 2 * p.ctas * (size_t)kTcTile * c.d);
        p.piece_bytes = align256(sizeof(CacheAttnPiece) * 2 * p.ctas);
    } else {
        // rows: a warp should have several pages to keep its loads going, but with few
        // units the pages spread over the SMs; float32: four rounds of the SMs
        const int64_t want = std::max<int64_t>(1, ((p.kernel == CACHE_ROWS ? 16 : 4) * sms + units - 1) / std::max<int64_t>(1, units));
        p.split_pages = (int)std::max<int64_t>(p.kernel == CACHE_ROWS ? 4 : 1, (pages + want - 1) / want);
        p.nsplit = (int)((pages + p.split_pages - 1) / p.split_pages);
        p.part_o_bytes = align256(sizeof(float) * (size_t)p.nsplit * c.T * c.H * c.d);
    }
    p.part_w_bytes = with_weights ? align256(sizeof(float) * (size_t)planes * c.B * p.lcap) : 0;
    return p;
}

bool cache_attn_fits(const CacheAttnArgs &a)
{
    const CacheCall &c = a.c;
    const double limit = 2147483647.0;
    const double w_blocks = (double)(a.plan.lcap / 256 + 1) * c.B;
    if (a.plan.kernel == CACHE_TC)  // TMA coordinates: rows of the pool's codes
        return (double)c.num_pages * c.H * std::max(kPage, c.d) < limit && w_blocks + c.B + 16.0 * a.plan.ctas < limit;
    return (double)c.B * a.plan.qtiles * c.H * a.plan.nsplit < limit &&
           ((double)c.max_seq_len * c.H * c.d / 1024 + 2) * c.B + w_blocks < limit;
}

cudaError_t launch_cache_attn(const CacheAttnArgs &a, bool bf16, cudaStream_t stream)
{
    if (a.c.B == 0)
        return launch_cache_no_sequences(a.c, stream);
    if (a.plan.kernel == CACHE_TC)
        return launch_cache_attn_tc(a, stream);
    const int64_t grid = (int64_t)a.c.B * a.plan.qtiles * a.c.H * a.plan.nsplit;
    cudaError_t e = cudaSuccess;
    if (grid > 0 && a.plan.kernel == CACHE_ROWS) {
        e = launch_cache_attn_rows(a, stream);
    } else if (grid > 0) {
        if (a.c.d == 32)
            cache_attn_f32_kernel<32><<<(unsigned)grid, kThreads, 0, stream>>>(a);
        else
            cache_attn_f32_kernel<64><<<(unsigned)grid, kThreads, 0, stream>>>(a);
        e = cudaGetLastError();
    }
    if (e != cudaSuccess)
        return e;
    return bf16 ? join<__nv_bfloat16>(a, stream) : join<float>(a, stream);
}

}  // namespace hstu
