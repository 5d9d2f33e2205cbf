// Attention of a few query rows (single tokens, short chunks) over the 8-bit cache.
//
//   O_i = inv_n sum_j SiLU(q_i . k_j + bias_ij) v_j,   a_j += |inv_n| sum_ih |SiLU|
//
// Bound by HBM: the codes of a page (64 d bytes of keys, as many of values per head) are
// read once for all rows.  A warp has a buffer for one block of keys and one of values,
// filled by bulk copies: while the values are used the next keys are on their way, and
// the other way round; three CTAs of four warps keep some 100 KB an SM in flight.
// (Loaded straight into registers, the blocks left two warps a scheduler: 4.1 TB/s.)
// Keys and dims are the rows of the 16-bit matrix instructions, the queries their eight
// columns, so that a page of d = 128 takes 64 of them for eight queries (with queries as
// the sixteen rows it took 128, and those were the bound: 200 us where this takes 160).
//   S^T = K Q^T, O^T = V^T P^T
// A page's layouts (keys [64][d], values [d][64]) are row-major A operands, and the order
// of the contracted index is free, so a lane's 16-byte read is four instructions' operand:
// lane (g, t) = (lane / 4, lane % 4) reads bytes [64 c + 16 t, + 16) of the key rows
// 16 (g / 2) + 4 m + g % 2 and + 2 for tile m, and bytes [16 t, + 16) (keys) of value rows
// 16 n + g and + 8.  Tile m of S^T then holds, after an 8 x 8 transposition in the warp,
// the B operand for word m of the values.
// Codes become f16 exactly.  q becomes f16 under a power of two per row that puts
// its largest magnitude into [2^14, 2^15): exact but for elements below 2^-28 of it.
// P becomes f16 under a power of two per page and row, of its largest magnitude, so
// its one rounding is 2^-11 of each value down to 2^-28 of the page's largest; each
// page's product starts from zero and is added to the float32 sums with the page's
// scale.
#include <algorithm>

#include "cache.cuh"
#include "tc_common.cuh"

namespace hstu {

namespace {

constexpr int kWarps = 4;
__device__ __forceinline__ void mma_f16(float *d, const uint32_t *a, uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi)
{
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}

// 8 x 8 transposition in the warp: lane (g, t) gives row g, columns 2 t, + 1
__device__ __forceinline__ uint32_t transpose8(uint32_t x)
{
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(y) : "r"(x));
    return y;
}

// 2^(14 - e) for a magnitude with exponent e (at least -100), and its inverse
__device__ __forceinline__ float to_range(float m, float *inverse)
{
    const int e = max((int)(__float_as_uint(m) >> 23 & 255), 27);
    *inverse = __int_as_float(max(e - 14, 1) << 23);
    return __int_as_float((268 - e) << 23);
}

// untiled copy of `bytes` (a multiple of 16) to shared memory
__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}

__device__ __forceinline__ uint32_t word(const uint4 &w, int i) { return i == 0 ? w.x : i == 1 ? w.y : i == 2 ? w.z : w.w; }

// RT: row tiles of 8 (1 or 2)
template <int D, int RT>
__global__ void __launch_bounds__(kWarps * 32, RT == 1 || D == 64 ? 3 : 2)
cache_attn_rows_kernel(const CacheAttnArgs a)
{
    constexpr int R = 8 * RT, NC = D / 64, VN = D / 16, kBiasLd = R + 2;
    constexpr int kBlock = kPage * D, kBiasRows = 8;
    extern __shared__ __align__(16) unsigned char smem[];  // blocks of keys and values per warp, biases
    __shared__ int row_pi[R];
    __shared__ int64_t row_ti[R];
    __shared__ __align__(8) uint64_t bars[kWarps][2];
    __shared__ volatile int abort_flag;
    const CacheCall &c = a.c;
    int x = blockIdx.x;
    const int h = x % c.H;
    x /= c.H;
    const int tile = x % a.plan.qtiles;  // of R query rows
    x /= a.plan.qtiles;
    const int part = x % a.plan.nsplit, b = x / a.plan.nsplit;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const CacheSeq s = cache_seq(c, b);
    const int r0 = tile * R, rows = min(s.n - r0, R);
    const int p0 = part * a.plan.split_pages, p1 = min((s.len + kPage - 1) / kPage, p0 + a.plan.split_pages);
    if (rows <= 0 || p0 >= p1)
        return;
    float *bias = reinterpret_cast<float *>(smem + kWarps * 2 * kBlock) + warp * kPage * kBiasLd;
    float *wplane = a.part_w ? a.part_w + ((int64_t)(tile * c.H + h) * c.B + b) * a.plan.lcap : nullptr;
    const unsigned char *kbuf = smem + warp * 2 * kBlock, *vbuf = kbuf + kBlock;
    const uint32_t kbar = smem_u32(&bars[warp][0]), vbar = smem_u32(&bars[warp][1]);
    if (lane == 0) {
        mbar_init(kbar, 1);
        mbar_init(vbar, 1);
        if (warp == 0)
            abort_flag = 0;
        fence_mbar_init();
    }
    __syncwarp();
    // by one lane, once the warp is done with what the buffer held
    auto load = [&](const uint8_t *codes, const unsigned char *buf, uint32_t bar, int page) {
        __syncwarp();
        if (lane == 0) {
            mbar_expect_tx(bar, kBlock);
            bulk_load(smem_u32(buf), codes + block_offset<D>(page, c.H, h), kBlock, bar);
        }
    };
    auto page_of = [&](int p) {
        if (p >= p1)
            return -1;
        const int page = table_page(c.table, c, b, p);
        if (page < 0 && h == 0 && tile == 0 && lane == 0)
            atomicOr(&c.hdr->flag, FLAG_CACHE_PAGE);
        return page;
    };
    int p = p0 + warp;
    int page = page_of(p);
    if (page >= 0) {
        if (!(a.withhold && blockIdx.x == 0 && warp == 0))
            load(c.k_codes, kbuf, kbar, page);
        load(c.v_codes, vbuf, vbar, page);
    }
    if (threadIdx.x < R) {
        const int i = r0 + min((int)threadIdx.x, rows - 1);
        row_pi[threadIdx.x] = s.pos + token_pos(i, s.hist, a.cand_own);
        row_ti[threadIdx.x] = c.ts[s.s0 + i];
    }
    // q: for step (cc, u), dims 64 cc + 16 t + 4 u .. + 3 of rows g and g + 8
    uint32_t qf[4 * NC][2 * RT];
    float qinv[RT][2];  // of queries 8 rt + 2 t, + 1
#pragma unroll
    for (int rt = 0; rt < RT; rt++) {
        const bool live = g + 8 * rt < rows;
        const __nv_bfloat16 *qp =
            static_cast<const __nv_bfloat16 *>(a.q) + (s.s0 + r0 + (live ? g + 8 * rt : 0)) * a.ldq + (int64_t)h * D + 16 * t;
        uint32_t w[8 * NC];
        float m = 0.f;
#pragma unroll
        for (int e = 0; e < 2 * NC; e++) {
            uint4 y = make_uint4(0u, 0u, 0u, 0u);
            if (live)
                y = *reinterpret_cast<const uint4 *>(qp + (e >> 1) * 64 + 8 * (e & 1));
            w[4 * e] = y.x, w[4 * e + 1] = y.y, w[4 * e + 2] = y.z, w[4 * e + 3] = y.w;
        }
#pragma unroll
        for (int e = 0; e < 8 * NC; e++)
            m = fmaxf(m, fmaxf(fabsf(__uint_as_float(w[e] << 16)), fabsf(__uint_as_float(w[e] & 0xffff0000u))));
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
        float inv;
        const float f = to_range(m, &inv);
#pragma unroll
        for (int e = 0; e < 2; e++)
            qinv[rt][e] = __shfl_sync(0xffffffffu, inv, 4 * (2 * t + e));
#pragma unroll
        for (int e = 0; e < 8 * NC; e++)  // word e: dims 2 e, 2 e + 1 of the lane's 16 NC
            qf[e >> 1][2 * rt + (e & 1)] =
                pack_f16(__uint_as_float(w[e] << 16) * f, __uint_as_float(w[e] & 0xffff0000u) * f);
    }
    float o[RT][VN][4];  // dims 16 n + g (+ 8), queries 8 rt + 2 t, + 1
#pragma unroll
    for (int rt = 0; rt < RT; rt++)
#pragma unroll
        for (int n = 0; n < VN; n++)
#pragma unroll
            for (int e = 0; e < 4; e++)
                o[rt][n][e] = 0.f;
    const float *rp = a.rab_pos + h * a.pos_hstride, *rt_ = a.rab_time + h * a.time_hstride;
    __syncthreads();
    bool ok = true;
    uint32_t loads = 0;  // blocks of each kind used so far
    for (; p < p1; p += kWarps) {
        const int count = min(s.len - p * kPage, kPage);
        const int next = page_of(p + kWarps);
        if (page < 0) {
            if (wplane)
                for (int j = lane; j < count; j += 32)
                    wplane[p * kPage + j] = 0.f;
            page = next;
            if (page >= 0) {
                load(c.k_codes, kbuf, kbar, page);
                load(c.v_codes, vbuf, vbar, page);
            }
            continue;
        }
        const float ks = c.k_scale[(int64_t)page * c.H + h], vs = c.v_scale[(int64_t)page * c.H + h];
        // biases of keys lane and lane + 32 for every row, the table reads of eight rows in flight
        __syncwarp();
        int pj[2];
        int64_t tj[2];
#pragma unroll
        for (int e = 0; e < 2; e++) {
            const int64_t at = (int64_t)page * kPage + lane + 32 * e;
            pj[e] = c.positions[at];
            tj[e] = c.timestamps[at];
        }
        if (rows == 1) {
#pragma unroll
            for (int e = 0; e < 2; e++)
                bias[(lane + 32 * e) * kBiasLd] =
                    rp[pos_index(row_pi[0], pj[e], a.pos_lo, a.pos_hi)] + rt_[time_bucket(row_ti[0], tj[e], a.nb)];
        } else {
#pragma unroll 1
            for (int r = 0; r < rows; r += kBiasRows) {  // rows behind the last repeat it
                float bp[2 * kBiasRows], bt[2 * kBiasRows];
#pragma unroll
                for (int x = 0; x < 2 * kBiasRows; x++) {
                    bp[x] = rp[pos_index(row_pi[r + (x >> 1)], pj[x & 1], a.pos_lo, a.pos_hi)];
                    bt[x] = rt_[time_bucket(row_ti[r + (x >> 1)], tj[x & 1], a.nb)];
                }
#pragma unroll
                for (int x = 0; x < 2 * kBiasRows; x++)
                    bias[(lane + 32 * (x & 1)) * kBiasLd + r + (x >> 1)] = bp[x] + bt[x];
            }
        }
        __syncwarp();
        if (!(ok = __all_sync(0xffffffffu, mbar_wait(kbar, loads & 1, &abort_flag, c.hdr, a.wait_limit)))) {
            mbar_drain(kbar, loads & 1);
            mbar_drain(vbar, loads & 1);
            break;
        }
        float sc[RT][4][4];  // keys of tile m: 16 (g / 2) + 4 m + g % 2 (+ 2), queries 2 t, + 1
        const int key0 = 16 * (g >> 1) + (g & 1);
        const unsigned char *krow = kbuf + key0 * D + 16 * t;
#pragma unroll
        for (int m = 0; m < 4; m++) {
            uint4 ka[NC], kb[NC];
#pragma unroll
            for (int cc = 0; cc < NC; cc++) {
                ka[cc] = *reinterpret_cast<const uint4 *>(krow + 4 * m * D + 64 * cc);
                kb[cc] = *reinterpret_cast<const uint4 *>(krow + (4 * m + 2) * D + 64 * cc);
            }
#pragma unroll
            for (int rt = 0; rt < RT; rt++)
                sc[rt][m][0] = sc[rt][m][1] = sc[rt][m][2] = sc[rt][m][3] = 0.f;
#pragma unroll
            for (int u = 0; u < 4 * NC; u++) {
                const uint32_t wa = word(ka[u >> 2], u & 3), wb = word(kb[u >> 2], u & 3);
                const uint32_t af[4] = {e4m3x2_to_f16x2(wa), e4m3x2_to_f16x2(wb), e4m3x2_to_f16x2(wa >> 16),
                                        e4m3x2_to_f16x2(wb >> 16)};
#pragma unroll
                for (int rt = 0; rt < RT; rt++)
                    mma_f16(sc[rt][m], af, qf[u][2 * rt], qf[u][2 * rt + 1]);
            }
        }
        if (next >= 0)
            load(c.k_codes, kbuf, kbar, next);
        // P^T: the B operand of word m is keys 16 t + 4 m .. + 3 of query g
        uint32_t pf[RT][4][2];
        float pinv[RT][2], wsum[8];
#pragma unroll
        for (int e = 0; e < 8; e++)
            wsum[e] = 0.f;
#pragma unroll
        for (int rt = 0; rt < RT; rt++) {
            const bool live[2] = {8 * rt + 2 * t < rows, 8 * rt + 2 * t + 1 < rows};
            const float f[2] = {0.5f * ks * qinv[rt][0], 0.5f * ks * qinv[rt][1]};
            float m[2] = {0.f, 0.f};
#pragma unroll
            for (int i = 0; i < 8; i++) {  // key key0 + 4 (i / 2) + 2 (i % 2)
                const int key = key0 + 2 * i;
                const float2 bb = *reinterpret_cast<const float2 *>(bias + key * kBiasLd + 8 * rt + 2 * t);
                float *y = &sc[rt][i >> 1][2 * (i & 1)];
#pragma unroll
                for (int e = 0; e < 2; e++) {
                    const float hh = fmaf(y[e], f[e], 0.5f * (e ? bb.y : bb.x));
                    y[e] = live[e] && key < count ? fmaf(hh, tanh_approx(hh), hh) : 0.f;
                    m[e] = fmaxf(m[e], fabsf(y[e]));
                    wsum[i] += fabsf(y[e]);
                }
            }
            float pr[2];
#pragma unroll
            for (int e = 0; e < 2; e++) {
#pragma unroll
                for (int x = 4; x < 32; x <<= 1)
                    m[e] = fmaxf(m[e], __shfl_xor_sync(0xffffffffu, m[e], x));
                pr[e] = to_range(m[e], &pinv[rt][e]);
                pinv[rt][e] *= vs;
            }
#pragma unroll
            for (int i = 0; i < 8; i++)
                pf[rt][i >> 1][i & 1] = transpose8(pack_f16(sc[rt][i >> 1][2 * (i & 1)] * pr[0], sc[rt][i >> 1][2 * (i & 1) + 1] * pr[1]));
        }
        if (wplane) {
#pragma unroll
            for (int i = 0; i < 8; i++) {
                if (rows > 2) {
                    wsum[i] += __shfl_xor_sync(0xffffffffu, wsum[i], 1);
                    wsum[i] += __shfl_xor_sync(0xffffffffu, wsum[i], 2);
                }
                if (t == 0)  // behind the end: zeros, within the plane's whole pages
                    wplane[p * kPage + key0 + 2 * i] = wsum[i];
            }
        }
        if (!(ok = __all_sync(0xffffffffu, mbar_wait(vbar, loads & 1, &abort_flag, c.hdr, a.wait_limit)))) {
            mbar_drain(kbar, (loads + (next >= 0)) & 1);
            mbar_drain(vbar, loads & 1);
            break;
        }
        uint32_t keep[4];  // codes behind the last token may be anything
#pragma unroll
        for (int e = 0; e < 4; e++) {
            const int n = count - 16 * t - 4 * e;
            keep[e] = n >= 4 ? 0xffffffffu : n <= 0 ? 0u : (1u << (8 * n)) - 1u;
        }
        const unsigned char *vrow = vbuf + g * kPage + 16 * t;
#pragma unroll
        for (int n = 0; n < VN; n++) {
            const uint4 va = *reinterpret_cast<const uint4 *>(vrow + n * 16 * kPage);
            const uint4 vb = *reinterpret_cast<const uint4 *>(vrow + (n * 16 + 8) * kPage);
            float acc[RT][4];
#pragma unroll
            for (int rt = 0; rt < RT; rt++)
                acc[rt][0] = acc[rt][1] = acc[rt][2] = acc[rt][3] = 0.f;
#pragma unroll
            for (int st = 0; st < 4; st++) {
                const uint32_t wa = word(va, st) & keep[st], wb = word(vb, st) & keep[st];
                const uint32_t af[4] = {e4m3x2_to_f16x2(wa), e4m3x2_to_f16x2(wb), e4m3x2_to_f16x2(wa >> 16),
                                        e4m3x2_to_f16x2(wb >> 16)};
#pragma unroll
                for (int rt = 0; rt < RT; rt++)
                    mma_f16(acc[rt], af, pf[rt][st][0], pf[rt][st][1]);
            }
#pragma unroll
            for (int rt = 0; rt < RT; rt++)
#pragma unroll
                for (int e = 0; e < 4; e++)
                    o[rt][n][e] = fmaf(acc[rt][e], pinv[rt][e & 1], o[rt][n][e]);
        }
        if (next >= 0)
            load(c.v_codes, vbuf, vbar, next);
        page = next;
        loads++;
    }
    // the warps' sums, in order
    __syncthreads();
    if (abort_flag)
        return;  // a copy never came: flagged, the output is incomplete
    float *sums = reinterpret_cast<float *>(smem);
#pragma unroll
    for (int rt = 0; rt < RT; rt++)
#pragma unroll
        for (int e = 0; e < 2; e++)
            if (8 * rt + 2 * t + e < rows)
#pragma unroll
                for (int n = 0; n < VN; n++) {
                    float *dst = sums + (warp * R + 8 * rt + 2 * t + e) * D + 16 * n + g;
                    dst[0] = o[rt][n][e];
                    dst[8] = o[rt][n][2 + e];
                }
    __syncthreads();
    for (int i = threadIdx.x; i < rows * D; i += kWarps * 32) {
        float sum = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; w++)
            sum += sums[w * R * D + i];
        a.part_o[(((int64_t)part * c.T + s.s0 + r0 + i / D) * c.H + h) * D + i % D] = sum;
    }
}

template <int D, int RT>
cudaError_t rows_launch(const CacheAttnArgs &a, cudaStream_t stream)
{
    constexpr int bytes = kWarps * (2 * kPage * D + kPage * (8 * RT + 2) * 4);
    static_assert(8 * RT * D * 4 <= 2 * kPage * D, "the sums fit where the blocks were");
    const cudaError_t e = cudaFuncSetAttribute(cache_attn_rows_kernel<D, RT>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess)
        return e;
    const int64_t grid = (int64_t)a.c.B * a.plan.nsplit * a.plan.qtiles * a.c.H;
    cache_attn_rows_kernel<D, RT><<<(unsigned)grid, kWarps * 32, bytes, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_cache_attn_rows(const CacheAttnArgs &a, cudaStream_t stream)
{
    if (a.c.max_seq_len <= 8)
        return a.c.d == 64 ? rows_launch<64, 1>(a, stream) : rows_launch<128, 1>(a, stream);
    return a.c.d == 64 ? rows_launch<64, 2>(a, stream) : rows_launch<128, 2>(a, stream);
}

}  // namespace hstu
