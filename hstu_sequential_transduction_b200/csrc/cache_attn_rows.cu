// Attention of a few query rows (single tokens, short chunks) over the 8-bit cache.
//
//   O_i = inv_n sum_j SiLU(q_i . k_j + bias_ij) v_j,   a_j += |inv_n| sum_ih |SiLU|
//
// Bound by HBM: the codes of a page (64 d bytes of keys, as many of values per head)
// are read once for all rows, straight into the registers of one warp, with no
// staging and no shuffles: a page's layouts (keys [64][d], values [d][64]) are the
// column-major B operands of the 16-bit matrix instructions, and the order of the
// contracted index is free, so a lane's 16-byte load is four instructions' operand:
//   S = Q K^T: lane (g, t) = (lane / 4, lane % 4) loads bytes [64 c + 16 t, + 16) of
//   key row 16 (g / 2) + 2 n + g % 2 for tile n; dims 4 u .. 4 u + 3 of that load
//   serve step (c, u).  The result then holds row g, keys 16 t + 2 n, + 1;
//   O = P V: which is the A operand for keys 16 t + 4 s .. + 3 of step s, word s of
//   the 16-byte load at keys 16 t of value row (dim) 8 n + g.
// Codes become f16 exactly.  q becomes f16 under a power of two per row that puts
// its largest magnitude into [2^14, 2^15): exact but for elements below 2^-28 of it.
// P becomes f16 under a power of two per page and row, of its largest magnitude, so
// its one rounding is 2^-11 of each value down to 2^-28 of the page's largest; each
// page's product starts from zero and is added to the float32 sums with the page's
// scale.  Legacy matrix instructions are enough: a page takes 128 of them per 16 KB.
#include <algorithm>

#include "cache.cuh"

namespace hstu {

namespace {

constexpr int kWarps = 4;
constexpr int kBiasLd = 68;  // floats of a row of staged biases

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

// 2^(14 - e) for a magnitude with exponent e (at least -100), and its inverse
__device__ __forceinline__ float to_range(float m, float *inverse)
{
    const int e = max((int)(__float_as_uint(m) >> 23 & 255), 27);
    *inverse = __int_as_float(max(e - 14, 1) << 23);
    return __int_as_float((268 - e) << 23);
}

__device__ __forceinline__ uint4 ldg_stream(const uint8_t *p)
{
    uint4 w;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];\n"
                 : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w)
                 : "l"(p));
    return w;
}

__device__ __forceinline__ uint32_t word(const uint4 &w, int i) { return i == 0 ? w.x : i == 1 ? w.y : i == 2 ? w.z : w.w; }

// RT: row tiles of 8 (1 or 2)
template <int D, int RT>
__global__ void __launch_bounds__(kWarps * 32, RT == 1 ? 2 : 1)
cache_attn_rows_kernel(const CacheAttnArgs a)
{
    constexpr int R = 8 * RT, NC = D / 64, KN = 8, VN = D / 8;
    extern __shared__ __align__(16) float smem[];
    __shared__ int row_pi[R];
    __shared__ int64_t row_ti[R];
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
    float *bias = smem + warp * R * kBiasLd;
    float *wplane = a.part_w ? a.part_w + ((int64_t)(tile * c.H + h) * c.B + b) * a.plan.lcap : nullptr;

    uint4 kr[KN * NC], vr[VN];
    auto load_k = [&](int page) {
        const uint8_t *kc = c.k_codes + block_offset<D>(page, c.H, h) + (16 * (g >> 1) + (g & 1)) * D + 16 * t;
#pragma unroll
        for (int n = 0; n < KN; n++)
#pragma unroll
            for (int cc = 0; cc < NC; cc++)
                kr[n * NC + cc] = ldg_stream(kc + 2 * n * D + 64 * cc);
    };
    auto load_v = [&](int page) {
        const uint8_t *vc = c.v_codes + block_offset<D>(page, c.H, h) + g * kPage + 16 * t;
#pragma unroll
        for (int n = 0; n < VN; n++)
            vr[n] = ldg_stream(vc + n * 8 * kPage);
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
        load_k(page);
        load_v(page);
    }
    if (threadIdx.x < R) {
        const int i = r0 + min((int)threadIdx.x, rows - 1);
        row_pi[threadIdx.x] = s.pos + token_pos(i, s.hist, a.cand_own);
        row_ti[threadIdx.x] = c.ts[s.s0 + i];
    }
    // q: for step (cc, u), dims 64 cc + 16 t + 4 u .. + 3 of rows g and g + 8
    uint32_t qf[4 * NC][2 * RT];
    float qinv[RT];
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
        const float f = to_range(m, &qinv[rt]);
#pragma unroll
        for (int e = 0; e < 8 * NC; e++)  // word e: dims 2 e, 2 e + 1 of the lane's 16 NC
            qf[e >> 1][rt + RT * (e & 1)] =
                pack_f16(__uint_as_float(w[e] << 16) * f, __uint_as_float(w[e] & 0xffff0000u) * f);
    }
    float o[VN][2 * RT];
#pragma unroll
    for (int n = 0; n < VN; n++)
#pragma unroll
        for (int e = 0; e < 2 * RT; e++)
            o[n][e] = 0.f;
    const float *rp = a.rab_pos + h * a.pos_hstride, *rt_ = a.rab_time + h * a.time_hstride;
    __syncthreads();
    for (; p < p1; p += kWarps) {
        const int count = min(s.len - p * kPage, kPage);
        const int next = page_of(p + kWarps);
        if (page < 0) {
            if (wplane)
                for (int j = lane; j < count; j += 32)
                    wplane[p * kPage + j] = 0.f;
            page = next;
            if (page >= 0) {
                load_k(page);
                load_v(page);
            }
            continue;
        }
        const float ks = c.k_scale[(int64_t)page * c.H + h], vs = c.v_scale[(int64_t)page * c.H + h];
        // biases of keys lane and lane + 32 for every row
        __syncwarp();
#pragma unroll
        for (int e = 0; e < 2; e++) {
            const int64_t at = (int64_t)page * kPage + lane + 32 * e;
            const int pj = c.positions[at];
            const int64_t tj = c.timestamps[at];
            for (int r = 0; r < rows; r++)
                bias[r * kBiasLd + lane + 32 * e] =
                    rp[pos_index(row_pi[r], pj, a.pos_lo, a.pos_hi)] + rt_[time_bucket(row_ti[r], tj, a.nb)];
        }
        __syncwarp();
        float sc[KN][4];
#pragma unroll
        for (int n = 0; n < KN; n++) {
            sc[n][0] = sc[n][1] = sc[n][2] = sc[n][3] = 0.f;
#pragma unroll
            for (int u = 0; u < 4 * NC; u++) {
                const uint32_t w = word(kr[n * NC + (u >> 2)], u & 3);
                uint32_t af[4] = {qf[u][0], 0u, qf[u][RT], 0u};
                if (RT == 2) {
                    af[1] = qf[u][1];
                    af[3] = qf[u][RT + 1];
                }
                mma_f16(sc[n], af, e4m3x2_to_f16x2(w), e4m3x2_to_f16x2(w >> 16));
            }
        }
        if (next >= 0)
            load_k(next);
        // P of rows g (and g + 8), keys 16 t + 2 n, + 1
        uint32_t pf[KN][RT];
        float pinv[RT], wsum[2 * KN];
#pragma unroll
        for (int e = 0; e < 2 * KN; e++)
            wsum[e] = 0.f;
#pragma unroll
        for (int rt = 0; rt < RT; rt++) {
            const bool live = g + 8 * rt < rows;
            const float f = 0.5f * ks * qinv[rt];
            const float *br = bias + (g + 8 * rt) * kBiasLd + 16 * t;
            float pv[2 * KN], m = 0.f;
#pragma unroll
            for (int e4 = 0; e4 < 2 * KN; e4 += 4) {
                const float4 b4 = live ? *reinterpret_cast<const float4 *>(br + e4) : make_float4(0.f, 0.f, 0.f, 0.f);
                const float bb[4] = {b4.x, b4.y, b4.z, b4.w};
#pragma unroll
                for (int e = e4; e < e4 + 4; e++) {
                    const float hh = fmaf(sc[e >> 1][2 * rt + (e & 1)], f, 0.5f * bb[e - e4]);
                    float th;
                    asm("tanh.approx.f32 %0, %1;" : "=f"(th) : "f"(hh));
                    pv[e] = live && 16 * t + e < count ? fmaf(hh, th, hh) : 0.f;
                    m = fmaxf(m, fabsf(pv[e]));
                    wsum[e] += fabsf(pv[e]);
                }
            }
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
            const float pr = to_range(m, &pinv[rt]);
#pragma unroll
            for (int n = 0; n < KN; n++)
                pf[n][rt] = pack_f16(pv[2 * n] * pr, pv[2 * n + 1] * pr);
            pinv[rt] *= vs;
        }
        if (wplane) {
            if (rows > 1) {
#pragma unroll
                for (int e = 0; e < 2 * KN; e++) {
                    wsum[e] += __shfl_xor_sync(0xffffffffu, wsum[e], 4);
                    wsum[e] += __shfl_xor_sync(0xffffffffu, wsum[e], 8);
                    wsum[e] += __shfl_xor_sync(0xffffffffu, wsum[e], 16);
                }
            }
            if (g == 0)
#pragma unroll
                for (int e = 0; e < 2 * KN; e += 4)  // behind the end: zeros, within the plane's whole pages
                    *reinterpret_cast<float4 *>(wplane + p * kPage + 16 * t + e) =
                        make_float4(wsum[e], wsum[e + 1], wsum[e + 2], wsum[e + 3]);
        }
        if (count < kPage) {  // codes behind the last token may be anything
            const int n = count - 16 * t;
            uint32_t m[4];
#pragma unroll
            for (int e = 0; e < 4; e++)
                m[e] = n >= 4 * e + 4 ? 0xffffffffu : n <= 4 * e ? 0u : (1u << (8 * (n - 4 * e))) - 1u;
#pragma unroll
            for (int i = 0; i < VN; i++)
                vr[i] = make_uint4(vr[i].x & m[0], vr[i].y & m[1], vr[i].z & m[2], vr[i].w & m[3]);
        }
#pragma unroll
        for (int n = 0; n < VN; n++) {
            float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int st = 0; st < 4; st++) {
                const uint32_t w = word(vr[n], st);
                uint32_t af[4] = {pf[2 * st][0], 0u, pf[2 * st + 1][0], 0u};
                if (RT == 2) {
                    af[1] = pf[2 * st][RT - 1];
                    af[3] = pf[2 * st + 1][RT - 1];
                }
                mma_f16(acc, af, e4m3x2_to_f16x2(w), e4m3x2_to_f16x2(w >> 16));
            }
#pragma unroll
            for (int e = 0; e < 2 * RT; e++)
                o[n][e] = fmaf(acc[e], pinv[e >> 1], o[n][e]);
        }
        if (next >= 0)
            load_v(next);
        page = next;
    }
    // the warps' sums, in order
    __syncthreads();
#pragma unroll
    for (int rt = 0; rt < RT; rt++)
        if (g + 8 * rt < rows)
#pragma unroll
            for (int n = 0; n < VN; n++)
                *reinterpret_cast<float2 *>(smem + (warp * R + g + 8 * rt) * D + 8 * n + 2 * t) =
                    make_float2(o[n][2 * rt], o[n][2 * rt + 1]);
    __syncthreads();
    for (int i = threadIdx.x; i < rows * D; i += kWarps * 32) {
        float sum = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; w++)
            sum += smem[w * R * D + i];
        a.part_o[(((int64_t)part * c.T + s.s0 + r0 + i / D) * c.H + h) * D + i % D] = sum;
    }
}

template <int D, int RT>
cudaError_t rows_launch(const CacheAttnArgs &a, cudaStream_t stream)
{
    constexpr int bytes = kWarps * 8 * RT * std::max(D, kBiasLd) * 4;
    static_assert(bytes <= 48 * 1024, "within the default dynamic shared memory");
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
