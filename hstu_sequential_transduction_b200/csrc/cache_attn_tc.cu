// Attention of many query rows (ranking, long chunks) over the 8-bit cache on the
// tensor cores (TMA + tcgen05, bf16 queries).
//
//   O_i = inv_n sum_j SiLU(q_i . k_j + bias_ij) v_j,   a_j += |inv_n| sum_ih |SiLU|
//
// Transposed: a tile is 128 keys (two pages) by up to 128 queries of one head,
//   S^T = K Q^T   (E4M3, A = the keys' codes as TMA brings them, B = the queries)
//   O^T += V^T P^T (bf16, A = the values in TMEM, B = P^T in shared memory),
// so that a thread owns a key: its token's bias, scale and weight sum are scalars.
// Candidates share one position and mostly one stamp, so their bias costs nothing
// per pair, and the weight a token receives is one add per pair, no reduction.
//
// Keys stay codes: a query is split into two E4M3 parts, q = (q1 + q2) 2^e, q1 the
// nearest code, q2 the nearest code of what is left.  Two four-bit significands hold
// bf16's eight exactly; below 2^-6 of the scale the parts go subnormal, so an element
// is held to 2^-18.8 of the largest magnitude of its scale.  The scale is shared by
// the 32 rows of a chunk if no row's largest is 2^3 or more below theirs, else each
// row has its own.  E4M3 runs at twice the bf16 rate, so both parts cost what one
// bf16 product would, and no key is ever converted.
// Values become bf16 (exactly, with their page's scale) in registers on the way from
// memory to TMEM; P is rounded to bf16 once.
//
// Bound: per 128 x 128 tile at d = 128, 1024 cycles of the tensor pipe, of MUFU (one
// tanh per pair) and of shared-memory bandwidth (512 S^T operands, 256 P^T stores,
// 256 P^T reads) alike; V^T as a TMEM operand is what keeps the last at 1024.
//
// Warp roles (448 threads): warp 0 loads keys (TMA, four stages); warp 1 owns TMEM
// and issues the MMAs; warps 2-5 and 6-9 take the even and the odd tiles' S^T and
// write P^T; warps 10-13 split queries and convert values.
// TMEM columns: S^T [0, 128) and [128, 256), O^T [256, 384), V^T [384, 448), [448, 512).
//
// Work: all (sequence, head, query tile) units' key tiles in one line, cut into equal
// runs, one per CTA.  A unit inside one run is written to `out`; a cut unit's pieces
// go to the CTA's two slots (the unit it starts in the middle of, the unit it leaves
// unfinished), and the join adds them in order.
#include <cudaTypedefs.h>

#include <algorithm>

#include "cache.cuh"
#include "tc_common.cuh"

namespace hstu {

namespace {

constexpr int kTile = 128;    // keys of a tile, query columns of a unit
constexpr int kThreads = 448;
constexpr int kStages = 4;    // key tiles in flight
constexpr int kPanel = 16384; // 64 query columns of P^T: 128 keys x 128 bytes

enum Bars { K_FULL = 0, K_EMPTY = K_FULL + kStages, S_FULL = K_EMPTY + kStages, P_FULL = S_FULL + 2,
            P_EMPTY = P_FULL + 2, V_FULL = P_EMPTY + 2, V_EMPTY = V_FULL + 2, Q_FULL = V_EMPTY + 2,
            Q_EMPTY = Q_FULL + 2, O_FULL = Q_EMPTY + 2, O_FREE = O_FULL + 1, NBARS = O_FREE + 1 };

// what the epilogue needs to know of a unit's queries
struct QueryInfo {
    float chunk_scale[4];  // one scale of the 32 columns, or -1: each its own
    int chunk_same[4];     // every column has row 0's position and stamp
    float scale[kTile];
    int pos[kTile];
    int64_t ts[kTile];
};

template <int D>
struct Layout {
    static constexpr int KT = kTile * D;  // a key tile, one part of the queries
    static constexpr int Q = 0;           // two buffers of two parts
    static constexpr int K = Q + 4 * KT;
    static constexpr int P = K + kStages * KT;
    static constexpr int INFO = P + 4 * kPanel;
    static constexpr int BAR = INFO + 2 * (int)sizeof(QueryInfo);
    static constexpr int MISC = BAR + NBARS * 8;
    static constexpr int BYTES = MISC + 128 + 1024;
    static_assert(BYTES <= 227 * 1024, "shared memory of an SM");
};

// K-major operand of D-byte rows: the 128-byte swizzle for d = 128, the 64-byte one for d = 64
template <int D>
__device__ __forceinline__ uint64_t code_desc(uint32_t addr)
{
    uint64_t d = (addr >> 4) & 0x3FFF;
    d |= (uint64_t)1 << 16;
    d |= (uint64_t)((8 * D) >> 4) << 32;
    d |= (uint64_t)1 << 46;
    d |= (uint64_t)(D == 128 ? 2 : 4) << 61;
    return d;
}

template <int D>
__device__ __forceinline__ int code_chunk(int row, int chunk)
{
    return D == 128 ? chunk ^ (row & 7) : chunk ^ ((row >> 1) & 3);
}

struct Sizes {
    int qt, kt;  // query tiles, key tiles
    __device__ int64_t tiles(int H) const { return (int64_t)qt * kt * H; }
};

__device__ __forceinline__ Sizes sizes(const CacheSeq &s)
{
    return {(s.n + kTile - 1) / kTile, (s.len + kTile - 1) / kTile};
}

// A CTA's run of tiles: pieces of units one after the other.
struct Walk {
    int b, unit, k;  // unit = h * qt + query tile
    int64_t left;    // tiles of the run from here on
    int piece;       // pieces so far
    CacheSeq s;
    Sizes z;
    __device__ int count() const { return (int)min((int64_t)(z.kt - k), left); }
    __device__ int head() const { return unit / z.qt; }
    __device__ int q0() const { return unit % z.qt * kTile; }
    __device__ int cols() const { return min(s.n - q0(), kTile); }
    __device__ void load(const CacheCall &c)
    {
        s = cache_seq(c, b);
        z = sizes(s);
    }
    __device__ void next(const CacheCall &c)
    {
        left -= count();
        piece++;
        k = 0;
        if (left <= 0)
            return;
        if (++unit == z.qt * c.H) {
            unit = 0;
            do {
                b++;
                load(c);
            } while (z.qt * z.kt == 0);
        }
    }
};

// The sequence in whose tiles the run starts, and the run's length; false: no tiles.
__device__ bool find_run(const CacheCall &c, int cta, int ctas, int64_t *sums, int64_t *found)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    constexpr int kW = kThreads / 32;
    // every thread a run of sequences; sums over warps, then the run that holds the start
    const int per = (c.B + kThreads - 1) / kThreads;
    const int b0 = min(tid * per, c.B), b1 = min(b0 + per, c.B);
    int64_t mine = 0;
    for (int b = b0; b < b1; b++) {
        mine += sizes(cache_seq(c, b)).tiles(c.H);
    }
    int64_t inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o)
            inc += y;
    }
    if (lane == 31)
        sums[warp] = inc;
    __syncthreads();
    int64_t before = 0, total = 0;
    for (int w = 0; w < kW; w++) {
        if (w < warp)
            before += sums[w];
        total += sums[w];
    }
    const int64_t start = total * cta / ctas, end = total * (cta + 1) / ctas;
    int64_t at = before + inc - mine;
    if (start < end && start >= at && start < at + mine) {
        for (int b = b0; b < b1; b++) {
            const int64_t n = sizes(cache_seq(c, b)).tiles(c.H);
            if (start < at + n) {
                found[0] = b;
                found[1] = start - at;
                break;
            }
            at += n;
        }
    }
    if (tid == 0)
        found[2] = end - start;
    __syncthreads();
    return start < end;
}

// eight codes to bf16, times 2^120: each code's sign, exponent and fraction at bf16's places
__device__ __forceinline__ uint32_t code2_to_bf16(uint32_t spread)
{
    return (spread & 0x80008000u) | ((spread >> 4) & 0x07f007f0u);
}

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b)
{
    uint32_t d;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

__device__ __forceinline__ uint32_t pow2_bf16x2(int e)  // two copies of 2^e, -126 <= e <= 127
{
    const uint32_t x = (uint32_t)(e + 127) << 7;
    return x | (x << 16);
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
cache_attn_tc_kernel(const CacheAttnArgs a, const __grid_constant__ CUtensorMap tk)
{
    using LY = Layout<D>;
    extern __shared__ unsigned char smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    unsigned char *sm = smem_raw + (base - raw);
    const CacheCall &c = a.c;
    WsHeader *hdr = c.hdr;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    auto bar = [&](int i) { return base + LY::BAR + 8u * i; };
    volatile int *abort_flag = reinterpret_cast<volatile int *>(sm + LY::MISC + 8);
    QueryInfo *info = reinterpret_cast<QueryInfo *>(sm + LY::INFO);

    int64_t *found = reinterpret_cast<int64_t *>(sm + LY::MISC + 16);
    const bool work = find_run(c, blockIdx.x, gridDim.x, reinterpret_cast<int64_t *>(sm + LY::P), found);
    CacheAttnPiece *pieces = a.pieces + 2 * blockIdx.x;
    if (threadIdx.x < 2)  // no piece, unless one is recorded at its end
        pieces[threadIdx.x].cols = 0;
    if (!work)
        return;
    Walk start;
    start.b = (int)found[0];
    start.left = found[2];
    start.piece = 0;
    start.load(c);
    start.unit = (int)(found[1] / start.z.kt);
    start.k = (int)(found[1] % start.z.kt);
    if (threadIdx.x == 0) {
        for (int i = 0; i < NBARS; i++) {
            int n = 1;
            if (i == P_FULL || i == P_FULL + 1 || i == Q_FULL || i == Q_FULL + 1)
                n = 4;
            else if (i == V_FULL || i == V_FULL + 1)
                n = D / 32;
            else if (i == Q_EMPTY || i == Q_EMPTY + 1)
                n = 9;
            else if (i == O_FREE)
                n = 8;
            mbar_init(bar(i), n);
        }
        *abort_flag = 0;
        fence_mbar_init();
        tma_prefetch(&tk);
    }
    if (warp == 1)
        tmem_alloc(base + LY::MISC, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(sm + LY::MISC);
    bool ok = true;
    auto wait = [&](int i, int parity) { return mbar_wait(bar(i), parity & 1, abort_flag, hdr); };

    if (warp == 0) {
        // ---------------- keys ----------------
        if (lane == 0) {
            int g = 0;
            for (Walk w = start; ok && w.left > 0; w.next(c)) {
                const int h = w.head(), pages = (w.s.len + kPage - 1) / kPage;
                for (int k = w.k; k < w.k + w.count(); k++, g++) {
                    const int st = g % kStages;
                    if (g >= kStages && !(ok = wait(K_EMPTY + st, g / kStages - 1)))
                        break;
                    int page[2];
#pragma unroll
                    for (int e = 0; e < 2; e++) {
                        page[e] = -1;
                        if (2 * k + e < pages) {
                            page[e] = table_page(c.table, c, w.b, 2 * k + e);
                            if (page[e] < 0)
                                atomicOr(&hdr->flag, FLAG_CACHE_PAGE);
                        }
                    }
                    mbar_expect_tx(bar(K_FULL + st), ((page[0] >= 0) + (page[1] >= 0)) * kPage * D);
#pragma unroll
                    for (int e = 0; e < 2; e++)
                        if (page[e] >= 0)
                            tma_load_2d(base + LY::K + st * LY::KT + e * kPage * D, &tk, 0,
                                        (page[e] * c.H + h) * kPage, bar(K_FULL + st));
                }
            }
        }
    } else if (warp == 1) {
        // ---------------- MMAs ----------------
        if (lane == 0) {
            int issued = 0, done = 0, k = start.k;
            Walk w = start;
            uint32_t ring = 0;  // two tiles in flight: first, last, 128 columns; tile g in bits 4 (g & 1)
            auto next_s = [&]() {
                if (w.left <= 0)
                    return true;
                const int st = issued % kStages, sb = issued & 1, qs = w.piece & 1, n = w.cols() > 64 ? 128 : 64;
                const bool first = k == w.k, last = k + 1 == w.k + w.count();
                if (first && !wait(Q_FULL + qs, w.piece >> 1))
                    return false;
                if (!wait(K_FULL + st, issued / kStages))
                    return false;
                tc_fence_after();
                const uint32_t id = idesc_e4m3(128, 0, 0, 0) | ((uint32_t)(n >> 3) << 17);
#pragma unroll
                for (int part = 0; part < 2; part++)
#pragma unroll
                    for (int ks = 0; ks < D / 32; ks++)
                        umma_e4m3(tmem + sb * kTile, code_desc<D>(base + LY::K + st * LY::KT + ks * 32),
                                  code_desc<D>(base + LY::Q + (2 * qs + part) * LY::KT + ks * 32), id, part + ks > 0);
                umma_commit(bar(K_EMPTY + st));
                umma_commit(bar(S_FULL + sb));
                if (last)
                    umma_commit(bar(Q_EMPTY + qs));
                ring = (ring & ~(15u << (4 * sb))) | ((first | last << 1 | (n == 128) << 2) << (4 * sb));
                issued++;
                if (last) {
                    w.next(c);
                    k = w.k;
                } else {
                    k++;
                }
                return true;
            };
            int piece = 0;
            ok = next_s() && next_s();
            while (ok && done < issued) {
                const int sb = done & 1;
                const uint32_t r = ring >> (4 * sb);
                ok = wait(P_FULL + sb, done >> 1) && wait(V_FULL + sb, done >> 1) &&
                     (!(r & 1) || piece == 0 || wait(O_FREE, piece - 1));
                if (!ok)
                    break;
                tc_fence_after();
                const uint32_t id = idesc_bf16(128, 0, 0, 1) | ((uint32_t)((r & 4 ? 128 : 64) >> 3) << 17);
#pragma unroll
                for (int ks = 0; ks < kTile / 16; ks++)
                    umma_bf16_ts(tmem + 256, tmem + 384 + sb * 64 + ks * 8,
                                 smem_desc_sw128(base + LY::P + sb * 2 * kPanel + ks * 2048, kPanel, 1024), id,
                                 !(r & 1) || ks > 0);
                umma_commit(bar(V_EMPTY + sb));
                umma_commit(bar(P_EMPTY + sb));
                if (r & 2) {
                    umma_commit(bar(O_FULL));
                    piece++;
                }
                done++;
                ok = next_s();
            }
        }
    } else if (warp >= 10) {
        // ---------------- queries and values ----------------
        const int quarter = warp & 3, dim = quarter * 32 + lane;
        const int row = threadIdx.x - 320;  // of the queries
        int g = 0;
        for (Walk w = start; ok && w.left > 0; w.next(c)) {
            const int qs = w.piece & 1, h = w.head(), q0 = w.q0(), cols = w.cols();
            if (w.piece >= 2 && !(ok = wait(Q_EMPTY + qs, (w.piece >> 1) - 1)))
                break;
            {
                QueryInfo &qi = info[qs];
                const bool have = row < cols;
                const __nv_bfloat16 *qp =
                    static_cast<const __nv_bfloat16 *>(a.q) + (w.s.s0 + q0 + (have ? row : 0)) * a.ldq + (int64_t)h * D;
                uint32_t m = 0;  // largest magnitude as bf16 bits
                uint4 x[D / 8];
#pragma unroll
                for (int e = 0; e < D / 8; e++) {
                    x[e] = make_uint4(0u, 0u, 0u, 0u);
                    if (have)
                        x[e] = *reinterpret_cast<const uint4 *>(qp + 8 * e);
                    const uint32_t ww[4] = {x[e].x, x[e].y, x[e].z, x[e].w};
#pragma unroll
                    for (int i = 0; i < 4; i++)
                        m = max(m, max((ww[i] & 0x7fffu) << 16, ww[i] & 0x7fff0000u));
                }
                const uint32_t all = __reduce_max_sync(0xffffffffu, m);
                // one scale for the warp's rows if none lies far below
                const bool far = m != 0 && (int)(all >> 23) - (int)(m >> 23) > 2;
                const bool one = !__any_sync(0xffffffffu, far);
                const float scale = block_scale(one ? all : m), inv = scale_inverse(scale);
                const int i0 = q0, i = q0 + (have ? row : 0);
                const int pi = w.s.pos + token_pos(i, w.s.hist, a.cand_own);
                const int64_t ti = c.ts[w.s.s0 + i];
                const bool same = pi == w.s.pos + token_pos(i0, w.s.hist, a.cand_own) && ti == c.ts[w.s.s0 + i0];
                const bool all_same = __all_sync(0xffffffffu, same);
                qi.scale[row] = scale;
                qi.pos[row] = pi;
                qi.ts[row] = ti;
                if (lane == 0) {
                    qi.chunk_scale[row >> 5] = one ? scale : -1.f;
                    qi.chunk_same[row >> 5] = all_same;
                }
                unsigned char *q1 = sm + LY::Q + 2 * qs * LY::KT + row * D, *q2 = q1 + LY::KT;
#pragma unroll
                for (int e = 0; e < D / 16; e++) {
                    const uint32_t ww[8] = {x[2 * e].x, x[2 * e].y, x[2 * e].z, x[2 * e].w,
                                            x[2 * e + 1].x, x[2 * e + 1].y, x[2 * e + 1].z, x[2 * e + 1].w};
                    uint32_t hi[4], lo[4];
#pragma unroll
                    for (int i4 = 0; i4 < 4; i4++) {
                        hi[i4] = lo[i4] = 0;
#pragma unroll
                        for (int e2 = 0; e2 < 2; e2++) {
                            const uint32_t y = ww[2 * i4 + e2];
                            const float y0 = __uint_as_float(y << 16) * inv, y1 = __uint_as_float(y & 0xffff0000u) * inv;
                            const uint32_t p = f32x2_to_e4m3x2(y0, y1);
                            const float2 f = e4m3x2_to_f32x2(p);
                            hi[i4] |= p << (16 * e2);
                            lo[i4] |= f32x2_to_e4m3x2(y0 - f.x, y1 - f.y) << (16 * e2);
                        }
                    }
                    const int at = code_chunk<D>(row, e) * 16;
                    *reinterpret_cast<uint4 *>(q1 + at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                    *reinterpret_cast<uint4 *>(q2 + at) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(bar(Q_FULL + qs));
            }
            if (dim >= D) {  // d = 64 has half the rows of V^T
                g += w.count();
                continue;
            }
            const int k1 = w.k + w.count();
            // this dim's codes of a page (zeros behind the end and for a missing page) and the page's scale
            auto fetch = [&](int p, uint4 *v, int *scale_exp) {
                const int n = w.s.len - p * kPage;
                const int page = n > 0 ? table_page(c.table, c, w.b, p) : -1;
                float sc = 0.f;
#pragma unroll
                for (int e = 0; e < 4; e++)
                    v[e] = make_uint4(0u, 0u, 0u, 0u);
                if (page >= 0) {
                    const uint8_t *vc = c.v_codes + block_offset<D>(page, c.H, h) + dim * kPage;
                    sc = c.v_scale[(int64_t)page * c.H + h];
#pragma unroll
                    for (int e = 0; e < 4; e++)
                        v[e] = *reinterpret_cast<const uint4 *>(vc + 16 * e);
                }
                *scale_exp = __float_as_int(sc);
            };
            uint4 v[2][4];
            int sc[2];
            fetch(2 * w.k, v[0], &sc[0]);
            fetch(2 * w.k + 1, v[1], &sc[1]);
            for (int k = w.k; k < k1; k++, g++) {
                const int vb = g & 1;
                if (g >= 2 && !(ok = wait(V_EMPTY + vb, (g >> 1) - 1)))
                    break;
                tc_fence_after();
#pragma unroll
                for (int e = 0; e < 2; e++) {
                    const int n = w.s.len - (2 * k + e) * kPage;
                    if (n < kPage) {  // codes behind the last token may be anything
#pragma unroll
                        for (int i = 0; i < 4; i++) {
                            auto keep = [&](uint32_t x, int at) {
                                return n >= at + 4 ? x : n <= at ? 0u : x & ((1u << (8 * (n - at))) - 1u);
                            };
                            v[e][i] = make_uint4(keep(v[e][i].x, 16 * i), keep(v[e][i].y, 16 * i + 4),
                                                 keep(v[e][i].z, 16 * i + 8), keep(v[e][i].w, 16 * i + 12));
                        }
                    }
                    // scale 2^x as two factors with the 2^120 of the conversion; NaN and 0 as they are
                    const int x = (sc[e] >> 23 & 255) - 127;
                    const bool odd = sc[e] == 0 || x == 128;
                    const int x1 = odd ? 120 : min(120 + x, 127);
                    const uint32_t f1 = pow2_bf16x2(x1);
                    const uint32_t f2 = odd ? (uint32_t)(sc[e] >> 16 & 0xffff) * 0x10001u : pow2_bf16x2(120 + x - x1);
                    const bool two = odd || 120 + x > 127;
#pragma unroll
                    for (int hf = 0; hf < 2; hf++) {
                        uint32_t pk[16];
#pragma unroll
                        for (int i = 0; i < 2; i++) {
                            const uint4 q = v[e][2 * hf + i];
                            const uint32_t ww[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                            for (int j = 0; j < 4; j++) {
                                pk[8 * i + 2 * j] = mul_bf16x2(code2_to_bf16(__byte_perm(ww[j], 0, 0x1404)), f1);
                                pk[8 * i + 2 * j + 1] = mul_bf16x2(code2_to_bf16(__byte_perm(ww[j], 0, 0x3424)), f1);
                            }
                        }
                        if (two)
#pragma unroll
                            for (int i = 0; i < 16; i++)
                                pk[i] = mul_bf16x2(pk[i], f2);
                        tmem_st16(tmem + ((uint32_t)(quarter * 32) << 16) + 384 + vb * 64 + e * 32 + hf * 16, pk);
                    }
                }
                if (k + 1 < k1) {
                    fetch(2 * k + 2, v[0], &sc[0]);
                    fetch(2 * k + 3, v[1], &sc[1]);
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(bar(V_FULL + vb));
            }
        }
    } else {
        // ---------------- S^T to P^T ----------------
        const int group = (warp - 2) >> 2, quarter = warp & 3;
        const int r = quarter * 32 + lane;  // key of the tile
        const uint32_t trow = tmem + ((uint32_t)(quarter * 32) << 16);
        int g0 = 0;  // tiles before this piece
        for (Walk w = start; ok && w.left > 0; w.next(c)) {
            const int qs = w.piece & 1, h = w.head(), q0 = w.q0(), cols = w.cols(), count = w.count();
            const float *rp = a.rab_pos + h * a.pos_hstride, *rt = a.rab_time + h * a.time_hstride;
            const QueryInfo &qi = info[qs];
            if (!(ok = wait(Q_FULL + qs, w.piece >> 1)))
                break;
            const int p_i = qi.pos[0];
            const int64_t t_i = qi.ts[0];
            float *plane = a.part_w ? a.part_w + ((int64_t)((q0 / kTile) * c.H + h) * c.B + w.b) * a.plan.lcap : nullptr;
            // this thread's key of tile k
            bool live = false;
            int pj = 0;
            int64_t tj = 0;
            float ks = 0.f;
            auto fetch = [&](int k) {
                const int j = k * kTile + r;
                const int page = j < w.s.len ? table_page(c.table, c, w.b, j / kPage) : -1;
                live = page >= 0;
                if (live) {
                    const int64_t at = (int64_t)page * kPage + j % kPage;
                    pj = c.positions[at];
                    tj = c.timestamps[at];
                    ks = c.k_scale[(int64_t)page * c.H + h];
                }
            };
            // the group's tiles of this piece: those with g % 2 = group
            const int first = (g0 & 1) == group ? 0 : 1;
            if (first < count)
                fetch(w.k + first);
            for (int t = first; t < count; t += 2) {
                const int g = g0 + t, k = w.k + t;
                const bool live_t = live;
                const int pj_t = pj;
                const int64_t tj_t = tj;
                const float ks_t = 0.5f * ks;
                const float bias = live ? 0.5f * (rp[pos_index(p_i, pj, a.pos_lo, a.pos_hi)] + rt[time_bucket(t_i, tj, a.nb)])
                                        : 0.f;
                if (t + 2 < count)
                    fetch(k + 2);
                if (!(ok = wait(S_FULL + group, g >> 1) && (g < 2 || wait(P_EMPTY + group, (g >> 1) - 1))))
                    break;
                tc_fence_after();
                const bool dead = __any_sync(0xffffffffu, !live_t);
                float wsum = 0.f;
                unsigned char *prow = sm + LY::P + group * 2 * kPanel + r * 128;
                for (int cc = 0; cc < cols; cc += 32) {
                    float sv[32];
                    tmem_ld32(trow + group * kTile + cc, sv);
                    tmem_wait_ld();
                    const float cs = qi.chunk_scale[cc >> 5];
                    if (qi.chunk_same[cc >> 5] && cs != -1.f) {
                        const float f = ks_t * cs;
#pragma unroll
                        for (int e = 0; e < 32; e++) {
                            const float hh = fmaf(sv[e], f, bias);
                            sv[e] = fmaf(hh, tanh_approx(hh), hh);
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < 32; e++) {
                            const float bi = live_t ? rp[pos_index(qi.pos[cc + e], pj_t, a.pos_lo, a.pos_hi)] +
                                                          rt[time_bucket(qi.ts[cc + e], tj_t, a.nb)]
                                                    : 0.f;
                            const float hh = fmaf(sv[e], ks_t * qi.scale[cc + e], 0.5f * bi);
                            sv[e] = fmaf(hh, tanh_approx(hh), hh);
                        }
                    }
                    if (plane) {
                        if (cc + 32 <= cols) {
#pragma unroll
                            for (int e = 0; e < 32; e++)
                                wsum += fabsf(sv[e]);
                        } else {
#pragma unroll
                            for (int e = 0; e < 32; e++)
                                wsum += cc + e < cols ? fabsf(sv[e]) : 0.f;
                        }
                    }
                    uint32_t pk[16];
#pragma unroll
                    for (int e = 0; e < 16; e++)
                        pk[e] = pack_bf16(sv[2 * e], sv[2 * e + 1]);
                    if (dead)
#pragma unroll
                        for (int e = 0; e < 16; e++)
                            pk[e] = live_t ? pk[e] : 0u;
                    unsigned char *dst = prow + (cc >> 6) * kPanel;
#pragma unroll
                    for (int e = 0; e < 4; e++)
                        *reinterpret_cast<uint4 *>(dst + ((((cc >> 3) & 4) + e) ^ (r & 7)) * 16) =
                            make_uint4(pk[4 * e], pk[4 * e + 1], pk[4 * e + 2], pk[4 * e + 3]);
                }
                fence_proxy_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(bar(P_FULL + group));
                if (plane && k * kTile + r < a.plan.lcap)
                    plane[k * kTile + r] = live_t ? wsum : 0.f;
            }
            g0 += count;
            if (!(ok = ok && wait(O_FULL, w.piece)))
                break;
            tc_fence_after();
            // O^T: lane = dim, column = query; this group's half of the columns
            const bool whole = w.k == 0 && count == w.z.kt;
            const int slot = w.k > 0 ? 0 : 1;
            const int dim = r;
            if (dim < D) {
                for (int cc = group * 64; cc < min(cols, group * 64 + 64); cc += 32) {
                    float ov[32];
                    tmem_ld32(trow + 256 + cc, ov);
                    tmem_wait_ld();
                    const int m = min(32, cols - cc);
                    const int64_t row = w.s.s0 + q0 + cc;
                    if (whole) {
                        const int64_t at = (row * c.H + h) * D + dim, step = (int64_t)c.H * D;
                        __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(a.out) + at;
                        const __nv_bfloat16 *add =
                            a.addend ? static_cast<const __nv_bfloat16 *>(a.addend) + at : nullptr;
#pragma unroll
                        for (int e = 0; e < 32; e++)
                            if (e < m) {
                                const float y = ov[e] * a.inv_n + (add ? __bfloat162float(add[e * step]) : 0.f);
                                out[e * step] = __float2bfloat16_rn(y);
                            }
                    } else {
                        float *part = a.part_o + ((int64_t)(2 * blockIdx.x + slot) * kTile + cc) * D + dim;
#pragma unroll
                        for (int e = 0; e < 32; e++)
                            if (e < m)
                                part[e * D] = ov[e];
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(bar(O_FREE));
                mbar_arrive(bar(Q_EMPTY + qs));
            }
            if (!whole && warp == 2 && lane == 0) {
                CacheAttnPiece p;
                p.row = w.s.s0 + q0;
                p.head = h;
                p.cols = cols;
                p.last = w.k + count == w.z.kt;
                pieces[slot] = p;
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1)
        tmem_dealloc(tmem, 512);
}

// The rest of the output and the weights.  Blocks [0, 4 ctas): a quarter of the columns
// of the unit that CTA x / 4 left unfinished.  Then one block per sequence for rows
// whose cache is empty, then the weights.
template <int D>
__global__ void __launch_bounds__(256)
cache_tc_join_kernel(const CacheAttnArgs a, int ctas, int w_blocks)
{
    const CacheCall &c = a.c;
    __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(a.out);
    const __nv_bfloat16 *add = static_cast<const __nv_bfloat16 *>(a.addend);
    int x = blockIdx.x;
    if (x < 4 * ctas) {
        const int cta = x >> 2, c0 = (x & 3) * 32;
        const CacheAttnPiece p = a.pieces[2 * cta + 1];
        const int n = min(p.cols - c0, 32) * D;
        if (n <= 0)
            return;
        int end = cta + 1;  // the CTA that ends the unit
        while (end < ctas && (a.pieces[2 * end].cols == 0 || !a.pieces[2 * end].last))
            end++;
        for (int i = threadIdx.x; i < n; i += 256) {
            const int64_t e = (int64_t)c0 * D + i;
            float sum = a.part_o[(int64_t)(2 * cta + 1) * kTile * D + e];
            for (int m = cta + 1; m <= end && m < ctas; m++)
                if (a.pieces[2 * m].cols)
                    sum += a.part_o[(int64_t)2 * m * kTile * D + e];
            const int64_t at = ((p.row + c0 + i / D) * c.H + p.head) * D + i % D;
            out[at] = __float2bfloat16_rn(sum * a.inv_n + (add ? __bfloat162float(add[at]) : 0.f));
        }
        return;
    }
    x -= 4 * ctas;
    if (x < c.B) {
        const CacheSeq s = cache_seq(c, x);
        if (s.bits && threadIdx.x == 0)
            atomicOr(&c.hdr->flag, s.bits);
        if (s.bits || s.len > 0)
            return;
        const int64_t width = (int64_t)c.H * D;
        for (int64_t i = s.s0 * width + threadIdx.x; i < (s.s0 + s.n) * width; i += 256)
            out[i] = add ? add[i] : __float2bfloat16_rn(0.f);
        return;
    }
    x -= c.B;
    const int b = x / w_blocks, j = (x % w_blocks) * 256 + threadIdx.x;
    cache_join_weight(a, b, j);
}

template <int D>
cudaError_t tc_launch(const CacheAttnArgs &a, cudaStream_t stream)
{
    const CacheCall &c = a.c;
    if (a.plan.ctas > 0) {
        CUtensorMap tk;
        cudaError_t e = make_tensor_map_2d(&tk, c.k_codes, CU_TENSOR_MAP_DATA_TYPE_UINT8,
                                           (int64_t)c.num_pages * c.H * kPage, D, D, D, kPage,
                                           D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B);
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(cache_attn_tc_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     Layout<D>::BYTES);
        if (e != cudaSuccess)
            return e;
        cache_attn_tc_kernel<D><<<a.plan.ctas, kThreads, Layout<D>::BYTES, stream>>>(a, tk);
        e = cudaGetLastError();
        if (e != cudaSuccess)
            return e;
    }
    const int w_blocks = a.weights_out ? (c.max_cache_len + 255) / 256 : 0;
    const int64_t grid = 4LL * a.plan.ctas + c.B + (int64_t)w_blocks * c.B;
    cache_tc_join_kernel<D><<<(unsigned)grid, 256, 0, stream>>>(a, a.plan.ctas, w_blocks);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_cache_attn_tc(const CacheAttnArgs &a, cudaStream_t stream)
{
    return a.c.d == 64 ? tc_launch<64>(a, stream) : tc_launch<128>(a, stream);
}

}  // namespace hstu
