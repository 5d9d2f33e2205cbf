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
// Warp roles (512 threads): warp 0 loads the codes (TMA); warp 1 owns TMEM and issues
// the MMAs (2 and 3 idle); warps 4-7 and 8-11 take the even and the odd tiles' S^T and
// write P^T; warps 12-15 split queries and convert values.
// TMEM columns: S^T [0, 128) and [128, 256), O^T [256, 384), V^T [384, 448), [448, 512).
//
// Work: all (sequence, head, query tile) units' key tiles in one line, cut into equal
// runs, one per CTA.  A unit inside one run is written to `out`; a cut unit's pieces
// go to the CTA's two slots (the unit it starts in the middle of, the unit it leaves
// unfinished), and the join adds them in order.
#include <cudaTypedefs.h>

#include <algorithm>
#include <climits>

#include "cache.cuh"
#include "tc_common.cuh"

namespace hstu {

namespace {

constexpr int kTile = 128;    // keys of a tile, query columns of a unit
constexpr int kThreads = 512;
constexpr int kKStages = 3, kVStages = 2;  // tiles of codes in flight
constexpr int kCutTiles = 8;  // what a cut unit costs (its pieces' traffic and the join), in tiles
constexpr int kPanel = 16384; // 64 query columns of P^T: 128 keys x 128 bytes

enum Bars { K_FULL = 0, K_EMPTY = K_FULL + kKStages, C_FULL = K_EMPTY + kKStages, C_EMPTY = C_FULL + kVStages,
            S_FULL = C_EMPTY + kVStages, P_FULL = S_FULL + 2, P_EMPTY = P_FULL + 2, V_FULL = P_EMPTY + 2,
            V_EMPTY = V_FULL + 2, Q_FULL = V_EMPTY + 2, Q_EMPTY = Q_FULL + 2, O_FULL = Q_EMPTY + 2,
            O_FREE = O_FULL + 1, NBARS = O_FREE + 1 };

// what the epilogue needs to know of a unit's queries
struct QueryInfo {
    float chunk_scale[4];  // one scale of the 32 columns, or -1: each its own
    int chunk_same[4];     // every column has row 0's position and stamp
    int pos_lo[4], pos_hi[4];  // a chunk's least and largest position and stamp
    int64_t ts_lo[4], ts_hi[4];
    float scale[kTile];
    int pos[kTile];
    int64_t ts[kTile];
};

template <int D>
struct Layout {
    static constexpr int KT = kTile * D;  // a key tile, one part of the queries
    static constexpr int Q = 0;           // two buffers of two parts
    static constexpr int K = Q + 4 * KT;
    static constexpr int V = K + kKStages * KT;  // value codes [2 pages][D][64]
    static constexpr int P = V + kVStages * KT;
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
    int lo = INT_MAX, hi = 0;  // least and most key tiles of a sequence
    for (int b = b0; b < b1; b++) {
        const Sizes z = sizes(cache_seq(c, b));
        mine += z.tiles(c.H);
        if (z.qt * z.kt > 0) {
            lo = min(lo, z.kt);
            hi = max(hi, z.kt);
        }
    }
    lo = __reduce_min_sync(0xffffffffu, lo);
    hi = __reduce_max_sync(0xffffffffu, hi);
    int64_t inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o)
            inc += y;
    }
    if (lane == 31) {
        sums[warp] = inc;
        sums[kW + warp] = lo;
        sums[2 * kW + warp] = hi;
    }
    __syncthreads();
    int64_t before = 0, total = 0;
    for (int w = 0; w < kW; w++) {
        if (w < warp)
            before += sums[w];
        total += sums[w];
        lo = min(lo, (int)sums[kW + w]);
        hi = max(hi, (int)sums[2 * kW + w]);
    }
    // equal units: whole ones, unless that makes the longest run much longer than the mean
    int64_t grain = 1;
    if (lo == hi && (total / hi + ctas - 1) / ctas * hi <= total / ctas + kCutTiles)
        grain = hi;
    const int64_t start = total / grain * cta / ctas * grain, end = total / grain * (cta + 1) / ctas * grain;
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

// Codes 0, 2 and 1, 3 of a word as bf16, times 2^-120: sign, exponent and fraction at
// bf16's places (E4M3's subnormals are bf16's).
__device__ __forceinline__ uint32_t even_codes(uint32_t w)
{
    return ((w << 8) & 0x80008000u) | ((w << 4) & 0x07f007f0u);
}

__device__ __forceinline__ uint32_t odd_codes(uint32_t w) { return (w & 0x80008000u) | ((w >> 4) & 0x07f007f0u); }

// Row of P^T of key r: the order in which the words above hold four keys.
__device__ __forceinline__ int key_row(int r) { return (r & ~3) | ((r & 1) << 1) | ((r >> 1) & 1); }

__device__ __forceinline__ uint64_t pack2(float x, float y)
{
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(x), "f"(y));
    return d;
}

__device__ __forceinline__ float2 unpack2(uint64_t d)
{
    float2 f;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(d));
    return f;
}

__device__ __forceinline__ uint64_t fma2(uint64_t x, uint64_t y, uint64_t z)
{
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(x), "l"(y), "l"(z));
    return d;
}

// SiLU(2 h) of two values
__device__ __forceinline__ float2 silu2(uint64_t h)
{
    const float2 f = unpack2(h);
    return unpack2(fma2(h, pack2(tanh_approx(f.x), tanh_approx(f.y)), h));
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

// 32 lanes x 8 consecutive 32-bit columns
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, float *v)
{
    uint32_t *r = reinterpret_cast<uint32_t *>(v);
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
}

// P^T of eight scores (zeros for a dead key) into 16 bytes of a row of the panel.
__device__ __forceinline__ void put_p8(const float *x, bool dead, bool live, unsigned char *dst)
{
    uint32_t pk[4];
#pragma unroll
    for (int e = 0; e < 4; e++) {
        pk[e] = pack_bf16(x[2 * e], x[2 * e + 1]);
        if (dead)
            pk[e] = live ? pk[e] : 0u;
    }
    *reinterpret_cast<uint4 *>(dst) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
}

// A chunk of 32 queries whose biases or scales differ: this key's P^T, and the sum of
// its magnitudes over the first n.  Where the whole warp's pairs share an index of a
// table, it is read once.  Eight queries at a time: the common loop keeps its registers.
__device__ __forceinline__ float chunk_general(uint32_t taddr, int cc, int n, const CacheAttnArgs &a, const float *rp,
                                               const float *rt, const QueryInfo &qi, bool dead, bool live, int pj,
                                               int64_t tj, float half_scale, unsigned char *dst, int row_p)
{
    const int ch = cc >> 5;
    const int i0 = pos_index(qi.pos_lo[ch], pj, a.pos_lo, a.pos_hi), i1 = pos_index(qi.pos_hi[ch], pj, a.pos_lo, a.pos_hi);
    const int u0 = time_bucket(qi.ts_lo[ch], tj, a.nb), u1 = time_bucket(qi.ts_hi[ch], tj, a.nb);
    const bool one_p = __all_sync(0xffffffffu, !live || i0 == i1), one_t = __all_sync(0xffffffffu, !live || u0 == u1);
    const float bp = live ? rp[i0] : 0.f, bt = live ? rt[u0] : 0.f;
    float w = 0.f;
#pragma unroll 1
    for (int e8 = 0; e8 < min(n, 32); e8 += 8) {
        float x[8], b[8];
        tmem_ld8(taddr + e8, x);
#pragma unroll
        for (int e = 0; e < 8; e++)
            b[e] = bp;
        if (!one_p && live)
#pragma unroll
            for (int e = 0; e < 8; e++)
                b[e] = rp[pos_index(qi.pos[cc + e8 + e], pj, a.pos_lo, a.pos_hi)];
        if (one_t) {
#pragma unroll
            for (int e = 0; e < 8; e++)
                b[e] += bt;
        } else if (live) {
#pragma unroll
            for (int e = 0; e < 8; e++)
                b[e] += rt[time_bucket(qi.ts[cc + e8 + e], tj, a.nb)];
        }
        __syncwarp();
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 8; e++) {
            const float hh = fmaf(x[e], half_scale * qi.scale[cc + e8 + e], 0.5f * b[e]);
            x[e] = fmaf(hh, tanh_approx(hh), hh);
            w += e8 + e < n ? fabsf(x[e]) : 0.f;
        }
        put_p8(x, dead, live, dst + ((((cc + e8) >> 3 & 7) ^ (row_p & 7)) * 16));
    }
    return w;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
cache_attn_tc_kernel(const __grid_constant__ CacheAttnArgs a, const __grid_constant__ CUtensorMap tk,
                     const __grid_constant__ CUtensorMap tv)
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
            else if (i == V_FULL || i == V_FULL + 1 || (i >= C_EMPTY && i < C_EMPTY + kVStages))
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
        tma_prefetch(&tv);
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
        // ---------------- codes ----------------
        int g = 0;
        for (Walk w = start; ok && w.left > 0; w.next(c)) {
            const int h = w.head(), pages = (w.s.len + kPage - 1) / kPage, count = w.count();
            int held = -1;  // lane: a page of this and the next 15 tiles
            for (int t = 0; t < count; t++, g++) {
                const int k = w.k + t, kst = g % kKStages, vst = g % kVStages;
                if (t % 16 == 0) {
                    held = -1;
                    if (2 * k + lane < pages) {
                        held = table_page(c.table, c, w.b, 2 * k + lane);
                        if (held < 0)
                            atomicOr(&hdr->flag, FLAG_CACHE_PAGE);
                    }
                }
                const int page[2] = {__shfl_sync(0xffffffffu, held, 2 * (t % 16)),
                                     __shfl_sync(0xffffffffu, held, 2 * (t % 16) + 1)};
                const uint32_t bytes = ((page[0] >= 0) + (page[1] >= 0)) * kPage * D;
                ok = __all_sync(0xffffffffu, g < kKStages || wait(K_EMPTY + kst, g / kKStages - 1));
                if (!ok)
                    break;
                if (lane == 0) {
                    mbar_expect_tx(bar(K_FULL + kst), bytes);
#pragma unroll
                    for (int e = 0; e < 2; e++)
                        if (page[e] >= 0)
                            tma_load_2d(base + LY::K + kst * LY::KT + e * kPage * D, &tk, 0,
                                        (page[e] * c.H + h) * kPage, bar(K_FULL + kst));
                }
                ok = __all_sync(0xffffffffu, g < kVStages || wait(C_EMPTY + vst, g / kVStages - 1));
                if (!ok)
                    break;
                if (lane == 0) {
                    mbar_expect_tx(bar(C_FULL + vst), bytes);
#pragma unroll
                    for (int e = 0; e < 2; e++)
                        if (page[e] >= 0)
                            tma_load_2d(base + LY::V + vst * LY::KT + e * kPage * D, &tv, 0,
                                        (page[e] * c.H + h) * D, bar(C_FULL + vst));
                }
                __syncwarp();
            }
        }
    } else if (warp == 1) {
        // ---------------- MMAs ----------------
        if (lane == 0) {
            int issued = 0, done = 0, t = 0, piece = 0;
            Walk w = start;
            int count = w.count(), n = w.cols() > 64 ? 128 : 64;
            uint32_t ring = 0;  // of the two tiles in flight: first, last, 128 columns; tile g in bits 4 (g & 1)
            while (ok) {
                if (w.left > 0 && issued < done + 2) {
                    const int st = issued % kKStages, sb = issued & 1, qs = w.piece & 1;
                    const bool first = t == 0, last = t + 1 == count;
                    ok = (!first || wait(Q_FULL + qs, w.piece >> 1)) && wait(K_FULL + st, issued / kKStages);
                    if (!ok)
                        break;
                    tc_fence_after();
                    const uint32_t id = idesc_e4m3(128, 0, 0, 0) | ((uint32_t)(n >> 3) << 17);
                    const uint64_t kd = code_desc<D>(base + LY::K + st * LY::KT);
                    const uint64_t qd = code_desc<D>(base + LY::Q + 2 * qs * LY::KT);
#pragma unroll
                    for (int i = 0; i < 2 * (D / 32); i++)  // 32 bytes of a row a step: 2 in the address field
                        umma_e4m3(tmem + sb * kTile, kd + 2 * (i % (D / 32)),
                                  qd + i / (D / 32) * (LY::KT >> 4) + 2 * (i % (D / 32)), id, i > 0);
                    umma_commit(bar(K_EMPTY + st));
                    umma_commit(bar(S_FULL + sb));
                    if (last)
                        umma_commit(bar(Q_EMPTY + qs));
                    ring = (ring & ~(15u << (4 * sb))) | ((first | last << 1 | (n == 128) << 2) << (4 * sb));
                    issued++;
                    t++;
                    if (last) {
                        w.next(c);
                        t = 0;
                        count = w.count();
                        n = w.cols() > 64 ? 128 : 64;
                    }
                    continue;
                }
                if (done == issued)
                    break;
                const int sb = done & 1;
                const uint32_t r = ring >> (4 * sb);
                ok = wait(P_FULL + sb, done >> 1) && wait(V_FULL + sb, done >> 1) &&
                     (!(r & 1) || piece == 0 || wait(O_FREE, piece - 1));
                if (!ok)
                    break;
                tc_fence_after();
                const uint32_t id = idesc_bf16(128, 0, 0, 1) | ((uint32_t)((r & 4 ? 128 : 64) >> 3) << 17);
                const uint64_t pd = smem_desc_sw128(base + LY::P + sb * 2 * kPanel, kPanel, 1024);
#pragma unroll
                for (int ks = 0; ks < kTile / 16; ks++)  // 16 rows of P^T a step
                    umma_bf16_ts(tmem + 256, tmem + 384 + sb * 64 + ks * 8, pd + ks * (2048 >> 4), id,
                                 !(r & 1) || ks > 0);
                umma_commit(bar(V_EMPTY + sb));
                umma_commit(bar(P_EMPTY + sb));
                if (r & 2) {
                    umma_commit(bar(O_FULL));
                    piece++;
                }
                done++;
            }
        }
    } else if (warp >= 12) {
        // ---------------- queries and values ----------------
        const int quarter = warp & 3, dim = quarter * 32 + lane;
        const int row = threadIdx.x - 384;  // of the queries
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
                auto load8 = [&](int e) {
                    return have ? *reinterpret_cast<const uint4 *>(qp + 8 * e) : make_uint4(0u, 0u, 0u, 0u);
                };
#pragma unroll
                for (int e = 0; e < D / 8; e++) {
                    const uint4 x = load8(e);
                    const uint32_t ww[4] = {x.x, x.y, x.z, x.w};
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
                // positions and stamps of the chunk: their range
                int plo = pi, phi = pi;
                int64_t tlo = ti, thi = ti;
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) {
                    plo = min(plo, __shfl_xor_sync(0xffffffffu, plo, o));
                    phi = max(phi, __shfl_xor_sync(0xffffffffu, phi, o));
                    tlo = min(tlo, __shfl_xor_sync(0xffffffffu, tlo, o));
                    thi = max(thi, __shfl_xor_sync(0xffffffffu, thi, o));
                }
                qi.scale[row] = scale;
                qi.pos[row] = pi;
                qi.ts[row] = ti;
                if (lane == 0) {
                    qi.chunk_scale[row >> 5] = one ? scale : -1.f;
                    qi.chunk_same[row >> 5] = all_same;
                    qi.pos_lo[row >> 5] = plo;
                    qi.pos_hi[row >> 5] = phi;
                    qi.ts_lo[row >> 5] = tlo;
                    qi.ts_hi[row >> 5] = thi;
                }
                unsigned char *q1 = sm + LY::Q + 2 * qs * LY::KT + row * D, *q2 = q1 + LY::KT;
#pragma unroll 2
                for (int e = 0; e < D / 16; e++) {  // read again: held, the row would not fit the registers
                    const uint4 x0 = load8(2 * e), x1 = load8(2 * e + 1);
                    const uint32_t ww[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
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
            const int count = w.count();
            // scale bits of page 2 k + e, 0 for none; its page id one tile earlier
            auto page_at = [&](int p) { return p * kPage < w.s.len ? table_page(c.table, c, w.b, p) : -1; };
            auto scale_at = [&](int page) {
                return page >= 0 ? __float_as_int(c.v_scale[(int64_t)page * c.H + h]) : 0;
            };
            int ids[2], sc[2];
#pragma unroll
            for (int e = 0; e < 2; e++) {
                sc[e] = scale_at(page_at(2 * w.k + e));
                ids[e] = count > 1 ? page_at(2 * w.k + 2 + e) : -1;
            }
            for (int t = 0; t < count; t++, g++) {
                const int k = w.k + t, vb = g & 1, vst = g % kVStages;
                int next[2];
#pragma unroll
                for (int e = 0; e < 2; e++) {
                    next[e] = t + 1 < count ? scale_at(ids[e]) : 0;
                    ids[e] = t + 2 < count ? page_at(2 * k + 4 + e) : -1;
                }
                if (!(ok = wait(C_FULL + vst, g / kVStages) && (g < 2 || wait(V_EMPTY + vb, (g >> 1) - 1))))
                    break;
                tc_fence_after();
#pragma unroll
                for (int e = 0; e < 2; e++) {
                    uint4 v[4];
                    const unsigned char *vrow = sm + LY::V + vst * LY::KT + e * kPage * D + dim * kPage;
#pragma unroll
                    for (int i = 0; i < 4; i++)
                        v[i] = *reinterpret_cast<const uint4 *>(vrow + (i ^ ((dim >> 1) & 3)) * 16);
                    // codes behind the last token, or of a page that was not loaded, may be anything
                    const int n = w.s.len - (2 * k + e) * kPage;
                    if (n < kPage || sc[e] == 0) {
#pragma unroll
                        for (int i = 0; i < 4; i++) {
                            auto keep = [&](uint32_t x, int at) {
                                return sc[e] == 0 || n <= at ? 0u : n >= at + 4 ? x : x & ((1u << (8 * (n - at))) - 1u);
                            };
                            v[i] = make_uint4(keep(v[i].x, 16 * i), keep(v[i].y, 16 * i + 4),
                                              keep(v[i].z, 16 * i + 8), keep(v[i].w, 16 * i + 12));
                        }
                    }
                    // times the scale 2^x and 2^120, in two factors where bf16 has no 2^(120 + x); a NaN scale as it is
                    const int x = (sc[e] >> 23 & 255) - 127;
                    const bool nan = x == 128;
                    const int x1 = nan ? 120 : min(120 + max(x, -126), 127);
                    const uint32_t f1 = pow2_bf16x2(x1);
                    const uint32_t f2 = nan ? 0x7fff7fffu : pow2_bf16x2(max(120 + x - x1, 0));
#pragma unroll
                    for (int hf = 0; hf < 2; hf++) {
                        uint32_t pk[16];
#pragma unroll
                        for (int i = 0; i < 2; i++) {
                            const uint4 q = v[2 * hf + i];
                            const uint32_t ww[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                            for (int j = 0; j < 4; j++) {
                                pk[8 * i + 2 * j] = mul_bf16x2(even_codes(ww[j]), f1);
                                pk[8 * i + 2 * j + 1] = mul_bf16x2(odd_codes(ww[j]), f1);
                            }
                        }
                        if (nan || 120 + x > 127)
#pragma unroll
                            for (int i = 0; i < 16; i++)
                                pk[i] = mul_bf16x2(pk[i], f2);
                        tmem_st16(tmem + ((uint32_t)(quarter * 32) << 16) + 384 + vb * 64 + e * 32 + hf * 16, pk);
                    }
                    sc[e] = next[e];
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(bar(C_EMPTY + vst));
                    mbar_arrive(bar(V_FULL + vb));
                }
            }
        }
    } else if (warp >= 4) {
        // ---------------- S^T to P^T ----------------
        const int group = (warp - 4) >> 2, quarter = warp & 3;
        const int r = quarter * 32 + lane, row_p = key_row(r);  // key of the tile, its row of P^T
        const uint32_t trow = tmem + ((uint32_t)(quarter * 32) << 16);
        int g0 = 0;  // tiles before this piece
        for (Walk w = start; ok && w.left > 0; w.next(c)) {
            const int qs = w.piece & 1, h = w.head(), q0 = w.q0(), cols = w.cols(), count = w.count();
            const float *rp = a.rab_pos + h * a.pos_hstride, *rt = a.rab_time + h * a.time_hstride;
            const QueryInfo &qi = info[qs];
            float *plane = a.part_w ? a.part_w + ((int64_t)((q0 / kTile) * c.H + h) * c.B + w.b) * a.plan.lcap : nullptr;
            // The group's tiles of this piece are those with g % 2 = group.  What a tile needs
            // of this thread's key is fetched ahead, one step of the chain a tile: the page, the
            // token's position, stamp and scale, the bias of column 0.
            struct Key {
                bool live;
                int pos;
                int64_t ts;
                float scale;
            };
            auto page_at = [&](int t) {
                const int j = (w.k + t) * kTile + r;
                return t < count && j < w.s.len ? table_page(c.table, c, w.b, j / kPage) : -1;
            };
            auto key_at = [&](int page) {
                Key y{page >= 0, 0, 0, 0.f};
                if (y.live) {
                    const int64_t at = (int64_t)page * kPage + r % kPage;
                    y.pos = c.positions[at];
                    y.ts = c.timestamps[at];
                    y.scale = c.k_scale[(int64_t)page * c.H + h];
                }
                return y;
            };
            const int first = (g0 & 1) == group ? 0 : 1;
            Key key = key_at(page_at(first)), ahead = key_at(page_at(first + 2));
            int page = page_at(first + 4);
            if (!(ok = wait(Q_FULL + qs, w.piece >> 1)))
                break;
            const int p_i = qi.pos[0];
            const int64_t t_i = qi.ts[0];
            float bp = 0.f, bt = 0.f;
            if (key.live) {
                bp = rp[pos_index(p_i, key.pos, a.pos_lo, a.pos_hi)];
                bt = rt[time_bucket(t_i, key.ts, a.nb)];
            }
            for (int t = first; t < count; t += 2) {
                const int g = g0 + t, k = w.k + t;
                const Key me = key;
                const float bias = 0.5f * (bp + bt), half_scale = 0.5f * me.scale;
                key = ahead;
                bp = bt = 0.f;
                if (key.live) {
                    bp = rp[pos_index(p_i, key.pos, a.pos_lo, a.pos_hi)];
                    bt = rt[time_bucket(t_i, key.ts, a.nb)];
                }
                ahead = key_at(page);
                page = page_at(t + 6);
                if (!(ok = wait(S_FULL + group, g >> 1) && (g < 2 || wait(P_EMPTY + group, (g >> 1) - 1))))
                    break;
                tc_fence_after();
                const bool dead = __any_sync(0xffffffffu, !me.live);
                float wsum = 0.f;
                unsigned char *prow = sm + LY::P + group * 2 * kPanel + row_p * 128;
#pragma unroll 1
                for (int cc = 0; cc < cols; cc += 32) {
                    unsigned char *dst = prow + (cc >> 6) * kPanel;
                    const uint32_t taddr = trow + group * kTile + cc;
                    const float cs = qi.chunk_scale[cc >> 5];
                    if (!qi.chunk_same[cc >> 5] || cs == -1.f) {
                        wsum += chunk_general(taddr, cc, cols - cc, a, rp, rt, qi, dead, me.live, me.pos, me.ts,
                                              half_scale, dst, row_p);
                        continue;
                    }
                    float x[32];
                    tmem_ld32(taddr, x);
                    tmem_wait_ld();
                    const uint64_t b2 = pack2(bias, bias), f2 = pack2(half_scale * cs, half_scale * cs);
#pragma unroll
                    for (int e = 0; e < 32; e += 2) {
                        const float2 y = silu2(fma2(pack2(x[e], x[e + 1]), f2, b2));
                        x[e] = y.x, x[e + 1] = y.y;
                    }
#pragma unroll
                    for (int e = 0; e < 4; e++)
                        put_p8(x + 8 * e, dead, me.live, dst + ((((cc >> 3) & 4) + e) ^ (row_p & 7)) * 16);
                    if (plane) {
                        const int n = cols - cc;
                        float w0 = 0.f, w1 = 0.f;
                        if (n >= 32) {
#pragma unroll
                            for (int e = 0; e < 32; e += 2)
                                w0 += fabsf(x[e]), w1 += fabsf(x[e + 1]);
                        } else {
#pragma unroll
                            for (int e = 0; e < 32; e++)
                                w0 += e < n ? fabsf(x[e]) : 0.f;
                        }
                        wsum += w0 + w1;
                    }
                }
                fence_proxy_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(bar(P_FULL + group));
                if (plane && k * kTile + r < a.plan.lcap)
                    plane[k * kTile + r] = me.live ? wsum : 0.f;
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
#pragma unroll 1
                for (int cc = group * 64; cc < min(cols, group * 64 + 64); cc += 16) {
                    float ov[16];
                    tmem_ld16(trow + 256 + cc, ov);
                    tmem_wait_ld();
                    const int m = min(16, cols - cc);
                    if (whole) {
                        const int64_t at = ((w.s.s0 + q0 + cc) * c.H + h) * D + dim;
                        const int step = c.H * D;
                        __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(a.out) + at;
#pragma unroll
                        for (int e = 0; e < 16; e++)
                            ov[e] *= a.inv_n;
                        if (a.addend) {  // all loads before the stores: it may be `out`
                            const __nv_bfloat16 *add = static_cast<const __nv_bfloat16 *>(a.addend) + at;
                            __nv_bfloat16 y[16];
#pragma unroll
                            for (int e = 0; e < 16; e++)
                                y[e] = add[(int64_t)min(e, m - 1) * step];
#pragma unroll
                            for (int e = 0; e < 16; e++)
                                ov[e] += __bfloat162float(y[e]);
                        }
#pragma unroll
                        for (int e = 0; e < 16; e++)
                            if (e < m)
                                out[(int64_t)e * step] = __float2bfloat16_rn(ov[e]);
                    } else {
                        float *part = a.part_o + ((int64_t)(2 * blockIdx.x + slot) * kTile + cc) * D + dim;
#pragma unroll
                        for (int e = 0; e < 16; e++)
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
            if (!whole && warp == 4 && lane == 0) {
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

// The rest of the output and the weights.  Blocks [0, 16 ctas): eight columns of the
// unit that CTA x / 16 left unfinished.  Then one block per sequence for rows whose
// cache is empty, then the weights.
template <int D>
__global__ void __launch_bounds__(256)
cache_tc_join_kernel(const CacheAttnArgs a, int ctas, int w_blocks)
{
    const CacheCall &c = a.c;
    __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(a.out);
    const __nv_bfloat16 *add = static_cast<const __nv_bfloat16 *>(a.addend);
    int x = blockIdx.x;
    if (x < 16 * ctas) {
        const int cta = x >> 4, col = (x & 15) * 8 + threadIdx.x / (D / 4), d = threadIdx.x % (D / 4) * 4;
        const CacheAttnPiece p = a.pieces[2 * cta + 1];
        if (threadIdx.x >= 2 * D || col >= p.cols)
            return;
        const int64_t e = (int64_t)col * D + d;
        float4 sum = *reinterpret_cast<const float4 *>(a.part_o + (int64_t)(2 * cta + 1) * kTile * D + e);
        for (int m = cta + 1; m < ctas; m++) {
            const CacheAttnPiece q = a.pieces[2 * m];
            if (q.cols == 0)  // a run without tiles
                continue;
            const float4 y = *reinterpret_cast<const float4 *>(a.part_o + (int64_t)2 * m * kTile * D + e);
            sum.x += y.x, sum.y += y.y, sum.z += y.z, sum.w += y.w;
            if (q.last)
                break;
        }
        const int64_t at = ((p.row + col) * c.H + p.head) * D + d;
        float y[4] = {sum.x * a.inv_n, sum.y * a.inv_n, sum.z * a.inv_n, sum.w * a.inv_n};
        if (add)
            for (int i = 0; i < 4; i++)
                y[i] += __bfloat162float(add[at + i]);
        *reinterpret_cast<uint2 *>(out + at) = make_uint2(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]));
        return;
    }
    x -= 16 * ctas;
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
    cache_join_weight(a, x / w_blocks, (x % w_blocks) * 256 + threadIdx.x);
}

template <int D>
cudaError_t tc_launch(const CacheAttnArgs &a, cudaStream_t stream)
{
    const CacheCall &c = a.c;
    if (a.plan.ctas > 0) {
        CUtensorMap tk, tv;
        cudaError_t e = make_tensor_map_2d(&tk, c.k_codes, CU_TENSOR_MAP_DATA_TYPE_UINT8,
                                           (int64_t)c.num_pages * c.H * kPage, D, D, D, kPage,
                                           D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B);
        if (e == cudaSuccess)
            e = make_tensor_map_2d(&tv, c.v_codes, CU_TENSOR_MAP_DATA_TYPE_UINT8, (int64_t)c.num_pages * c.H * D,
                                   kPage, kPage, kPage, D, CU_TENSOR_MAP_SWIZZLE_64B);
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(cache_attn_tc_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     Layout<D>::BYTES);
        if (e != cudaSuccess)
            return e;
        cache_attn_tc_kernel<D><<<a.plan.ctas, kThreads, Layout<D>::BYTES, stream>>>(a, tk, tv);
        e = cudaGetLastError();
        if (e != cudaSuccess)
            return e;
    }
    const int w_blocks = a.weights_out ? (c.max_cache_len + 255) / 256 : 0;
    const int64_t grid = 16LL * a.plan.ctas + c.B + (int64_t)w_blocks * c.B;
    cache_tc_join_kernel<D><<<(unsigned)grid, 256, 0, stream>>>(a, a.plan.ctas, w_blocks);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_cache_attn_tc(const CacheAttnArgs &a, cudaStream_t stream)
{
    return a.c.d == 64 ? tc_launch<64>(a, stream) : tc_launch<128>(a, stream);
}

}  // namespace hstu
