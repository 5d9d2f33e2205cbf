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
// is held to 2^-17.8 of the largest magnitude under its scale.  A scale is shared by the
// 16 rows of a chunk if no row's largest is 2^3 or more below theirs, else each row has
// its own.  E4M3 runs at twice the bf16 rate, so both parts cost what one bf16 product
// would, and no key is ever converted.
// Values become bf16 (exactly, with their page's scale) in registers on the way from
// memory to TMEM; P is rounded to bf16 once.
//
// Per 128 x 128 tile at d = 128 the tensor pipe, MUFU (one tanh per pair) and shared
// memory need 1024 cycles each; V^T as a TMEM operand is what keeps the last there.  The
// kernel takes ~2,700 (10,784 tiles of 109 columns on average, 256-512 candidates over
// 8k-16k tokens: 196,000 cycles an SM): it is bound by its issue slots, 68 % busy with
// ~7,300 warp instructions a tile, half of them the math, and by the code that seven roles
// fetch (waits whose loops were inlined cost a fifth).  72 registers a thread are all that
// 896 threads leave, and some spill (268 bytes of stores at d = 128, 144 at d = 64).  So what
// a tile needs besides is spread over many warps:
// Warp roles (896 threads): 0 loads the codes (TMA); 1 issues S^T and owns TMEM; 2 issues
// O^T (3 idle); 4-19, four groups, take 64 columns of a tile in turn from S^T to P^T,
// each with a buffer of S^T and one of P^T; 20-27, two groups, take every other tile's
// keys (bias, scale) and values (conversion), and together split the queries.
// (16 users x 512 candidates over 2048 tokens, 2 heads: 37 us; one conversion group 43,
// the keys' data fetched by the epilogue warps 45, two epilogue groups of 128 columns 48.)
// TMEM columns: S^T 4 x 64, O^T [256, 384), V^T [384, 448), [448, 512).
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
constexpr int kThreads = 896;
constexpr int kKStages = 3, kVStages = 2;  // tiles of codes in flight
// What a cut unit costs (its pieces' traffic and the join), in tiles: units of one length stay
// whole where that makes no run longer by more.  Without it 16 x 512 candidates over 2048 tokens
// of 2 heads take 43.5 us for 37.0, and 30 x 512 over 1024 take 55 for 43 (but 40 x 128 over 512
// of 4 heads 32.6 for 34.2); with no limit 20 x 512 over 2048 take 62 for 47.
constexpr int kCutTiles = 8;
constexpr int kPanel = 16384; // 64 query columns of P^T: 128 keys x 128 bytes

constexpr int kKeySlots = 4;  // tiles of key data ahead

enum Bars { K_FULL = 0, K_EMPTY = K_FULL + kKStages, C_FULL = K_EMPTY + kKStages, C_EMPTY = C_FULL + kVStages,
            S_FULL = C_EMPTY + kVStages, P_FULL = S_FULL + 4, V_FULL = P_FULL + 4,
            V_EMPTY = V_FULL + 2, KEY_FULL = V_EMPTY + 2, KEY_EMPTY = KEY_FULL + kKeySlots,
            Q_FULL = KEY_EMPTY + kKeySlots, Q_EMPTY = Q_FULL + 2, O_FULL = Q_EMPTY + 2, O_FREE = O_FULL + 1,
            MMA_DONE = O_FREE + 1, NBARS = MMA_DONE + 2 };

// what the epilogue needs to know of a tile's keys: the bias against column 0 and the scale, both halved (scale -1:
// no token), position and stamp
struct KeyInfo {
    float2 bias_scale[kTile];
    int pos[kTile];
    int64_t ts[kTile];
};

// A piece of the run, and what the epilogue needs to know of its queries.  Written by the
// warps that split the queries; the MMA and epilogue warps know the run from here alone.
struct QueryInfo {
    int64_t row;    // first row
    int64_t plane;  // of part_w: the first 64 queries' weights of the piece's first key
    int count, cols;  // tiles (0: the run has ended), queries
    int head, k, whole, last;  // first tile; the whole unit; up to the unit's end
    float chunk_scale[8];  // one scale of 16 columns, or -1: each its own
    int chunk_same[8];     // every column has row 0's position and stamp
    int pos_lo[8], pos_hi[8];  // a chunk's least and largest position and stamp
    int64_t ts_lo[8], ts_hi[8];
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
    static constexpr int KEYS = INFO + 2 * (int)sizeof(QueryInfo);
    static constexpr int BAR = KEYS + kKeySlots * (int)sizeof(KeyInfo);
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
    for (int w = 0; w < min(kW, (c.B + 32 * per - 1) / (32 * per)); w++) {
        if (w < warp)
            before += sums[w];
        total += sums[w];
        lo = min(lo, (int)sums[kW + w]);
        hi = max(hi, (int)sums[2 * kW + w]);
    }
    // equal units: whole ones, unless that makes the longest run much longer than the mean
    int64_t start, end;
    if (total <= 0xffffffffu / (unsigned)(ctas + kCutTiles + 1)) {  // a 64-bit division takes hundreds of cycles
        const unsigned all = (unsigned)total, n = (unsigned)ctas;
        unsigned grain = 1;
        if (lo == hi && (all / hi + n - 1) / n * hi <= all / n + kCutTiles)
            grain = hi;
        const unsigned units = all / grain;
        start = units * (unsigned)cta / n * grain;
        end = units * (unsigned)(cta + 1) / n * grain;
    } else {
        start = total / ctas * cta + total % ctas * cta / ctas;
        end = total / ctas * (cta + 1) + total % ctas * (cta + 1) / ctas;
    }
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

// SiLU(2 h)
__device__ __forceinline__ float silu_half(float h) { return fmaf(h, tanh_approx(h), h); }

// One lane of a converged warp.  Under this predicate the compiler knows that one thread
// issues; under `lane == 0` it wraps every TMA, MMA and commit in a loop over the active
// lanes, which took 100 cycles an MMA.
__device__ __forceinline__ bool elect_one()
{
    uint32_t p;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
    return p != 0;
}

// 32 lanes x 4 consecutive 32-bit columns
__device__ __forceinline__ void tmem_ld4(uint32_t taddr, float *v)
{
    uint32_t *r = reinterpret_cast<uint32_t *>(v);
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];\n"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(taddr));
}

// P^T of eight scores into 16 bytes of a row of the panel.
__device__ __forceinline__ void put_p8(const float *x, unsigned char *dst)
{
    *reinterpret_cast<uint4 *>(dst) =
        make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
}

// A chunk of 16 queries whose biases or scales differ: this key's P^T, and the sum of
// its magnitudes over the first n.  Where the whole warp's pairs share an index of a
// table, it is read once.
__device__ __forceinline__ float chunk_general(uint32_t taddr, int cc, int n, const CacheAttnArgs &a,
                                               const QueryInfo &qi, bool live, int pj,
                                               int64_t tj, float half_scale, unsigned char *dst, int row_p)
{
    const int ch = cc >> 4;
    const float *rp = a.rab_pos + qi.head * a.pos_hstride, *rt = a.rab_time + qi.head * a.time_hstride;
    const int i0 = pos_index(qi.pos_lo[ch], pj, a.pos_lo, a.pos_hi), i1 = pos_index(qi.pos_hi[ch], pj, a.pos_lo, a.pos_hi);
    const int u0 = time_bucket(qi.ts_lo[ch], tj, a.nb), u1 = time_bucket(qi.ts_hi[ch], tj, a.nb);
    const bool one_p = __all_sync(0xffffffffu, !live || i0 == i1), one_t = __all_sync(0xffffffffu, !live || u0 == u1);
    const float bp = live ? rp[i0] : 0.f, bt = live ? rt[u0] : 0.f;
    float w = 0.f;
    // rolled: short runs pay for every line of code they fetch for the first time
#pragma unroll 1
    for (int e0 = 0; e0 < 16; e0 += 4) {
        float x[4], b[4];
        tmem_ld4(taddr + e0, x);
#pragma unroll
        for (int e = 0; e < 4; e++)
            b[e] = one_p ? bp : rp[pos_index(qi.pos[cc + e0 + e], pj, a.pos_lo, a.pos_hi)];
#pragma unroll
        for (int e = 0; e < 4; e++)
            b[e] += one_t ? bt : rt[time_bucket(qi.ts[cc + e0 + e], tj, a.nb)];
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 4; e++) {
            x[e] = silu_half(fmaf(x[e], half_scale * qi.scale[cc + e0 + e], 0.5f * b[e]));
            w += e0 + e < n ? fabsf(x[e]) : 0.f;
        }
        *reinterpret_cast<uint2 *>(dst + ((((cc + e0) >> 3 & 7) ^ (row_p & 7)) * 16) + 2 * (e0 & 4)) =
            make_uint2(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]));
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
    KeyInfo *keys = reinterpret_cast<KeyInfo *>(sm + LY::KEYS);

    int2 *v_scales = reinterpret_cast<int2 *>(sm + LY::MISC + 48);  // of the tiles in the value ring, as bits

    if (threadIdx.x == 0) {
        for (int i = 0; i < NBARS; i++) {
            int n = 1;
            if (i >= S_FULL && i < S_FULL + 4)
                n = 2;  // S^T is there, and P^T of the item four back has been read
            else if ((i >= P_FULL && i < P_FULL + 4) || (i >= KEY_FULL && i < KEY_FULL + kKeySlots))
                n = 4;
            else if (i == Q_FULL || i == Q_FULL + 1)
                n = 8;
            else if (i == V_FULL || i == V_FULL + 1 || (i >= C_EMPTY && i < C_EMPTY + kVStages))
                n = D / 32;
            else if (i == Q_EMPTY || i == Q_EMPTY + 1)
                n = 18;
            else if (i == O_FREE)
                n = 16;
            mbar_init(bar(i), n);
        }
        *abort_flag = 0;
        fence_mbar_init();
        for (int i = 0; i < 4; i++)  // nothing to read before the first items
            mbar_arrive(bar(S_FULL + i));
        tma_prefetch(&tk);
        tma_prefetch(&tv);
    }
    if (warp == 1)
        tmem_alloc(base + LY::MISC, 512);
    int64_t *found = reinterpret_cast<int64_t *>(sm + LY::MISC + 16);
    const bool work = find_run(c, blockIdx.x, gridDim.x, reinterpret_cast<int64_t *>(sm + LY::P), found);
    CacheAttnPiece *pieces = a.pieces + 2 * blockIdx.x;
    if (threadIdx.x < 2)  // no piece, unless one is recorded at its end
        pieces[threadIdx.x].cols = 0;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(sm + LY::MISC);
    if (!work) {
        if (warp == 1)
            tmem_dealloc(tmem, 512);
        return;
    }
    Walk start;
    start.b = (int)found[0];
    start.left = found[2];
    start.piece = 0;
    start.load(c);
    if (found[1] >> 31) {
        start.unit = (int)(found[1] / start.z.kt);
        start.k = (int)(found[1] % start.z.kt);
    } else {
        start.unit = (int)found[1] / start.z.kt;
        start.k = (int)found[1] % start.z.kt;
    }
    bool ok = true;
    auto wait = [&](int i, int parity) { return mbar_wait_warp(bar(i), parity & 1, abort_flag, hdr, a.wait_limit); };

    if (warp == 0) {
        // ---------------- codes ----------------
        int g = 0, k_loads = 0, v_loads = 0;
        for (Walk w = start; ok && w.left > 0; w.next(c)) {
            const int h = w.head(), pages = (w.s.len + kPage - 1) / kPage, count = w.count();
            int held = -1, held_scale = 0;  // lane: a page of this and the next 15 tiles, its v_scale's bits
            for (int t = 0; t < count; t++, g++) {
                const int k = w.k + t, kst = g % kKStages, vst = g % kVStages;
                if (t % 16 == 0) {
                    held = -1;
                    if (2 * k + lane < pages) {
                        held = table_page(c.table, c, w.b, 2 * k + lane);
                        if (held < 0)
                            atomicOr(&hdr->flag, FLAG_CACHE_PAGE);
                    }
                    held_scale = held >= 0 ? __float_as_int(c.v_scale[(int64_t)held * c.H + h]) : 0;
                }
                const int page[2] = {__shfl_sync(0xffffffffu, held, 2 * (t % 16)),
                                     __shfl_sync(0xffffffffu, held, 2 * (t % 16) + 1)};
                const int sc0 = __shfl_sync(0xffffffffu, held_scale, 2 * (t % 16));
                const int sc1 = __shfl_sync(0xffffffffu, held_scale, 2 * (t % 16) + 1);
                const uint32_t bytes = ((page[0] >= 0) + (page[1] >= 0)) * kPage * D;
                ok = g < kKStages || wait(K_EMPTY + kst, g / kKStages - 1);
                if (!ok)
                    break;
                // (the hook: of the last CTA, whose run has tiles if any has)
                if (elect_one() && !(a.withhold && g == 0 && blockIdx.x == gridDim.x - 1)) {
                    mbar_expect_tx(bar(K_FULL + kst), bytes);
#pragma unroll
                    for (int e = 0; e < 2; e++)
                        if (page[e] >= 0)
                            tma_load_2d(base + LY::K + kst * LY::KT + e * kPage * D, &tk, 0,
                                        (page[e] * c.H + h) * kPage, bar(K_FULL + kst));
                }
                k_loads = g + 1;
                ok = g < kVStages || wait(C_EMPTY + vst, g / kVStages - 1);
                if (!ok)
                    break;
                if (elect_one()) {
                    v_scales[vst] = make_int2(sc0, sc1);
                    mbar_expect_tx(bar(C_FULL + vst), bytes);
#pragma unroll
                    for (int e = 0; e < 2; e++)
                        if (page[e] >= 0)
                            tma_load_2d(base + LY::V + vst * LY::KT + e * kPage * D, &tv, 0,
                                        (page[e] * c.H + h) * D, bar(C_FULL + vst));
                }
                v_loads = g + 1;
                __syncwarp();
            }
        }
        for (int i = max(k_loads - kKStages, 0); i < k_loads; i++)
            mbar_drain(bar(K_FULL + i % kKStages), i / kKStages & 1);
        for (int i = max(v_loads - kVStages, 0); i < v_loads; i++)
            mbar_drain(bar(C_FULL + i % kVStages), i / kVStages & 1);
    } else if (warp == 1) {
        // ---------------- S^T = K Q^T ----------------
        int g = 0, it = 0;
        for (int piece = 0; ok; piece++) {
            const int qs = piece & 1;
            if (!(ok = wait(Q_FULL + qs, piece >> 1)))
                break;
            const int count = info[qs].count, halves = info[qs].cols > 64 ? 2 : 1;
            if (count == 0)
                break;
            for (int t = 0; ok && t < count; t++, g++) {
                const int st = g % kKStages;
                // the key data too: S_FULL then stands for both
                if (!(ok = wait(K_FULL + st, g / kKStages) && wait(KEY_FULL + g % kKeySlots, g / kKeySlots)))
                    break;
                // both halves at once where their buffers are neighbours
                const int wide = halves == 2 && (it & 1) == 0 ? 2 : 1;
                for (int hf = 0; hf < halves; hf += wide, it += wide) {
                    // a buffer is free once the item four back has become P^T
                    ok = (it < 4 || wait(P_FULL + (it & 3), (it >> 2) - 1)) &&
                         (wide == 1 || it < 4 || wait(P_FULL + (it & 3) + 1, (it >> 2) - 1));
                    if (!ok)
                        break;
                    tc_fence_after();
                    if (elect_one()) {
                        const uint32_t id = idesc_e4m3(128, 0, 0, 0) | ((uint32_t)(64 * wide >> 3) << 17);
                        const uint64_t kd = code_desc<D>(base + LY::K + st * LY::KT);
                        const uint64_t qd = code_desc<D>(base + LY::Q + 2 * qs * LY::KT + hf * 64 * D);
#pragma unroll
                        for (int i = 0; i < 2 * (D / 32); i++)  // 32 bytes of a row a step: 2 in the address field
                            umma_e4m3(tmem + (it & 3) * 64, kd + 2 * (i % (D / 32)),
                                      qd + i / (D / 32) * (LY::KT >> 4) + 2 * (i % (D / 32)), id, i > 0);
                        umma_commit(bar(S_FULL + (it & 3)));
                        if (wide == 2)
                            umma_commit(bar(S_FULL + (it & 3) + 1));
                        if (hf + wide == halves) {
                            umma_commit(bar(K_EMPTY + st));
                            if (t + 1 == count)
                                umma_commit(bar(Q_EMPTY + qs));
                        }
                    }
                    __syncwarp();
                }
            }
        }
    } else if (warp == 2) {
        // ---------------- O^T += V^T P^T ----------------
        int g = 0, it = 0;
        for (int piece = 0; ok; piece++) {
            const int qs = piece & 1;
            if (!(ok = wait(Q_FULL + qs, piece >> 1)))
                break;
            const int count = info[qs].count, halves = info[qs].cols > 64 ? 2 : 1;
            if (count == 0)
                break;
            __syncwarp();
            if (lane == 0)
                mbar_arrive(bar(Q_EMPTY + qs));
            if (piece > 0 && !(ok = wait(O_FREE, piece - 1)))
                break;
            for (int t = 0; ok && t < count; t++, g++) {
                const int vb = g & 1;
                if (!(ok = wait(V_FULL + vb, g >> 1)))
                    break;
                for (int hf = 0; hf < halves; hf++, it++) {
                    if (!(ok = wait(P_FULL + (it & 3), it >> 2)))
                        break;
                    tc_fence_after();
                    if (elect_one()) {
                        constexpr uint32_t id = idesc_bf16(128, 64, 0, 1);
                        const uint64_t pd = smem_desc_sw128(base + LY::P + (it & 3) * kPanel, kPanel, 1024);
#pragma unroll
                        for (int ks = 0; ks < kTile / 16; ks++)  // 16 rows of P^T a step
                            umma_bf16_ts(tmem + 256 + hf * 64, tmem + 384 + vb * 64 + ks * 8, pd + ks * (2048 >> 4), id,
                                         ks > 0 || t > 0);
                        umma_commit(bar(S_FULL + (it & 3)));
                        if (hf + 1 == halves) {
                            mbar_arrive(bar(KEY_EMPTY + g % kKeySlots));  // every P^T of the tile is there
                            umma_commit(bar(V_EMPTY + vb));
                            if (t + 1 == count)
                                umma_commit(bar(O_FULL));
                        }
                    }
                    __syncwarp();
                }
            }
        }
    } else if (warp >= 20) {
        // ---------------- queries, keys' biases and values ----------------
        // Two groups of four warps take every other tile each: the thread is a key of the
        // tile first, then a dim of its values.
        const int group = (warp - 20) >> 2, quarter = warp & 3, r = quarter * 32 + lane;
        int g0 = 0, pieces_done = 0;
        for (Walk w = start; ok && w.left > 0; w.next(c)) {
            const int qs = w.piece & 1, h = w.head(), q0 = w.q0(), cols = w.cols(), count = w.count();
            const float *rp = a.rab_pos + h * a.pos_hstride, *rt = a.rab_time + h * a.time_hstride;
            // What a tile needs of a key is fetched ahead, one step of the chain a tile: its page,
            // its position, stamp and scale (-2: no token), its biases against column 0.
            struct Key {
                int pos;
                int64_t ts;
                float scale;
            };
            auto page_at = [&](int t) {
                const int j = (w.k + t) * kTile + r;
                return t < count && j < w.s.len ? table_page(c.table, c, w.b, j / kPage) : -1;
            };
            auto key_at = [&](int page) {
                const int64_t at = page >= 0 ? (int64_t)page * kPage + r % kPage : 0;
                return Key{c.positions[at], c.timestamps[at], page >= 0 ? c.k_scale[(int64_t)page * c.H + h] : -2.f};
            };
            const int first = (g0 ^ group) & 1, page0 = page_at(first), page1 = page_at(first + 2);
            int page = page_at(first + 4);
            const int p_i = w.s.pos + token_pos(q0, w.s.hist, a.cand_own);
            const int64_t t_i = c.ts[w.s.s0 + q0];
            Key now, next;
            float bp, bt;
            if (w.piece >= 2 && !(ok = wait(Q_EMPTY + qs, (w.piece >> 1) - 1)))
                break;
            {
                // the queries' split: 16 rows a warp, LR lanes a row, eight elements a lane.  The
                // row passes through the places of its two parts (eight bytes a lane in each),
                // read back by the lane that wrote.
                QueryInfo &qi = info[qs];
                constexpr int LR = D / 8, RI = 32 / LR, NI = 16 / RI;
                const int chunk = warp - 20, lr = lane / LR, lc = lane % LR, row = 16 * chunk + (lane & 15);
                const __nv_bfloat16 *qp =
                    static_cast<const __nv_bfloat16 *>(a.q) + (w.s.s0 + q0) * a.ldq + (int64_t)h * D + 8 * lc;
                unsigned char *q1 = sm + LY::Q + 2 * qs * LY::KT;
                auto place = [&](int rr) { return q1 + rr * D + code_chunk<D>(rr, lc >> 1) * 16 + 8 * (lc & 1); };
                uint4 x[NI];
#pragma unroll
                for (int j = 0; j < NI; j++) {
                    const int rr = 16 * chunk + RI * j + lr;
                    x[j] = rr < cols ? *reinterpret_cast<const uint4 *>(qp + rr * a.ldq) : make_uint4(0u, 0u, 0u, 0u);
                }
                now = key_at(page0);
                next = key_at(page1);
                // positions and stamps of the chunk: their range
                const int i = q0 + (row < cols ? row : 0);
                const int pi = w.s.pos + token_pos(i, w.s.hist, a.cand_own);
                const int64_t ti = c.ts[w.s.s0 + i];
                const bool all_same = __all_sync(0xffffffffu, pi == p_i && ti == t_i);
                int plo = pi, phi = pi;
                int64_t tlo = ti, thi = ti;
                if (!all_same) {
#pragma unroll
                    for (int o = 8; o > 0; o >>= 1) {
                        plo = min(plo, __shfl_xor_sync(0xffffffffu, plo, o));
                        phi = max(phi, __shfl_xor_sync(0xffffffffu, phi, o));
                        tlo = min(tlo, __shfl_xor_sync(0xffffffffu, tlo, o));
                        thi = max(thi, __shfl_xor_sync(0xffffffffu, thi, o));
                    }
                }
                // largest magnitude of each row, as bf16 bits at a float's place
                auto row_max = [&](const uint32_t *ww) {
                    uint32_t m = 0;
#pragma unroll
                    for (int e = 0; e < 4; e++)
                        m = max(m, max((ww[e] & 0x7fffu) << 16, ww[e] & 0x7fff0000u));
#pragma unroll
                    for (int o = LR / 2; o > 0; o >>= 1)
                        m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
                    return m;
                };
                uint32_t all = 0, least = 0xffffffffu;
#pragma unroll
                for (int j = 0; j < NI; j++) {
                    const uint32_t ww[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
                    const uint32_t m = row_max(ww);
                    all = max(all, m);
                    least = min(least, m ? m : 0xffffffffu);
                    unsigned char *at = place(16 * chunk + RI * j + lr);
                    *reinterpret_cast<uint2 *>(at) = make_uint2(ww[0], ww[1]);
                    *reinterpret_cast<uint2 *>(at + LY::KT) = make_uint2(ww[2], ww[3]);
                }
                all = __reduce_max_sync(0xffffffffu, all);
                least = __reduce_min_sync(0xffffffffu, least);
                bp = rp[pos_index(p_i, now.pos, a.pos_lo, a.pos_hi)];
                bt = rt[time_bucket(t_i, now.ts, a.nb)];
                // one scale for the chunk's rows if none lies far below
                const bool one = all == 0 || (all >> 23) - (least >> 23) <= 2;
                if (lane < 16) {
                    qi.pos[row] = pi;
                    qi.ts[row] = ti;
                }
                if (chunk == 0 && lane == 0) {
                    qi.row = w.s.s0 + q0;
                    qi.plane = ((int64_t)(q0 / 64 * c.H + h) * c.B + w.b) * a.plan.lcap + (int64_t)w.k * kTile;
                    qi.count = count;
                    qi.cols = cols;
                    qi.head = h;
                    qi.k = w.k;
                    qi.whole = w.k == 0 && count == w.z.kt;
                    qi.last = w.k + count == w.z.kt;
                }
                if (lane == 0) {
                    qi.chunk_scale[chunk] = one ? block_scale(all) : -1.f;
                    qi.chunk_same[chunk] = all_same;
                    qi.pos_lo[chunk] = plo;
                    qi.pos_hi[chunk] = phi;
                    qi.ts_lo[chunk] = tlo;
                    qi.ts_hi[chunk] = thi;
                }
#pragma unroll 4
                for (int j = 0; j < NI; j++) {
                    const int rr = 16 * chunk + RI * j + lr;
                    unsigned char *at = place(rr);
                    const uint2 x0 = *reinterpret_cast<const uint2 *>(at);
                    const uint2 x1 = *reinterpret_cast<const uint2 *>(at + LY::KT);
                    const uint32_t ww[4] = {x0.x, x0.y, x1.x, x1.y};
                    const float scale = block_scale(one ? all : row_max(ww)), inv = scale_inverse(scale);
                    if (lc == 0)
                        qi.scale[rr] = scale;
                    uint32_t hi[2] = {0, 0}, lo[2] = {0, 0};
#pragma unroll
                    for (int e = 0; e < 4; e++) {
                        const float y0 = __uint_as_float(ww[e] << 16) * inv, y1 = __uint_as_float(ww[e] & 0xffff0000u) * inv;
                        const uint32_t p = f32x2_to_e4m3x2(y0, y1);
                        const float2 f = e4m3x2_to_f32x2(p);
                        hi[e >> 1] |= p << (16 * (e & 1));
                        lo[e >> 1] |= f32x2_to_e4m3x2(y0 - f.x, y1 - f.y) << (16 * (e & 1));
                    }
                    *reinterpret_cast<uint2 *>(at) = make_uint2(hi[0], hi[1]);
                    *reinterpret_cast<uint2 *>(at + LY::KT) = make_uint2(lo[0], lo[1]);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(bar(Q_FULL + qs));
            }
            for (int t = first; t < count; t += 2) {
                const int g = g0 + t, k = w.k + t, slot = g % kKeySlots;
                if (g >= kKeySlots && !(ok = wait(KEY_EMPTY + slot, g / kKeySlots - 1)))
                    break;
                KeyInfo &ki = keys[slot];
                ki.bias_scale[r] = make_float2(0.5f * (bp + bt), 0.5f * now.scale);
                ki.pos[r] = now.pos;
                ki.ts[r] = now.ts;
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(bar(KEY_FULL + slot));
                now = next;
                bp = rp[pos_index(p_i, now.pos, a.pos_lo, a.pos_hi)];
                bt = rt[time_bucket(t_i, now.ts, a.nb)];
                next = key_at(page);
                page = page_at(t + 6);
                if (r >= D)  // d = 64 has half the rows of V^T
                    continue;
                if (!(ok = wait(C_FULL + group, g >> 1) && (g < 2 || wait(V_EMPTY + group, (g >> 1) - 1))))
                    break;
                const int2 sc = v_scales[group];
                tc_fence_after();
                const unsigned char *vrow = sm + LY::V + group * LY::KT + r * kPage;
                const uint32_t dst = tmem + ((uint32_t)(quarter * 32) << 16) + 384 + group * 64;
                auto codes = [&](int i) {  // 16 keys of the tile
                    return *reinterpret_cast<const uint4 *>(vrow + (i >> 2) * kPage * D + ((i & 3) ^ ((r >> 1) & 3)) * 16);
                };
                // times the scale 2^x and the 2^120 that the conversion leaves out: one factor
                // where bf16 has 2^(120 + x)
                const int x0 = (sc.x >> 23 & 255) - 127, x1 = (sc.y >> 23 & 255) - 127;
                const bool plain = (k + 1) * kTile <= w.s.len && sc.x != 0 && sc.y != 0 && max(x0, x1) <= 7;
                if (plain) {
                    uint4 v[8];
#pragma unroll
                    for (int i = 0; i < 8; i++)
                        v[i] = codes(i);
#pragma unroll
                    for (int q = 0; q < 4; q++) {
                        const uint32_t f = pow2_bf16x2(120 + (q < 2 ? x0 : x1));
                        uint32_t pk[16];
#pragma unroll
                        for (int i = 0; i < 8; i++) {
                            const uint4 &y = v[2 * q + (i >> 2)];
                            const uint32_t c4 = (i & 3) == 0 ? y.x : (i & 3) == 1 ? y.y : (i & 3) == 2 ? y.z : y.w;
                            pk[2 * i] = mul_bf16x2(even_codes(c4), f);
                            pk[2 * i + 1] = mul_bf16x2(odd_codes(c4), f);
                        }
                        tmem_st16(dst + 16 * q, pk);
                    }
                } else {
                    // a ragged or missing page (codes there may be anything), a scale of 0, NaN or
                    // above 2^7: two factors, a NaN scale as it is
#pragma unroll 1
                    for (int q = 0; q < 4; q++) {
                        const int bits = q < 2 ? sc.x : sc.y, x = q < 2 ? x0 : x1;
                        const int n = bits == 0 ? 0 : w.s.len - k * kTile - 32 * q;
                        const int e1 = x == 128 ? 120 : min(120 + max(x, -126), 127);
                        const uint32_t f1 = pow2_bf16x2(e1);
                        const uint32_t f2 = x == 128 ? 0x7fff7fffu : pow2_bf16x2(max(120 + x - e1, 0));
                        const uint4 y0 = codes(2 * q), y1 = codes(2 * q + 1);
                        const uint32_t c8[8] = {y0.x, y0.y, y0.z, y0.w, y1.x, y1.y, y1.z, y1.w};
                        uint32_t pk[16];
#pragma unroll
                        for (int i = 0; i < 8; i++) {
                            const uint32_t c4 = n >= 4 * i + 4 ? c8[i] : n <= 4 * i ? 0u : c8[i] & ((1u << (8 * (n - 4 * i))) - 1u);
                            pk[2 * i] = mul_bf16x2(mul_bf16x2(even_codes(c4), f1), f2);
                            pk[2 * i + 1] = mul_bf16x2(mul_bf16x2(odd_codes(c4), f1), f2);
                        }
                        tmem_st16(dst + 16 * q, pk);
                    }
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(bar(C_EMPTY + group));
                    mbar_arrive(bar(V_FULL + group));
                }
            }
            g0 += count;
            pieces_done++;
        }
        const int qs = pieces_done & 1;
        if (ok && (pieces_done < 2 || wait(Q_EMPTY + qs, (pieces_done >> 1) - 1))) {
            if (warp == 20 && lane == 0)
                info[qs].count = 0;
            __syncwarp();
            if (lane == 0)
                mbar_arrive(bar(Q_FULL + qs));
        }
    } else if (warp >= 4) {
        // ---------------- S^T to P^T ----------------
        const int group = (warp - 4) >> 2, quarter = warp & 3;
        const int r = quarter * 32 + lane, row_p = key_row(r);  // key of the tile, its row of P^T
        const uint32_t trow = tmem + ((uint32_t)(quarter * 32) << 16), taddr = trow + group * 64;
        unsigned char *prow = sm + LY::P + group * kPanel + row_p * 128;
        int it0 = 0, g0 = 0;  // items and tiles before this piece
        for (int piece = 0; ok; piece++) {
            const int qs = piece & 1;
            const QueryInfo &qi = info[qs];
            if (!(ok = wait(Q_FULL + qs, piece >> 1)))
                break;
            const int count = qi.count;
            if (count == 0)
                break;
            // Items (a tile's 64 columns) go round the groups; a group keeps its buffer, and
            // within a unit its half.
            const int halves = qi.cols > 64 ? 2 : 1, i0 = (group - it0) & 3;  // the group's first item here
            const int hf = halves == 2 ? i0 & 1 : 0, first = halves == 2 ? i0 >> 1 : i0, step = 4 / halves;
            const int c0 = hf * 64, n = min(qi.cols - c0, 64);
            const float *cs = qi.chunk_scale + 4 * hf;  // the scales of the half's chunks
            bool same = true;
#pragma unroll
            for (int i = 0; i < 4; i++)
                same = same && (16 * i >= n || (qi.chunk_same[4 * hf + i] && cs[i] != -1.f));
            for (int t = first; t < count; t += step) {
                const int it = it0 + halves * t + hf, slot = (g0 + t) % kKeySlots;
                if (!(ok = wait(S_FULL + group, it >> 2)))
                    break;
                tc_fence_after();
                const float2 bs = keys[slot].bias_scale[r];
                const bool live = bs.y != -1.f;
                float wsum = 0.f;
                if (same) {
#pragma unroll 1
                    for (int q = 0; 32 * q < n; q++) {
                        float x[32];
                        tmem_ld32(taddr + 32 * q, x);
                        tmem_wait_ld();
                        const float f0 = bs.y * cs[2 * q], f1 = bs.y * cs[2 * q + 1];
#pragma unroll
                        for (int e = 0; e < 32; e++)
                            x[e] = silu_half(fmaf(x[e], e < 16 ? f0 : f1, bs.x));
#pragma unroll
                        for (int e = 0; e < 4; e++)
                            put_p8(x + 8 * e, prow + ((4 * q + e) ^ (row_p & 7)) * 16);
                        if (a.part_w) {
                            float w0 = 0.f, w1 = 0.f;
                            if (n >= 32 * q + 32) {
#pragma unroll
                                for (int e = 0; e < 32; e += 2)
                                    w0 += fabsf(x[e]), w1 += fabsf(x[e + 1]);
                            } else {
#pragma unroll
                                for (int e = 0; e < 32; e++)
                                    w0 += 32 * q + e < n ? fabsf(x[e]) : 0.f;
                            }
                            wsum += w0 + w1;
                        }
                    }
                } else {
                    const int pj = keys[slot].pos[r];
                    const int64_t tj = keys[slot].ts[r];
                    for (int cc = 0; cc < n; cc += 16)
                        wsum += chunk_general(taddr + cc, c0 + cc, n - cc, a, qi, live, pj, tj, bs.y, prow, row_p);
                }
                if (!live)  // no token, and S^T of whatever the tile holds there: P is 0
                    for (int e = 0; e < 8; e++)
                        *reinterpret_cast<uint4 *>(prow + e * 16) = make_uint4(0u, 0u, 0u, 0u);
                fence_proxy_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(bar(P_FULL + group));
                if (a.part_w && (qi.k + t) * kTile + r < a.plan.lcap)
                    a.part_w[qi.plane + (int64_t)hf * c.H * c.B * a.plan.lcap + t * kTile + r] = live ? wsum : 0.f;
            }
            g0 += count;
            it0 += count * halves;
            const bool whole = qi.whole;
            // this group's quarter of the columns; the addend of a whole unit, before the wait
            const int col0 = group * 32, nc = min(qi.cols - col0, 32);
            const int64_t at = ((qi.row + col0 + (lane >> 2)) * c.H + qi.head) * D + quarter * 32 + 8 * (lane & 3);
            const int64_t eight = (int64_t)8 * c.H * D;  // eight queries on
            uint4 add[4];
            if (whole && a.addend && quarter * 32 < D)
#pragma unroll
                for (int i = 0; i < 4; i++)
                    if (8 * i + (lane >> 2) < nc)
                        add[i] = *reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(a.addend) + at + i * eight);
            if (!(ok = ok && wait(O_FULL, piece)))
                break;
            tc_fence_after();
            // O^T: lane = dim, column = query.  A whole unit leaves through the warp's own rows of
            // its P^T buffer, 32 queries x 32 dims, so that memory sees 16-byte accesses.
            const int slot = qi.k > 0 ? 0 : 1;
            if (quarter * 32 < D && nc > 0) {
                unsigned char *stage = sm + LY::P + group * kPanel + quarter * 4096;
                float ov[32];
                tmem_ld32(trow + 256 + col0, ov);
                tmem_wait_ld();
                if (!whole) {
                    float *part = a.part_o + ((int64_t)(2 * blockIdx.x + slot) * kTile + col0) * D + r;
#pragma unroll
                    for (int e = 0; e < 32; e++)
                        if (e < nc)
                            part[e * D] = ov[e];
                } else {
                    // odd queries with fours of dims swapped, against bank conflicts
#pragma unroll
                    for (int e = 0; e < 32; e++)
                        *reinterpret_cast<float *>(stage + e * 128 + (lane ^ ((e & 1) << 2)) * 4) = ov[e] * a.inv_n;
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < 4; i++) {
                        const int qq = 8 * i + (lane >> 2), x0 = (8 * (lane & 3)) ^ ((qq & 1) << 2);
                        const float *src = reinterpret_cast<const float *>(stage + qq * 128);
                        const float4 y0 = *reinterpret_cast<const float4 *>(src + x0);
                        const float4 y1 = *reinterpret_cast<const float4 *>(src + (x0 ^ 4));
                        if (qq < nc) {
                            float y[8] = {y0.x, y0.y, y0.z, y0.w, y1.x, y1.y, y1.z, y1.w};
                            if (a.addend) {
                                const uint32_t aw[4] = {add[i].x, add[i].y, add[i].z, add[i].w};
#pragma unroll
                                for (int e = 0; e < 4; e++) {
                                    y[2 * e] += __uint_as_float(aw[e] << 16);
                                    y[2 * e + 1] += __uint_as_float(aw[e] & 0xffff0000u);
                                }
                            }
                            *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.out) + at + i * eight) =
                                make_uint4(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]), pack_bf16(y[4], y[5]),
                                           pack_bf16(y[6], y[7]));
                        }
                    }
                    __syncwarp();
                }
            }
            if (!whole && warp == 4 && lane == 0)
                pieces[slot] = CacheAttnPiece{qi.row, qi.head, qi.cols, qi.last};
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(bar(O_FREE));
                mbar_arrive(bar(Q_EMPTY + qs));
            }
        }
    }
    if (warp == 1 || warp == 2) {  // MMAs that an aborting CTA left
        if (elect_one())
            umma_commit(bar(MMA_DONE + warp - 1));
        __syncwarp();
        mbar_drain(bar(MMA_DONE + warp - 1), 0);
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
        if (threadIdx.x == 0) {
            const int bits = s.bits | cache_offset_bits(c, x);
            if (bits)
                atomicOr(&c.hdr->flag, bits);
        }
        if (s.bits || s.len > 0)
            return;
        const int64_t width = (int64_t)c.H * D;
        for (int64_t i = s.s0 * width + threadIdx.x; i < (s.s0 + s.n) * width; i += 256)
            out[i] = add ? add[i] : __float2bfloat16_rn(0.f);
        return;
    }
    x -= c.B;
    cache_join_weights(a, x / w_blocks, ((x % w_blocks) * 256 + threadIdx.x) * 4);
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
    const int w_blocks = a.weights_out ? (c.max_cache_len + 1023) / 1024 : 0;
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
