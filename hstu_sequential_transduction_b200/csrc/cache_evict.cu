// Eviction from the 8-bit key/value cache by accumulated attention weight.
//
// Select (one CTA per sequence): weights become integers that compare as the weights
// do (NaN 0), the first 16 a thread in registers.  Histograms in shared memory of 11, 11
// and 10 bits find the m-th largest of the unprotected tokens; the first digit holds two
// bits of the fraction, for weights share few exponents and would crowd into few bins.
// Two scans then place the kept indices, ties to the lowest.  Bound by one SM's
// instructions: a thread takes four neighbours at a time, which share a page lookup and
// count as one byte of a packed scan (14 us for 32 sequences of 12,288 tokens; 25 with
// a lookup and a ballot per token, 33 with a count per bit of the key).
//
// Move (one CTA per new block and head, a thread per dim): keys are gathered as rows of
// 16-byte pieces.  Values are stored transposed: a thread takes its dim's row of every
// source page the block draws on, the next page's on its way meanwhile, through a
// shared-memory row of its own (no barriers wider than a warp), and picks the kept bytes;
// memory sees the warp's 32 rows as 512-byte accesses.  The block gets
// its own scale from the largest decoded magnitude.  The kept keys and the source pages of
// the values are read once, the new block written: 88 us for 32 sequences cut from
// 12,288 tokens to 4,096 (4 heads, d = 128), 4.6 TB/s of that traffic, with shared
// memory 83 % busy picking bytes.
#include <algorithm>

#include "cache.cuh"

namespace hstu {

namespace {


__device__ __forceinline__ uint32_t weight_key(float w)
{
    if (w != w)
        return 0u;
    const uint32_t u = __float_as_uint(w == 0.f ? 0.f : w);  // -0 ties with 0
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

constexpr int kSelGroups = 4;  // of four neighbours each: the keys a thread keeps in registers

// In place, exclusive prefix sums of counts[0, N); returns the total.
template <int N>
__device__ __forceinline__ int scan_counts(int *counts, int *total)
{
    __syncthreads();
    if (threadIdx.x < 32) {
        const int lane = threadIdx.x;
        int x[N / 32], sum = 0;
#pragma unroll
        for (int e = 0; e < N / 32; e++)
            sum += x[e] = counts[lane * (N / 32) + e];
        int inc = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o)
                inc += y;
        }
        if (lane == 31)
            *total = inc;
        int before = inc - sum;
#pragma unroll
        for (int e = 0; e < N / 32; e++) {
            counts[lane * (N / 32) + e] = before;
            before += x[e];
        }
    }
    __syncthreads();
    return *total;
}

// How many of the bits of each group (a nibble of `bits`) the lanes below hold, a byte a
// group (a warp holds 128 at most); the warp's counts go to counts[group * warps + warp].
__device__ __forceinline__ uint32_t rank_groups(uint32_t bits, int *counts, int warps)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t mine = 0;
#pragma unroll
    for (int i = 0; i < kSelGroups; i++)
        mine |= __popc(bits >> (4 * i) & 15u) << (8 * i);
    uint32_t inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o)
            inc += y;
    }
    if (lane == 31)
#pragma unroll
        for (int i = 0; i < kSelGroups; i++)
            counts[i * warps + warp] = inc >> (8 * i) & 255u;
    return inc - mine;
}

template <int kSelThreads>
__global__ void __launch_bounds__(kSelThreads)
cache_select_kernel(const CacheCall c, int keep, int first, int recent, const int32_t *__restrict__ new_pages,
                    int32_t *__restrict__ new_table, int32_t *__restrict__ new_lens, int32_t *__restrict__ kept,
                    uint32_t *__restrict__ keys, int64_t cap)
{
    constexpr int kSelWarps = kSelThreads / 32, kBins = 2048;
    __shared__ int slots[2][32], counts[kSelGroups * kSelWarps], bins[kBins], found[3], total;
    const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
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
    constexpr int kStep = 4 * kSelThreads, kRound = kSelGroups * kStep;
    uint32_t *rest = keys + (int64_t)b * cap;  // the keys from kRound on
    const int32_t *table = c.table + (int64_t)b * c.max_pages;
    bool bad = false;
    auto open = [&](int j) { return (unsigned)(j - early) < (unsigned)(L - late - early); };
    // of the four tokens from j on: which are open, and their keys (on a page that is none: 0)
    auto load4 = [&](int j, int entry, uint32_t *key) {
        const bool known = entry >= 0 && entry < c.num_pages;
        bad |= !known && j < L;
        const float *w = c.weights + (int64_t)(known ? entry : 0) * kPage + j % kPage;
        uint32_t bits = 0;
#pragma unroll
        for (int e = 0; e < 4; e++) {
            const float x = w[e];
            key[e] = known ? weight_key(x) : 0u;
            bits |= (uint32_t)open(j + e) << e;
        }
        return bits;
    };
    // the thread's tokens are 4 tid + kStep i + (0 .. 3)
    uint32_t key[4 * kSelGroups], opens = 0;
    int entry[kSelGroups];
#pragma unroll
    for (int i = 0; i < kSelGroups; i++)
        entry[i] = table[min(4 * tid + kStep * i, L - 1) / kPage];
#pragma unroll
    for (int i = 0; i < kSelGroups; i++)
        opens |= load4(4 * tid + kStep * i, entry[i], key + 4 * i) << (4 * i);
    for (int j = kRound + 4 * tid; j < L; j += kStep) {  // read again by this thread only
        uint32_t k4[4];
        load4(j, table[j / kPage], k4);
        for (int e = 0; e < min(L - j, 4); e++)
            rest[j + e] = k4[e];
    }
    if (bad)
        atomicOr(&c.hdr->flag, FLAG_CACHE_PAGE);
    // prefix: the m-th largest open key, of whose equals the first `ties` are kept; with
    // `exact`, the digits so far already part exactly m keys from the others
    uint32_t prefix = 0, mask = 0;
    int turn = 0, ties = m;
    bool exact = false;
    for (int shift = 21, n = kBins; m > 0 && !exact; shift = max(shift - 11, 0)) {
        for (int i = tid; i < n; i += kSelThreads)
            bins[i] = 0;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 4 * kSelGroups; i++)
            if ((opens >> i & 1) && (key[i] & mask) == prefix)
                atomicAdd(&bins[key[i] >> shift & (n - 1)], 1);
        for (int j = kRound + 4 * tid; j < L; j += kStep)
            for (int e = 0; e < min(L - j, 4); e++)
                if (open(j + e) && (rest[j + e] & mask) == prefix)
                    atomicAdd(&bins[rest[j + e] >> shift & (n - 1)], 1);
        __syncthreads();
        // from the highest bin down, the one in which the running count reaches `ties`
        const int per = n / kSelThreads, top = n - 1 - tid * per;
        int sum = 0;
        for (int e = 0; e < per; e++)
            sum += bins[top - e];
        int inc = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o)
                inc += y;
        }
        int *slot = slots[turn ^= 1];
        if (lane == 31)
            slot[warp] = inc;
        __syncthreads();
        int run = inc - sum + __reduce_add_sync(0xffffffffu, lane < warp ? slot[lane] : 0);
        if (run < ties && run + sum >= ties)
            for (int e = 0; e < per; e++) {
                const int x = bins[top - e];
                if (run < ties && run + x >= ties) {
                    found[0] = top - e;
                    found[1] = ties - run;
                    found[2] = x;
                }
                run += x;
            }
        __syncthreads();
        prefix |= (uint32_t)found[0] << shift;
        mask |= (uint32_t)(n - 1) << shift;
        ties = found[1];
        exact = found[1] == found[2];
        if (shift == 0)
            break;
        n = shift == 21 ? kBins : 1024;  // digits at 21, 10 and 0
        __syncthreads();
    }
    // in rounds of kRound tokens, in order of group, warp, lane
    int ties_before = 0, out_before = 0;
    for (int j0 = 0; j0 < L; j0 += kRound) {
        if (j0 > 0) {
            opens = 0;
#pragma unroll
            for (int i = 0; i < 4 * kSelGroups; i++) {
                const int j = j0 + 4 * tid + kStep * (i / 4) + i % 4;
                key[i] = j < L ? rest[j] : 0u;
                opens |= (uint32_t)open(j) << i;
            }
        }
        uint32_t take = 0, tie = 0;  // bit i: the thread's token i
#pragma unroll
        for (int i = 0; i < 4 * kSelGroups; i++) {
            take |= (uint32_t)(exact ? (key[i] & mask) >= prefix : key[i] > prefix) << i;
            tie |= (uint32_t)(key[i] == prefix) << i;
        }
        uint32_t live = 0;
#pragma unroll
        for (int i = 0; i < kSelGroups; i++) {
            const int left = L - (j0 + 4 * tid + kStep * i);
            live |= (left >= 4 ? 15u : left > 0 ? (1u << left) - 1u : 0u) << (4 * i);
        }
        take = ((m > 0 ? take : 0u) | ~opens) & live;
        if (m > 0 && !exact) {
            tie &= opens;
            const uint32_t below = rank_groups(tie, counts, kSelWarps);
            const int n_ties = scan_counts<kSelGroups * kSelWarps>(counts, &total);
#pragma unroll
            for (int i = 0; i < kSelGroups; i++) {
                int rank = ties_before + counts[i * kSelWarps + warp] + (int)(below >> (8 * i) & 255u);
#pragma unroll
                for (int e = 4 * i; e < 4 * i + 4; e++)
                    if (tie >> e & 1)
                        take |= (uint32_t)(rank++ < ties) << e;
            }
            ties_before += n_ties;
            __syncwarp();
        }
        const uint32_t below = rank_groups(take, counts, kSelWarps);
        const int n_out = scan_counts<kSelGroups * kSelWarps>(counts, &total);
#pragma unroll
        for (int i = 0; i < kSelGroups; i++) {
            int at = out_before + counts[i * kSelWarps + warp] + (int)(below >> (8 * i) & 255u);
#pragma unroll
            for (int e = 0; e < 4; e++)
                if (take >> (4 * i + e) & 1)
                    out[at++] = j0 + 4 * tid + kStep * i + e;
        }
        out_before += n_out;
        __syncwarp();
    }
}

__device__ __forceinline__ __half2 codes_half2(uint32_t codes)
{
    const uint32_t h = e4m3x2_to_f16x2(codes);
    return *reinterpret_cast<const __half2 *>(&h);
}

// the larger of m and four codes' magnitudes, two and two; NaN wins
__device__ __forceinline__ __half2 max_codes(__half2 m, uint32_t w)
{
    return __hmax2_nan(m, __hmax2_nan(__habs2(codes_half2(w)), __habs2(codes_half2(w >> 16))));
}

// bits of the larger of a pair of magnitudes, times the scale
__device__ __forceinline__ uint32_t magnitude(__half2 m, float scale)
{
    return __float_as_uint(__half2float(__hmax_nan(__low2half(m), __high2half(m))) * scale) & 0x7fffffffu;
}

// four codes re-rounded, each with its own ratio: one rounding, the products are exact
__device__ __forceinline__ uint32_t put4(uint32_t w, float r0, float r1, float r2, float r3)
{
    const float2 lo = e4m3x2_to_f32x2(w), hi = e4m3x2_to_f32x2(w >> 16);
    return f32x2_to_e4m3x2(lo.x * r0, lo.y * r1) | f32x2_to_e4m3x2(hi.x * r2, hi.y * r3) << 16;
}

// the same in 16 bits, for ratios of at most 2^15: a 4-bit significand times a power of
// two is exact down to f16's last place, 2^-24, far below E4M3's first tie at 2^-10
__device__ __forceinline__ uint32_t put4h(uint32_t w, __half2 r01, __half2 r23)
{
    const __half2 x = __hmul2(codes_half2(w), r01), y = __hmul2(codes_half2(w >> 16), r23);
    unsigned short lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(lo) : "r"(*reinterpret_cast<const uint32_t *>(&x)));
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(hi) : "r"(*reinterpret_cast<const uint32_t *>(&y)));
    return (uint32_t)lo | (uint32_t)hi << 16;
}

// A code that is not 0 has a ratio below 2^18, for the new scale keeps it within 448; a
// zero's ratio may be anything, infinite even.
__device__ __forceinline__ float code_ratio(float scale, float inverse) { return fminf(scale * inverse, 1048576.f); }

template <int D>
__global__ void __launch_bounds__(D, D == 32 ? 16 : 1280 / D)
cache_move_kernel(const CacheCall c, int keep, int blocks, const int32_t *__restrict__ new_pages,
                  const int32_t *__restrict__ kept)
{
    constexpr int LD = 17;  // words of a row: byte reads of 32 rows meet no bank conflict
    __shared__ uint32_t src[D * LD], dst[D * LD];
    __shared__ __align__(16) int tok_page[kPage], tok_slot[kPage];
    __shared__ __align__(16) float tok_ks[kPage], tok_vs[kPage];
    __shared__ uint32_t smax[2][D / 32];
    __shared__ __align__(8) __half tok_rk[kPage], tok_rv[kPage];  // ratios
    const int h = (int)(blockIdx.x % (unsigned)c.H);
    const int j = (int)(blockIdx.x / (unsigned)c.H % (unsigned)blocks);
    const int b = (int)(blockIdx.x / ((unsigned)c.H * (unsigned)blocks));
    const int tid = threadIdx.x, lane = tid & 31;
    const CacheSeq s = cache_seq(c, b);
    if (s.len <= keep)
        return;
    const int count = min(keep - j * kPage, kPage);
    const int to = table_page(new_pages, c, b, j);
    if (to < 0) {
        if (h == 0 && tid == 0)
            atomicOr(&c.hdr->flag, FLAG_CACHE_PAGE);
        return;
    }
    for (int u = tid; u < kPage; u += D) {
        int page = -1, slot = 0;
        if (u < count) {
            const int i = kept[(int64_t)b * keep + j * kPage + u];
            page = table_page(c.table, c, b, i / kPage);
            slot = i % kPage;
        }
        tok_page[u] = page;
        tok_slot[u] = slot;
        tok_ks[u] = page < 0 ? 0.f : c.k_scale[(int64_t)page * c.H + h];
        tok_vs[u] = page < 0 ? 0.f : c.v_scale[(int64_t)page * c.H + h];
        if (h == 0 && page >= 0) {
            const int64_t from = (int64_t)page * kPage + slot, at = (int64_t)to * kPage + u;
            c.timestamps[at] = c.timestamps[from];
            c.positions[at] = c.positions[from];
            c.weights[at] = c.weights[from];
        }
    }
    __syncthreads();
    // 16 codes each of four of the keys
    constexpr int PK = D / 16;  // pieces of a key
    uint4 kw[4];
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const int x = tid + i * D, u = x / PK, page = tok_page[u];
        kw[i] = page < 0 ? make_uint4(0u, 0u, 0u, 0u)
                         : *reinterpret_cast<const uint4 *>(c.k_codes + block_offset<D>(page, c.H, h) +
                                                            tok_slot[u] * D + x % PK * 16);
    }
    // values: runs of tokens of one source page (kept is ascending)
    uint64_t starts = 0;
    {
        const int u0 = lane, u1 = lane + 32;
        const uint32_t lo = __ballot_sync(0xffffffffu, u0 < count && (u0 == 0 || tok_page[u0] != tok_page[u0 - 1]));
        const uint32_t hi = __ballot_sync(0xffffffffu, u1 < count && tok_page[u1] != tok_page[u1 - 1]);
        starts = (uint64_t)hi << 32 | lo;
    }
    uint4 v[4];
    // the warp's 32 rows of a block: piece i of a lane is bytes [16 (lane % 4), + 16) of row 8 i + lane / 4
    const int warp_row = tid & ~31, my_row = lane >> 2, my_piece = lane & 3;
    auto fetch = [&](int u) {  // of token u's page
        const int page = tok_page[u];
        const uint8_t *p = c.v_codes + block_offset<D>(page < 0 ? 0 : page, c.H, h) + warp_row * kPage + 16 * lane;
#pragma unroll
        for (int i = 0; i < 4; i++)
            v[i] = page < 0 ? make_uint4(0u, 0u, 0u, 0u) : *reinterpret_cast<const uint4 *>(p + 512 * i);
    };
    uint32_t *srow = src + tid * LD, *drow = dst + tid * LD;
    const uint8_t *sbytes = reinterpret_cast<const uint8_t *>(srow);
    uint8_t *dbytes = reinterpret_cast<uint8_t *>(drow);
    uint32_t mk = 0, mv = 0;
#pragma unroll
    for (int i = 0; i < 16; i++)
        drow[i] = 0u;
    fetch(0);
    for (int u = 0; u < count;) {
        starts &= starts - 1;
        const int end = starts ? __ffsll((long long)starts) - 1 : count;
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 4; i++) {
            uint32_t *x = src + (warp_row + 8 * i + my_row) * LD + 4 * my_piece;
            x[0] = v[i].x, x[1] = v[i].y, x[2] = v[i].z, x[3] = v[i].w;
        }
        __syncwarp();
        if (end < count)
            fetch(end);
        __half2 top = __half2half2(__ushort_as_half(0));
        const float vs = tok_vs[u];
        while (u < end) {
            if ((u & 3) == 0 && u + 4 <= end) {
                const int4 sl = *reinterpret_cast<const int4 *>(&tok_slot[u]);
                const uint32_t lo = __byte_perm(sbytes[sl.x], sbytes[sl.y], 0x0040);
                const uint32_t hi = __byte_perm(sbytes[sl.z], sbytes[sl.w], 0x0040);
                const uint32_t x = __byte_perm(lo, hi, 0x5410);
                drow[u >> 2] = x;
                top = max_codes(top, x);
                u += 4;
            } else {
                const uint32_t x = sbytes[tok_slot[u]];
                dbytes[u++] = (uint8_t)x;
                top = max_codes(top, x);
            }
        }
        mv = max(mv, magnitude(top, vs));
    }
#pragma unroll
    for (int i = 0; i < 4; i++) {
        __half2 top = __half2half2(__ushort_as_half(0));
        top = max_codes(max_codes(max_codes(max_codes(top, kw[i].x), kw[i].y), kw[i].z), kw[i].w);
        mk = max(mk, magnitude(top, tok_ks[(tid + i * D) / PK]));
    }
    mk = __reduce_max_sync(0xffffffffu, mk);
    mv = __reduce_max_sync(0xffffffffu, mv);
    if (lane == 0) {
        smax[0][tid >> 5] = mk;
        smax[1][tid >> 5] = mv;
    }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < D / 32; w++) {
        mk = max(mk, smax[0][w]);
        mv = max(mv, smax[1][w]);
    }
    const float ks = block_scale(mk), vs = block_scale(mv);
    const float ki = scale_inverse(ks), vi = scale_inverse(vs);
    if (tid == 0) {
        c.k_scale[(int64_t)to * c.H + h] = ks;
        c.v_scale[(int64_t)to * c.H + h] = vs;
    }
    bool large = false;  // a ratio that f16 does not hold
    for (int u = tid; u < count; u += D) {
        const float rk = code_ratio(tok_ks[u], ki), rv = code_ratio(tok_vs[u], vi);
        large |= rk > 32768.f || rv > 32768.f;
        tok_rk[u] = __float2half_rn(rk);
        tok_rv[u] = __float2half_rn(rv);
    }
    large = __syncthreads_or(large);
    uint8_t *kc = c.k_codes + block_offset<D>(to, c.H, h);
    if (!large) {
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const int x = tid + i * D, u = x / PK;
            const __half2 r = __half2half2(tok_rk[u]);
            if (u < count)
                *reinterpret_cast<uint4 *>(kc + u * D + x % PK * 16) = make_uint4(
                    put4h(kw[i].x, r, r), put4h(kw[i].y, r, r), put4h(kw[i].z, r, r), put4h(kw[i].w, r, r));
        }
#pragma unroll
        for (int i = 0; i < 16; i++) {
            const uint2 r = *reinterpret_cast<const uint2 *>(&tok_rv[4 * i]);
            drow[i] = put4h(drow[i], *reinterpret_cast<const __half2 *>(&r.x), *reinterpret_cast<const __half2 *>(&r.y));
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const int x = tid + i * D, u = x / PK;
            const float r = code_ratio(tok_ks[u], ki);
            if (u < count)
                *reinterpret_cast<uint4 *>(kc + u * D + x % PK * 16) =
                    make_uint4(put4(kw[i].x, r, r, r, r), put4(kw[i].y, r, r, r, r), put4(kw[i].z, r, r, r, r),
                               put4(kw[i].w, r, r, r, r));
        }
#pragma unroll 1
        for (int i = 0; i < 16; i++) {
            const float4 r = *reinterpret_cast<const float4 *>(&tok_vs[4 * i]);
            drow[i] = put4(drow[i], code_ratio(r.x, vi), code_ratio(r.y, vi), code_ratio(r.z, vi), code_ratio(r.w, vi));
        }
    }
    __syncwarp();
    uint8_t *vc = c.v_codes + block_offset<D>(to, c.H, h) + warp_row * kPage + 16 * lane;
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const uint32_t *x = dst + (warp_row + 8 * i + my_row) * LD + 4 * my_piece;
        uint32_t w[4] = {x[0], x[1], x[2], x[3]};
        uint4 *g = reinterpret_cast<uint4 *>(vc + 512 * i);
        if (16 * my_piece + 16 > count) {  // slots behind the last token keep their bytes
            const uint4 was = *g;
            const uint32_t old[4] = {was.x, was.y, was.z, was.w};
#pragma unroll
            for (int e = 0; e < 4; e++) {
                const int n = count - 16 * my_piece - 4 * e;
                const uint32_t mask = n >= 4 ? 0xffffffffu : n <= 0 ? 0u : (1u << (8 * n)) - 1u;
                w[e] = (w[e] & mask) | (old[e] & ~mask);
            }
        }
        *g = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

template <int D>
void move(const CacheCall &c, int keep, int blocks, const int32_t *new_pages, const int32_t *kept, cudaStream_t stream)
{
    cache_move_kernel<D><<<(unsigned)((int64_t)c.B * blocks * c.H), D, 0, stream>>>(c, keep, blocks, new_pages,
                                                                                       kept);
}

}  // namespace

cudaError_t launch_cache_evict(const CacheCall &c, int keep, int first, int recent, const int32_t *new_pages,
                               int32_t *new_table, int32_t *new_lens, int32_t *kept, uint32_t *keys, int64_t cap,
                               cudaStream_t stream)
{
    if (c.B == 0)
        return cudaSuccess;
    // all keys in the registers of 256 threads, whose barriers are cheap, or of 1024
    if (c.max_cache_len <= 4 * kSelGroups * 256)
        cache_select_kernel<256><<<c.B, 256, 0, stream>>>(c, keep, first, recent, new_pages, new_table, new_lens, kept,
                                                          keys, cap);
    else
        cache_select_kernel<1024><<<c.B, 1024, 0, stream>>>(c, keep, first, recent, new_pages, new_table, new_lens,
                                                            kept, keys, cap);
    if (c.max_cache_len > keep && c.max_pages > 0) {
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
