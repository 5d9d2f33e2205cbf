// Host-side launchers shared between the kernel files and the C-ABI layer.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace hstu {

struct WsHeader;
struct AttnParams;

// A call on the 8-bit cache: the pool and its pages, the call's jagged tokens
// (none for the eviction: seq_offsets null) and the lengths behind the table.
struct CacheCall {
    uint8_t *k_codes, *v_codes;
    float *k_scale, *v_scale;
    int64_t *timestamps;
    int32_t *positions;
    float *weights;
    int num_pages, H, d, max_pages;
    int B, max_seq_len, max_cache_len;
    int64_t T;
    const int64_t *seq_offsets;
    const int32_t *num_targets;
    const int64_t *ts;  // [T] stamps of the call's tokens
    const int32_t *table, *cache_lens, *seq_pos;
    WsHeader *hdr;
};

// SM count and L2 size of the current device (cached per device).
struct DeviceInfo {
    int sms = 148;
    int64_t l2_bytes = 126 << 20;
};
DeviceInfo device_info();

// Tile rows of the work items each attention implementation consumes: 64 for
// the fp32 kernels (the work list is always sized for this, the finer tiling),
// 128 for the tcgen05 kernels.
constexpr int kF32Tile = 64;
constexpr int kTcTile = 128;

cudaError_t launch_schedule(const int64_t *off, const int32_t *nt, int B, int64_t T, int max_len,
                            int tile, int is_bwd, int2 *items, int capacity, WsHeader *hdr,
                            int32_t *count_out, cudaStream_t stream);

cudaError_t launch_debug_indices(const int64_t *off, const int64_t *ts, const int32_t *nt, int B,
                                 int lo, int hi, int nb, bool own, const int64_t *rows, int64_t n,
                                 int32_t *pos_out, int32_t *bkt_out, cudaStream_t stream);

// bf16 attention on tcgen05 / TMA (sm_100a), 128-row tiles, head dims 64 and 128.
// tensor_maps_available: the driver exposes cuTensorMapEncodeTiled (without it no
// tcgen05 kernel can run).  attn_tc_supported: the shape is one the kernels take.
bool tensor_maps_available();
bool attn_tc_supported(const AttnParams &p);
cudaError_t launch_attn_fwd_tc(const AttnParams &p, int grid_items, cudaStream_t stream);
// 2-D bf16 tensor map over [rows, cols] with a row stride, 64 x 128 boxes, 128B swizzle.
cudaError_t make_row_tensor_map(CUtensorMap *map, const void *base, int64_t rows, int cols,
                                int64_t row_stride_elems);
// General 2-D tensor map (row stride in bytes, box of box_cols x box_rows elements).
cudaError_t make_tensor_map_2d(CUtensorMap *map, const void *base, CUtensorMapDataType dtype,
                               int64_t rows, int64_t cols, int64_t row_stride_bytes, int box_cols,
                               int box_rows, CUtensorMapSwizzle swizzle);
// bf16 backward on tcgen05 (head dims 64, 128), key tiles of 128 rows; dq_acc
// receives dQ / (0.5 * inv_n) (apply that scale when converting).
cudaError_t launch_attn_bwd_tc(const AttnParams &p, int grid_items, cudaStream_t stream);

// fp32 attention on CUDA cores, 64-row tiles.
cudaError_t launch_attn_fwd_f32(const AttnParams &p, int grid_items, cudaStream_t stream);
cudaError_t launch_attn_bwd_f32(const AttnParams &p, int grid_items, cudaStream_t stream);

// dq (bf16, rows of stride sdq, 16-byte aligned) <- scale * dq_acc (fp32 [T, H d]).
cudaError_t launch_convert_dq(const float *acc, void *dq, int64_t T, int H, int d, int64_t sdq,
                              float scale, cudaStream_t stream);

// C[M, N] = act(A[M, K] B[K, N] + bias[N]) on tcgen05 / TMA (sm_100a); act =
// SiLU if silu.  Row strides lda, ldc in elements; B is dense [K, N]; K a
// multiple of 8, N of 32.  hdr receives a timeout flag if a pipeline wait ever
// gives up.  launch_gemm_f32 is the same in fp32 on CUDA cores.
bool gemm_tc_supported(const void *A, int64_t lda, const void *Bm, void *C, int64_t ldc, int64_t M, int N, int K);
cudaError_t launch_gemm_tc(const void *A, int64_t lda, const void *Bm, const void *bias, void *C, int64_t ldc,
                           int64_t M, int N, int K, bool silu, WsHeader *hdr, cudaStream_t stream);
cudaError_t launch_gemm_f32(const float *A, int64_t lda, const float *Bm, const float *bias,
                            float *C, int64_t ldc, int64_t M, int N, int K, bool silu,
                            cudaStream_t stream);

// General tcgen05 GEMM C[M, N] = epi(A B) (bf16 operands, fp32 accumulation).
//   A: a_mn = false -> A[m][k] at A + m*lda + k;  a_mn = true -> at A + k*lda + m
//   B: b_k = false  -> B[k][n] at B + k*ldb + n;  b_k = true  -> at B + n*ldb + k
//   GEMM_ACT:    C bf16 = acc + bias (optionally SiLU)
//   GEMM_DSILU:  C bf16 = aux * SiLU'(acc + bias), aux bf16 [M, N] (row stride ldaux)
//   GEMM_RED_F32: C32 fp32 += acc, the k range split over `splits` CTAs (C32 must
//                 hold its initial value, e.g. zeros); ldc in elements.
// A may be the column concatenation of three stored matrices with the same row
// count: a_seg > 0 (a multiple of 64) is the width of each, A, A1, A2 their
// bases and lda, lda1, lda2 their row strides.  The stored columns are K for a
// K-major A and M for an MN-major A, so the concatenation runs along K or M.
enum GemmEpilogue { GEMM_ACT = 0, GEMM_DSILU = 1, GEMM_RED_F32 = 2 };
struct GemmOperands {
    const void *A;
    int64_t lda;
    const void *A1, *A2;
    int64_t lda1, lda2;
    int a_seg;
    bool a_mn;
    const void *B;
    int64_t ldb;
    bool b_k;
    const void *bias;
    const void *aux;
    int64_t ldaux;
    void *C;
    float *C32;
    int64_t ldc;
};
bool gemm_tc_ok(const GemmOperands &op, int64_t M, int N, int K);
cudaError_t launch_gemm_tc_ex(const GemmOperands &op, int64_t M, int N, int K, GemmEpilogue epi, bool silu,
                              int splits, WsHeader *hdr, cudaStream_t stream);

// E4M3 GEMM on tcgen05 (kind::f8f6f4): C bf16 [M, N] = (A B^T) * sa[m] * sb[n]
// + bias[n], optionally SiLU.  A codes [M, K] (row stride lda bytes), B codes
// [N, K] (row stride ldb bytes), both K-major; sa [M], sb [N] float32.
bool gemm_e4m3_ok(const void *A, int64_t lda, const void *B, int64_t ldb, const void *C, int64_t ldc, int64_t M,
                  int N, int K);
cudaError_t launch_gemm_e4m3(const void *A, int64_t lda, const float *sa, const void *B, int64_t ldb,
                             const float *sb, const void *bias, void *C, int64_t ldc, int64_t M, int N, int K,
                             bool silu, WsHeader *hdr, cudaStream_t stream);
// Per-row E4M3 quantisation of a bf16 [R, K] matrix (row stride ldx elements):
// codes [R, K] (row stride ldq bytes) and scales [R]; K a multiple of 8.
cudaError_t launch_quantize_rows_e4m3(const void *x, int64_t ldx, int64_t R, int K, void *q, int64_t ldq,
                                      float *scale, cudaStream_t stream);
// Per-column E4M3 quantisation of a bf16 weight [K, N]: codes [N, K] (the
// transpose) and scales [N].
cudaError_t launch_quantize_cols_e4m3(const void *w, int64_t K, int N, void *q, float *scale, cudaStream_t stream);

// G[t, :] = LayerNorm(O[t, :]) * U[t, :] over F features.
cudaError_t launch_norm_gate(bool bf16, const void *O, int64_t ldo, const void *U, int64_t ldu,
                             const float *gamma, const float *beta, float eps, void *G,
                             int64_t ldg, int64_t T, int F, cudaStream_t stream);

// Backward of G = LayerNorm(O) * U (bf16): writes dO and dU (row strides in
// elements) and adds the parameter gradients to dgamma, dbeta (fp32 [F]).
cudaError_t launch_norm_gate_bwd(const void *dG, int64_t ldd, const void *O, int64_t ldo, const void *U,
                                 int64_t ldu, const float *gamma, const float *beta, float eps, void *dO,
                                 int64_t lddo, void *dU, int64_t lddu, float *dgamma, float *dbeta, int64_t T,
                                 int F, bool cat, cudaStream_t stream);
// cat: dG is the last F-wide block of rows [dU' | dO' | dG] whose first two
// blocks (direct gradients through an output projection over [U | O | G]) are
// added to dU and dO.
// out[t, :] = [a[t, :] | b[t, :] | c[t, :]], each block `bytes` wide (a multiple
// of 4); row strides lda, ldb, ldc in bytes.
cudaError_t launch_concat3(const void *a, int64_t lda, const void *b, int64_t ldb, const void *c, int64_t ldc,
                           void *out, int64_t T, int64_t bytes, cudaStream_t stream);
// out[n] += sum over T rows of A[row, n] (bf16 A, fp32 out).
cudaError_t launch_colsum_bf16(const void *A, int64_t lda, int64_t T, int N, float *out, cudaStream_t stream);

// Attention truncation (at most kTruncateMaxSeqs sequences: the new offsets
// live in shared memory): out_off [B+1] = offsets of every sequence's last
// min(hist, keep) history tokens plus its candidates; out = those rows of in
// (row_bytes a multiple of 4; 16-byte copies when it is a multiple of 16).
constexpr int kTruncateMaxSeqs = 12288;
cudaError_t launch_jagged_truncate(const int64_t *off, const int32_t *nt, int B, int64_t T, int keep,
                                   int64_t row_bytes, const void *in, void *out, int64_t *out_off,
                                   cudaStream_t stream);

// 8-bit cache: an append or attention of no sequences checks its offsets all the same.
cudaError_t launch_cache_no_sequences(const CacheCall &c, cudaStream_t stream);

// 8-bit cache: append of new tokens (k, v rows ldk, ldv elements apart).
int cache_append_blocks(int max_seq_len);
cudaError_t launch_cache_append(const CacheCall &c, bool bf16, const void *k, int64_t ldk, const void *v, int64_t ldv,
                                int32_t *new_lens, int32_t *new_pos, cudaStream_t stream);

// 8-bit cache: eviction.  kept [B, keep] receives the old indices (then -1);
// keys [B, cap] is scratch.
cudaError_t launch_cache_evict(const CacheCall &c, int keep, int first, int recent, const int32_t *new_pages,
                               int32_t *new_table, int32_t *new_lens, int32_t *kept, uint32_t *keys, int64_t cap,
                               cudaStream_t stream);

// 8-bit cache: attention over the cache.  Three kernels: float32 on CUDA cores, bf16
// of up to kCacheRows query rows a sequence, bf16 of more (tensor cores).  The first
// two cut the key axis into `nsplit` parts of `split_pages` pages, whose sums go to
// part_o [nsplit, T, H, d] (float32); the third cuts all its tiles into `ctas` runs,
// with two slots [128, d] of part_o and two piece records each.  Where weights are
// taken, those of plane_rows queries and one head go to a plane of part_w [planes, B, lcap].  A second
// kernel joins them in a fixed order.
// At 64 rows both sides win somewhere (d = 128, 4 heads, few rows' kernel / tensor cores): one
// user's 2,048 cached tokens 14 / 23-31 us (candidates - history), 16,384 tokens 47 / 37-48;
// 32 users' 1,024 tokens 71 / 25-46, 8,192 tokens 332 / 83-180.  At 8 rows the first one wins
// (11 / 23, 18 / 35-38, 19 / 23-29) but for the longest batch's candidates (81 / 78-99).
constexpr int kCacheRows = 64;
enum CacheKernel { CACHE_F32, CACHE_ROWS, CACHE_TC };
struct CacheAttnPlan {
    CacheKernel kernel;
    int nsplit, split_pages;
    int ctas;
    int qtiles;      // query tiles of a sequence (16 rows; 128 on the tensor cores)
    int plane_rows;  // query rows of a plane (16; 64 on the tensor cores)
    int64_t lcap;
    size_t part_o_bytes, part_w_bytes, piece_bytes;
};
struct CacheAttnPiece {
    int64_t row;  // first row of the unit's queries
    int head, cols, last;
};
struct CacheAttnArgs {
    CacheCall c;
    CacheAttnPlan plan;
    const void *q;
    int64_t ldq;
    const float *rab_pos, *rab_time;
    int64_t pos_hstride, time_hstride;
    int pos_lo, pos_hi, nb, cand_own;
    float inv_n;
    const void *addend;
    void *out;
    float *weights_out;
    float *part_o, *part_w;
    CacheAttnPiece *pieces;
    // cycles after which a wait of the bf16 kernels gives up, and its test hook: one
    // CTA's first block of keys is never loaded
    long long wait_limit;
    int withhold;
};
CacheAttnPlan cache_attn_plan(const CacheCall &c, bool bf16, bool with_weights);
bool cache_attn_fits(const CacheAttnArgs &a);  // its launches and coordinates stay below their limits
cudaError_t launch_cache_attn(const CacheAttnArgs &a, bool bf16, cudaStream_t stream);
cudaError_t launch_cache_attn_rows(const CacheAttnArgs &a, cudaStream_t stream);
cudaError_t launch_cache_attn_tc(const CacheAttnArgs &a, cudaStream_t stream);

}  // namespace hstu
