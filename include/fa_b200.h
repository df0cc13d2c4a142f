/*
 * fa_b200.h - C ABI of the B200 (sm_100a) exact-attention library libfa_b200.so.
 *
 * Exact scaled-dot-product attention O = softmax(scale * Q K^T [+ causal mask]) V,
 * computed tile by tile with an online softmax so that the N x N score matrix
 * never reaches device memory ("DL101 chapter 9", handsonai.io, section 3.3
 * FlashAttention; "Flash Attention: principle & practice", holysheep.ai,
 * sections 2.1 Online Softmax and 2.2 Tiling).
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 *  - Tensors are contiguous, row-major, in device memory, and 16-byte aligned.
 *    "bf16" arguments are void pointers to IEEE bfloat16 bit patterns.
 *  - Q, K, V, O, dO, dQ, dK, dV are [B, H, N, d] (batch, head, sequence, head
 *    dimension; the multi-head layout of "DL101 chapter 9", section 3).
 *    LSE and D are [B, H, N] float32.  The ragged-batch entry points
 *    (_varlen) take sequences packed token-major, [total, heads, d], and the
 *    paged decode takes page pools; each states its layout.
 *  - Supported head dimensions: d = 64 and d = 128 (fa_fwd_fp8: 128).  Any
 *    N >= 0 (ragged tails are masked inside the kernels).
 *  - Key / value tensors may have fewer heads than queries (Hkv dividing H;
 *    the _gqa, _ext, _varlen, _paged and _fp8 entry points): query head h
 *    attends key / value head h / (H / Hkv) ("DL101 chapter 9", sections 3.1
 *    MQA and 3.2 GQA).
 *  - scale multiplies Q K^T before the softmax; callers normally pass
 *    1/sqrt(d) ("DL101 chapter 9", section 1.1).
 *  - Causal masking keeps key j for query i iff j <= i + Nk - Nq (diagonal
 *    included; with Nq = Nk = N simply j <= i).  With Nq != Nk (the _ext
 *    entry points) the Nq queries are the last Nq positions of the Nk-token
 *    sequence, i.e. a chunk of new tokens over a cache ("DL101 chapter 9",
 *    section 1.1: token t attends K_{<=t}).  A query that sees no key
 *    (only when Nq > Nk) gets O = 0 and LSE = -inf.
 *  - LSE is the natural-log log-sum-exp of the row's scaled, masked scores:
 *    LSE_i = ln sum_j exp(scale * q_i . k_j).
 *  - The caller allocates and owns every buffer, workspaces included.  The
 *    library allocates no device memory; it keeps only per-process state
 *    (a driver entry point, device properties and a device error word).
 *  - All calls are asynchronous and ordered on `stream` (a cudaStream_t; NULL
 *    is the legacy default stream).  Argument errors are reported before any
 *    launch and leave the outputs untouched.  A failed launch returns
 *    FA_ERR_CUDA.  A kernel whose bounded wait expired records FA_ERR_TIMEOUT
 *    in the device error word (read it with fa_get_device_error); kernels
 *    never trap.
 *  - The current CUDA device must be the one that holds the buffers.
 *  - No C++ exception crosses this interface.
 */
#ifndef FA_B200_H
#define FA_B200_H

#include <stddef.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st* fa_stream_t; /* same type as cudaStream_t */
typedef struct CUevent_st* fa_event_t;   /* same type as cudaEvent_t  */

typedef enum {
    FA_OK = 0,
    FA_ERR_INVALID_ARG = 1,  /* null pointer, bad size, misaligned pointer      */
    FA_ERR_UNSUPPORTED = 2,  /* head dimension other than 64 / 128, no sm_100   */
    FA_ERR_WORKSPACE = 3,    /* workspace missing or smaller than required      */
    FA_ERR_CUDA = 4,         /* a CUDA runtime / driver call failed             */
    FA_ERR_TIMEOUT = 5,      /* a kernel's bounded wait expired (device word)   */
    FA_ERR_BOUNDS = 6        /* debug build only: a kernel's bounds check failed
                                and the access was skipped (device word)        */
} fa_status;

/*
 * Forward pass.  "DL101 chapter 9", section 3.3 (tiled FlashAttention:
 * running max m and sum l, O <- O*c + P V, final O / l) and "Flash Attention:
 * principle & practice", section 2.1 (online softmax).
 *   q, k, v : bf16 [B, H, N, d], read only.
 *   o       : bf16 [B, H, N, d], written.
 *   lse     : float32 [B, H, N], written; may be NULL when not needed.
 *   causal  : 0 or 1.
 * Returns FA_OK, FA_ERR_INVALID_ARG, FA_ERR_UNSUPPORTED or FA_ERR_CUDA.
 */
fa_status fa_fwd(const void* q, const void* k, const void* v, void* o, float* lse,
                 int B, int H, int N, int d, int causal, float scale,
                 fa_stream_t stream);

/*
 * Grouped-query forward ("DL101 chapter 9", sections 3.1 MQA and 3.2 GQA):
 * k and v are bf16 [B, Hkv, N, d] and query head h of batch b attends key /
 * value head h / (H / Hkv) of that batch.  Hkv must divide H; Hkv = H is
 * fa_fwd, Hkv = 1 multi-query attention.  Everything else as fa_fwd.
 */
fa_status fa_fwd_gqa(const void* q, const void* k, const void* v, void* o, float* lse,
                     int B, int H, int Hkv, int N, int d, int causal, float scale,
                     fa_stream_t stream);

/*
 * Forward with separate query and key lengths, grouped heads allowed (the
 * non-square Lq x Lk problem of "DL101 chapter 9", section 3.3):
 *   q       : bf16 [B, H, Nq, d], read only.
 *   k, v    : bf16 [B, Hkv, Nk, d], read only.
 *   o       : bf16 [B, H, Nq, d], written.
 *   lse     : float32 [B, H, Nq], written; may be NULL.
 * Nq, Nk >= 0 with Nq + Nk < 2^31.  Causal masking is bottom-right aligned
 * (see the conventions above).  Nk = 0 writes O = 0 and LSE = -inf.
 * Pointers to arrays of zero size may be NULL.
 * fa_fwd_gqa(..., N, ...) is fa_fwd_ext(..., N, N, ...).  Returns as fa_fwd.
 */
fa_status fa_fwd_ext(const void* q, const void* k, const void* v, void* o, float* lse,
                     int B, int H, int Hkv, int Nq, int Nk, int d, int causal, float scale,
                     fa_stream_t stream);

/*
 * Forward over a ragged batch: B sequences of different lengths packed
 * without padding (each sequence is the attention problem of its own rows;
 * "DL101 chapter 9", section 3.3 for Lq x Lk).
 *   q            : bf16 [total_q, H, d], token-major: the rows of sequence b
 *                  are cu_seqlens_q[b] .. cu_seqlens_q[b+1]-1; read only.
 *   k, v         : bf16 [total_k, Hkv, d], likewise with cu_seqlens_k.
 *   o            : bf16 [total_q, H, d], written.
 *   lse          : float32 [H, total_q], written; may be NULL.
 *   cu_seqlens_q,
 *   cu_seqlens_k : int32 [B + 1] in DEVICE memory: 0, then the running sums
 *                  of the lengths, ending at total_q / total_k.  A sequence
 *                  whose range leaves the packed array is treated as empty.
 *   max_seqlen_q : host upper bound of the query lengths (sizes the launch).
 *                  A longer sequence records FA_ERR_INVALID_ARG in the device
 *                  error word and its rows past max_seqlen_q are not written.
 * Causal masking is bottom-right aligned per sequence (query i of a sequence
 * keeps key j iff j <= i + Lk_b - Lq_b).  A sequence with no keys gets O = 0,
 * LSE = -inf.  Pointers to empty arrays may be NULL.  Returns as fa_fwd.
 */
fa_status fa_fwd_varlen(const void* q, const void* k, const void* v, void* o, float* lse,
                        const int* cu_seqlens_q, const int* cu_seqlens_k,
                        int B, int H, int Hkv, int total_q, int total_k, int max_seqlen_q,
                        int d, int causal, float scale, fa_stream_t stream);

/*
 * Forward with 8-bit float inputs (e4m3, OCP FP8): the FP8 path the pages
 * mention for FlashAttention-3 ("Flash Attention La Gi?", FlashAttention-3).
 * The pages give no scaling convention; here each input tensor carries one
 * descale factor (real value = stored e4m3 value x factor), the products run
 * on the tensor core's 8-bit path with f32 accumulation, and the softmax
 * probabilities are rounded to e4m3 before the P V product (relative error
 * up to 2^-4 per probability, so O carries a few percent relative error).
 *   q       : e4m3 [B, H, Nq, 128] (bytes), read only.
 *   k       : e4m3 [B, Hkv, Nk, 128], read only.
 *   vt      : e4m3 [B, Hkv, 128, Nk]: V transposed (row r holds component r
 *             of every value), read only.  Nk must be a multiple of 16.
 *   q_scale, k_scale, v_scale : the descale factors.
 *   o       : bf16 [B, H, Nq, 128], written (real, descaled values).
 *   lse     : float32 [B, H, Nq], written; may be NULL.
 *   d       : must be 128.
 * Masking, grouping, scale and errors as fa_fwd_ext; FA_ERR_UNSUPPORTED for
 * d != 128 or Nk not a multiple of 16.
 */
fa_status fa_fwd_fp8(const void* q, const void* k, const void* vt, void* o, float* lse,
                     float q_scale, float k_scale, float v_scale,
                     int B, int H, int Hkv, int Nq, int Nk, int d, int causal, float scale,
                     fa_stream_t stream);

/*
 * Bytes of device workspace fa_bwd needs: D = rowsum(dO * O) and
 * log2(e) * LSE as float32 [B, H, Np] with Np = N rounded up to a multiple
 * of 128, the float32 dQ accumulator [B, H, N, d] and one uint32
 * completion counter per (b, h), each region 256-byte aligned.  Returns 0
 * for invalid sizes.
 */
size_t fa_bwd_workspace_size(int B, int H, int N, int d);

/*
 * Backward pass with recomputation ("Flash Attention La Gi?", thienlv.com,
 * Recomputation: scores are recomputed from Q, K, V and the saved LSE
 * instead of being stored).  Gradients of sum(O * dO):
 *   dV = P^T dO, dP = dO V^T, D = rowsum(dO * O), dS = P * (dP - D),
 *   dQ = scale dS K, dK = scale dS^T Q.
 *   q, k, v, o, dout : bf16 [B, H, N, d], read only (o and lse from fa_fwd).
 *   lse              : float32 [B, H, N], read only.
 *   dq, dk, dv       : bf16 [B, H, N, d], written.
 *   workspace        : device buffer of at least fa_bwd_workspace_size bytes,
 *                      256-byte aligned, owned by the caller; contents on
 *                      entry are ignored, on exit unspecified.
 * Returns FA_OK, FA_ERR_INVALID_ARG, FA_ERR_UNSUPPORTED, FA_ERR_WORKSPACE or
 * FA_ERR_CUDA.
 */
fa_status fa_bwd(const void* q, const void* k, const void* v, const void* o,
                 const void* dout, const float* lse, void* dq, void* dk, void* dv,
                 void* workspace, size_t ws_bytes,
                 int B, int H, int N, int d, int causal, float scale,
                 fa_stream_t stream);

/*
 * Grouped-query backward: k, v, dk, dv are [B, Hkv, N, d]; the gradient of a
 * shared key / value head is the sum over its H / Hkv query heads.  The
 * workspace is fa_bwd_workspace_size(B, H, N, d).  Everything else as fa_bwd.
 */
fa_status fa_bwd_gqa(const void* q, const void* k, const void* v, const void* o,
                     const void* dout, const float* lse, void* dq, void* dk, void* dv,
                     void* workspace, size_t ws_bytes,
                     int B, int H, int Hkv, int N, int d, int causal, float scale,
                     fa_stream_t stream);

/*
 * Backward with separate query and key lengths (the inverse of fa_fwd_ext):
 *   q, o, dout : bf16 [B, H, Nq, d], read only;  lse : float32 [B, H, Nq].
 *   k, v       : bf16 [B, Hkv, Nk, d], read only.
 *   dq         : bf16 [B, H, Nq, d], written.
 *   dk, dv     : bf16 [B, Hkv, Nk, d], written.
 *   workspace  : fa_bwd_workspace_size(B, H, Nq, d) bytes (not needed when
 *                Nq or Nk is 0).
 * Queries with LSE = -inf (they saw no key) contribute nothing.  Nq = 0
 * writes dK = dV = 0; Nk = 0 writes dQ = 0.  Pointers to arrays of zero size
 * may be NULL.  Returns as fa_bwd.
 */
fa_status fa_bwd_ext(const void* q, const void* k, const void* v, const void* o,
                     const void* dout, const float* lse, void* dq, void* dk, void* dv,
                     void* workspace, size_t ws_bytes,
                     int B, int H, int Hkv, int Nq, int Nk, int d, int causal, float scale,
                     fa_stream_t stream);

/*
 * Bytes of device workspace fa_bwd_varlen needs: D and log2(e) * LSE as
 * float32 [H, P] (every sequence's rows in their own padded segment, P about
 * total_q + 132 B), then the float32 dQ accumulator [total_q, H, d], each
 * region 256-byte aligned.  Returns 0 for invalid sizes.
 */
size_t fa_bwd_varlen_workspace_size(int B, int H, int total_q, int d);

/*
 * Backward over a ragged batch (the inverse of fa_fwd_varlen; recomputation
 * as fa_bwd):
 *   q, o, dout   : bf16 [total_q, H, d] token-major, read only.
 *   lse          : float32 [H, total_q] from fa_fwd_varlen, read only.
 *   k, v         : bf16 [total_k, Hkv, d], read only.
 *   dq           : bf16 [total_q, H, d], written.
 *   dk, dv       : bf16 [total_k, Hkv, d], written (zero for keys that no
 *                  query sees and for rows outside every sequence).
 *   cu_seqlens_q,
 *   cu_seqlens_k : int32 [B + 1] in device memory, as fa_fwd_varlen.
 *   max_seqlen_k : host upper bound of the key lengths (sizes the launch).
 *   workspace    : fa_bwd_varlen_workspace_size(B, H, total_q, d) bytes,
 *                  256-byte aligned, owned by the caller.
 * Returns FA_OK, FA_ERR_INVALID_ARG, FA_ERR_UNSUPPORTED, FA_ERR_WORKSPACE or
 * FA_ERR_CUDA.
 */
fa_status fa_bwd_varlen(const void* q, const void* k, const void* v, const void* o,
                        const void* dout, const float* lse, void* dq, void* dk, void* dv,
                        const int* cu_seqlens_q, const int* cu_seqlens_k,
                        void* workspace, size_t ws_bytes,
                        int B, int H, int Hkv, int total_q, int total_k, int max_seqlen_k,
                        int d, int causal, float scale, fa_stream_t stream);

/*
 * Bytes of device workspace fa_decode needs for the split-KV partials
 * (per batch, head and split: running max, running sum and an unnormalised
 * d-vector, float32) for caches of capacity Lmax.  Returns 0 for invalid
 * sizes.
 */
size_t fa_decode_workspace_size(int B, int H, int Lmax, int d);

/*
 * KV-cache decode: one new query per (batch, head) attends the cached keys
 * and values at positions 0 .. seqlens[b]-1 ("DL101 chapter 9", section 1.1
 * Key/Value Caching), split over chunks of the cache whose partial softmax
 * states are merged afterwards with the rescale-and-add rule of "Flash
 * Attention: principle & practice", section 2.1.
 *   q       : bf16 [B, H, d], read only.
 *   kcache,
 *   vcache  : bf16 [B, H, Lmax, d], read only; rows at or beyond seqlens[b]
 *             are never read.
 *   seqlens : int32 [B] in DEVICE memory, 0 <= seqlens[b] <= Lmax (values
 *             outside are clamped to that range).
 *   o       : bf16 [B, H, d], written (zeros where seqlens[b] == 0).
 *   lse     : float32 [B, H], written (-inf where seqlens[b] == 0); may be NULL.
 *   workspace : at least fa_decode_workspace_size(B, H, Lmax, d) bytes,
 *             256-byte aligned, owned by the caller.
 * Returns FA_OK, FA_ERR_INVALID_ARG, FA_ERR_UNSUPPORTED, FA_ERR_WORKSPACE or
 * FA_ERR_CUDA.
 */
fa_status fa_decode(const void* q, const void* kcache, const void* vcache,
                    const int* seqlens, void* o, float* lse,
                    int B, int H, int Lmax, int d, float scale,
                    void* workspace, size_t ws_bytes, fa_stream_t stream);

/*
 * Grouped-query decode: kcache and vcache are [B, Hkv, Lmax, d] and query
 * head h reads cache head h / (H / Hkv).  The workspace is
 * fa_decode_workspace_size(B, H, Lmax, d).  Everything else as fa_decode.
 */
fa_status fa_decode_gqa(const void* q, const void* kcache, const void* vcache,
                        const int* seqlens, void* o, float* lse,
                        int B, int H, int Hkv, int Lmax, int d, float scale,
                        void* workspace, size_t ws_bytes, fa_stream_t stream);

/*
 * Decode over a paged KV cache.  The pages name PagedAttention without
 * describing it; this is the addressing it implies: the cache of every
 * sequence is a list of fixed-size pages drawn from one pool, so sequences
 * grow without reserving Lmax rows each.  The arithmetic is fa_decode's
 * ("DL101 chapter 9", section 1.1; split-KV merge of "Flash Attention:
 * principle & practice", section 2.1).
 *   kpages,
 *   vpages      : bf16 [num_pages, Hkv, page_size, d], read only; row r of
 *                 head h of pool page p holds the key / value of one position.
 *   block_table : int32 [B, pages_per_seq] in DEVICE memory: position j of
 *                 sequence b lives in row j % page_size of pool page
 *                 block_table[b][j / page_size].  Entries past a sequence's
 *                 last page are never read.  An entry outside
 *                 [0, num_pages) is never dereferenced: its positions count
 *                 as masked and FA_ERR_INVALID_ARG is recorded in the device
 *                 error word (read it with fa_get_device_error).
 *   seqlens     : int32 [B], device; clamped to [0, pages_per_seq * page_size].
 *   page_size   : a power of two from 1 to 65536.
 *   workspace   : fa_decode_workspace_size(B, H, pages_per_seq * page_size, d).
 * q, o, lse, scale and the grouping Hkv as fa_decode_gqa.  Returns
 * FA_OK, FA_ERR_INVALID_ARG, FA_ERR_UNSUPPORTED, FA_ERR_WORKSPACE or
 * FA_ERR_CUDA.
 */
fa_status fa_decode_paged(const void* q, const void* kpages, const void* vpages,
                          const int* block_table, const int* seqlens, void* o, float* lse,
                          int B, int H, int Hkv, int page_size, int pages_per_seq,
                          int num_pages, int d, float scale,
                          void* workspace, size_t ws_bytes, fa_stream_t stream);

/*
 * Size in bytes of the device array that fa_decode_static uses as scratch
 * (16 MiB, held by every device that loads the library until exit).
 */
#define FA_DECODE_STATIC_SCRATCH_BYTES (16u * 1024u * 1024u)

/*
 * fa_decode without a caller-provided workspace, for callers that cannot
 * call cudaMalloc (a plug-in whose host program owns nearly all device memory
 * through its own pool, or a latency-critical loop that must not trigger the
 * device-wide synchronisation an allocation can cause).  The pages have no
 * counterpart: this is an interface convenience, not part of the method.
 *   Arguments, layouts, ownership and results are those of fa_decode, minus
 *   workspace / ws_bytes.  The split-KV partials go to a library-owned device
 *   array of FA_DECODE_STATIC_SCRATCH_BYTES bytes; a problem whose
 *   fa_decode_workspace_size(B, H, Lmax, d) exceeds that returns
 *   FA_ERR_WORKSPACE before any launch.  Allocates nothing.
 *   The first call on a device looks up the array's device address (with
 *   that device current); make it before any stream capture.  All calls
 *   share the array: calls that overlap on the GPU race and must be
 *   serialised by the caller.
 * Returns FA_OK, FA_ERR_INVALID_ARG, FA_ERR_UNSUPPORTED, FA_ERR_WORKSPACE or
 * FA_ERR_CUDA.
 */
fa_status fa_decode_static(const void* q, const void* kcache, const void* vcache,
                           const int* seqlens, void* o, float* lse,
                           int B, int H, int Lmax, int d, float scale,
                           fa_stream_t stream);

/*
 * Norm of queries and keys per head with the position rotation in the same
 * pass, in front of the attention.  The pages stop at Q, K and V; the formulas
 * are the library's own statement of the two operations.  For a row x of d
 * values (one token, one head) with weight w:
 *   r = 1 / sqrt(mean(x^2) + eps),  y = x r w   (weight NULL: y = x, no norm),
 * then the first rotary_dim values of y are rotated in pairs, the pair being
 * (i, i + rotary_dim / 2), or (2i, 2i + 1) with interleaved = 1, by the angle
 * a = position * inv_freq[i]:
 *   out_1 = y_1 cos a - y_2 sin a,   out_2 = y_2 cos a + y_1 sin a.
 * The angle is the product in 64 bits, reduced there; norms and products are
 * in 32 bits; only the outputs are rounded to bf16.
 *   q, k      : bf16, one row of d values per (batch, head, token), read only.
 *   q_out, k_out : the same shapes, written.  Each may be the input itself
 *               (same pointer, same strides); any other overlap is an error
 *               that is not detected.
 *   strides   : HOST array [4][3]: element strides {batch, head, token} of q, k,
 *               q_out and k_out; the d values of a row are contiguous.
 *               Strides are multiples of 8 and rows 16-byte aligned.  Packed
 *               token-major tensors [T, H, d] are B = 1, N = T.  Inputs may
 *               repeat rows (stride 0), outputs may not.
 *   q_weight, k_weight : [d] bf16 or float32 (weight_type), or NULL.
 *   positions : int32, token n of batch b at b * pos_batch_stride + n (stride
 *               0: the same positions for every batch), on the device.
 *   inv_freq  : float32 [rotary_dim / 2], on the device.  One that is infinite
 *               or NaN makes its pair NaN at every position.
 *   rotary_dim: 0 to d, a multiple of 16 (0: no rotation; positions and
 *               inv_freq may then be NULL).
 *   H, Hkv    : heads of q and of k; one of them may be 0.
 *   eps       : >= 0.
 * Any B, N >= 0 with B * N < 2^31 - 65536.  Returns FA_OK, FA_ERR_INVALID_ARG,
 * FA_ERR_UNSUPPORTED (d, rotary_dim % 16, no sm_100) or FA_ERR_CUDA.
 */
enum {
    FA_WEIGHT_BF16 = 0,
    FA_WEIGHT_F32 = 1
};
fa_status fa_qk_norm_rope(const void* q, const void* k, const void* q_weight,
                          const void* k_weight, int weight_type, const int* positions,
                          long long pos_batch_stride, const float* inv_freq,
                          void* q_out, void* k_out, const long long* strides,
                          int B, int H, int Hkv, int N, int d, int rotary_dim,
                          int interleaved, float eps, fa_stream_t stream);

/*
 * Its gradient.  From the inputs and g = dL/d out:
 *   dy = the rotation of g by -a,  c = mean(w dy x r),
 *   dx = r (w dy - x r c),         dw = sum over all rows of dy x r.
 *   q, k      : the forward's inputs; not read (may be NULL) where the weight
 *               is NULL.
 *   dq_out, dk_out : bf16, gradients of the outputs, read only.
 *   dq, dk    : bf16, written.
 *   dq_weight, dk_weight : float32 [d], written (zeros when there are no rows);
 *               not touched (may be NULL) where the weight is NULL.
 *   strides   : HOST array [6][3] of q, k, dq_out, dk_out, dq and dk.
 *   workspace : fa_qk_norm_rope_bwd_workspace_size(d) bytes, 256-byte aligned;
 *               not needed without weights.
 * The weight gradients are summed in a fixed order: equal calls give equal
 * bits.  Other arguments and returns as fa_qk_norm_rope, and FA_ERR_WORKSPACE.
 */
size_t fa_qk_norm_rope_bwd_workspace_size(int d);
fa_status fa_qk_norm_rope_bwd(const void* q, const void* k, const void* dq_out,
                              const void* dk_out, const void* q_weight,
                              const void* k_weight, int weight_type, const int* positions,
                              long long pos_batch_stride, const float* inv_freq,
                              void* dq, void* dk, float* dq_weight, float* dk_weight,
                              const long long* strides, int B, int H, int Hkv, int N,
                              int d, int rotary_dim, int interleaved, float eps,
                              void* workspace, size_t ws_bytes, fa_stream_t stream);

/*
 * The serving form: T new tokens, packed token-major.  Queries are normed and
 * rotated into q_out; keys are normed and rotated, values copied, into the
 * pages that fa_decode_paged reads.
 *   q, k, v   : bf16 [T, H, d], [T, Hkv, d], [T, Hkv, d].
 *   strides   : HOST array [4][3] of q, k, v and q_out (batch stride unused).
 *   positions : int32 [T], rotary position of each token.
 *   cache_positions : int32 [T], place of each token in its sequence's cache;
 *               NULL: positions.  A negative place marks a padded token:
 *               nothing of it is written, q_out included.
 *   batch_idx : int32 [T], block-table row of each token; NULL: token t
 *               belongs to row t (then T <= B).
 *   kpages, vpages : bf16 [num_pages, Hkv, page_size, d], written at the
 *               tokens' rows and nowhere else.
 *   block_table : int32 [B, pages_per_seq], row stride table_stride >=
 *               pages_per_seq.  A token whose row, place or page entry is out
 *               of range is not stored and FA_ERR_INVALID_ARG is recorded in
 *               the device error word; its query is still written.
 * Two tokens of one call with the same place leave a mixture of their rows.
 * Hkv >= 1; page_size a power of two from 1 to 65536.  Everything else as
 * fa_qk_norm_rope.
 */
fa_status fa_append_paged(const void* q, const void* k, const void* v,
                          const void* q_weight, const void* k_weight, int weight_type,
                          const int* positions, const int* cache_positions,
                          const int* batch_idx, const float* inv_freq, void* q_out,
                          void* kpages, void* vpages, const int* block_table,
                          const long long* strides, int T, int H, int Hkv, int d, int rotary_dim, int interleaved,
                          float eps, int B, int page_size, int pages_per_seq,
                          long long table_stride, int num_pages, fa_stream_t stream);

/*
 * Pages of a KV cache: who holds which page of the pools, kept on the device so
 * that a captured loop can run it.
 *   refs        : int32 [num_pages], how many sequences hold each page (0: free).
 *   block_table : int32 [B, pages_per_seq], row stride table_stride >=
 *                 pages_per_seq: the pages of each sequence first, -1 behind them.
 *   seqlens     : int32 [B], tokens of each sequence.
 *   pools       : HOST array of n_pools device pointers, page_bytes a HOST array:
 *                 pool i is [num_pages] pages of page_bytes[i] bytes (a multiple
 *                 of 16), one after another; both arrays are read before the call
 *                 returns.  A cache has two pools per layer, all under one table.
 *                 Pools must not overlap.
 * refs and block_table have to agree: refs[p] is the number of rows that list p.
 * Pages are taken lowest index first, items of a call in their order, so equal
 * states give equal results.  The tables of one cache are changed by one call at
 * a time (calls on one stream).  Workspaces are
 * fa_pages_workspace_size(num_pages, n) bytes, 256-byte aligned, with n the
 * items of the call (0 for fa_pages_compact).
 * Returns FA_OK, FA_ERR_INVALID_ARG, FA_ERR_UNSUPPORTED (no sm_100),
 * FA_ERR_WORKSPACE or FA_ERR_CUDA; item errors, found on the device, leave the
 * item undone and record FA_ERR_INVALID_ARG in the device error word.
 */
size_t fa_pages_workspace_size(int num_pages, int n);

/* Copies page src[i] onto page dst[i] in every pool, i < n (int32, device).  A
 * destination may be named once and be no source; a pair with a negative index
 * is left out, one past the pool is reported. */
fa_status fa_pages_copy(void* const* pools, const size_t* page_bytes, int n_pools,
                        int num_pages, const int* src, const int* dst, int n,
                        fa_stream_t stream);

/* Lets row seq_ids[i] hold the pages of new_lens[i] tokens (int32, device):
 * takes those it lacks from the free pages, and none if it holds enough.
 * granted[i] = 1, or 0 where the free pages left by the items before it do not
 * suffice (they count as taken even if not granted: no later item overtakes).
 * A length below 0 counts as 0.
 * An unknown row, a row given twice, or more pages than the table is wide is
 * an item error.  seqlens is the caller's to set. */
fa_status fa_pages_reserve(int* block_table, long long table_stride, int* refs,
                           const int* seq_ids, const int* new_lens, int* granted,
                           int B, int pages_per_seq, int num_pages, int page_size, int n,
                           void* workspace, size_t ws_bytes, fa_stream_t stream);

/* Makes row dst[i] a copy of row src[i] (int32, device): the full pages are
 * shared (refs grows), a last page that is only partly filled is copied to a
 * free page in every pool, and seqlens follows.  made[i] = 1, or 0 where no
 * page was left (as in fa_pages_reserve).  The row dst[i] must hold no pages and
 * be named once, and no item's source may be a destination (item errors). */
fa_status fa_pages_fork(void* const* pools, const size_t* page_bytes, int n_pools,
                        int* block_table, long long table_stride, int* seqlens, int* refs,
                        const int* src, const int* dst, int* made, int B,
                        int pages_per_seq, int num_pages, int page_size, int n,
                        void* workspace, size_t ws_bytes, fa_stream_t stream);

/* Lets go of every page of rows seq_ids[i] (int32, device): refs falls, the row
 * becomes -1 and its length 0.  A row may be named twice. */
fa_status fa_pages_free(int* block_table, long long table_stride, int* seqlens, int* refs,
                        const int* seq_ids, int B, int pages_per_seq, int num_pages, int n,
                        fa_stream_t stream);

/* Makes the used pages the first ones: with U in use, those at U and above move
 * to the free pages below U, lowest to lowest, in every pool; refs and
 * block_table follow.  *used (int32, device) = U.  Other tables that name pages
 * (prefix tables) are not known here and have to be rows of block_table. */
fa_status fa_pages_compact(void* const* pools, const size_t* page_bytes, int n_pools,
                           int* block_table, long long table_stride, int* refs, int* used,
                           int B, int pages_per_seq, int num_pages,
                           void* workspace, size_t ws_bytes, fa_stream_t stream);

/*
 * Decode of a batch whose sequences share long prefixes: the prefix's keys and
 * values are read once for all the queries over them.  Groups of consecutive
 * batch entries share a prefix; sequence b of group g attends the
 * prefix_lens[g] positions of its group's prefix and the seqlens[b] positions
 * of its own behind them,
 *   o = softmax(scale q [K_prefix; K_own]^T) [V_prefix; V_own],
 * one softmax over both parts (their partial states are merged with the
 * rescale-and-add rule of "Flash Attention: principle & practice", section 2.1).
 *   q, kpages, vpages, o, lse, scale, Hkv, page_size : as fa_decode_paged.
 *   prefix_table : int32 [G, prefix_pages], row stride prefix_stride, device:
 *                 the pages of each prefix.  Its rows may be rows of the block
 *                 table.
 *   prefix_lens : int32 [G], device; clamped to [0, prefix_pages * page_size].
 *   cu_batch    : int32 [G + 1], device: group g is batch entries cu_batch[g] ..
 *                 cu_batch[g+1]-1.  NULL with G = 1: the whole batch.  Entries
 *                 of no group have no prefix.  A group that runs backwards or
 *                 leaves the batch is taken as empty and FA_ERR_INVALID_ARG is
 *                 recorded in the device error word; a group behind it begins no
 *                 earlier than the largest end of the groups before it.
 *   block_table : int32 [B, pages_per_seq], row stride table_stride, and
 *   seqlens     : int32 [B], device: each sequence's own pages and length,
 *                 both without the prefix: own position 0 is row 0 of the first
 *                 page listed.  pages_per_seq bounds the own lengths, and
 *                 the own keys are shared out by it: each warp takes at least
 *                 1/62 of a full row (up to 1/8 where B * H * d is large), so a
 *                 table far wider than the lengths leaves the keys to few warps.
 *                 Pass as many columns as the longest sequence needs (a slice by
 *                 the strides).
 *   workspace   : fa_decode_shared_workspace_size(...) bytes, 256-byte aligned.
 * A row with no key at all gets O = 0 and LSE = -inf.  Scores, softmax states and
 * sums are held in 32 bits; the probabilities are rounded to bf16 for the product
 * with V, of the prefix and of the own keys, as in fa_decode_gqa with grouped heads
 * (fa_decode_paged with Hkv = H holds them in 32 bits).  Bad page entries are
 * treated and reported as in fa_decode_paged.  G = 0, prefix_pages = 0 and
 * pages_per_seq = 0 are allowed.  Returns as fa_decode_paged.
 */
size_t fa_decode_shared_workspace_size(int B, int H, int Hkv, int G, int page_size,
                                       int prefix_pages, int pages_per_seq, int d);
fa_status fa_decode_shared(const void* q, const void* kpages, const void* vpages,
                           const int* prefix_table, long long prefix_stride,
                           const int* prefix_lens, const int* cu_batch,
                           const int* block_table, long long table_stride,
                           const int* seqlens, void* o, float* lse, int B, int H, int Hkv,
                           int G, int page_size, int prefix_pages, int pages_per_seq,
                           int num_pages, int d, float scale,
                           void* workspace, size_t ws_bytes, fa_stream_t stream);

/*
 * Measurement hook.  With non-NULL events, every later call records `start`
 * on its stream just before launching its dominant kernel and `stop` just
 * after it: the attention kernel of fa_fwd*, the main kernel of fa_bwd*
 * (not the D = rowsum(dO o O) preprocess or the dQ conversion), the split-KV
 * kernel of fa_decode* (not the combine), the prefix kernel of fa_decode_shared.
 * The calls on rows and pages record nothing.  cudaEventElapsedTime(start, stop)
 * then times that kernel alone.  The events are created and owned by the
 * caller; pass NULL, NULL to turn the hook off.  Process-wide and not
 * thread-safe.  Always returns FA_OK.
 */
fa_status fa_set_timing_events(fa_event_t start, fa_event_t stop);

/*
 * Work-distribution override, for tests and measurements that must exercise
 * one particular schedule.  It changes only how work is spread over the SMs,
 * never a result.  Process-wide (it applies to every later call on every
 * device and host thread) until changed again.
 *   fwd_schedule : FA_SCHEDULE_AUTO lets the library choose per call;
 *                  FA_SCHEDULE_GRID launches the forward with one CTA per
 *                  256-row query tile; FA_SCHEDULE_PERSISTENT launches about
 *                  one CTA per SM (at most a third of the tiles), each looping
 *                  over several tiles.
 *   bwd_order    : FA_SCHEDULE_AUTO; FA_SCHEDULE_GRID orders the backward's
 *                  CTAs head-major (a head's key tiles adjacent);
 *                  FA_SCHEDULE_PERSISTENT launches the longest causal key
 *                  tiles of every head first.
 * Returns FA_ERR_INVALID_ARG for any other value (nothing is changed), else
 * FA_OK.
 */
enum {
    FA_SCHEDULE_AUTO = 0,
    FA_SCHEDULE_GRID = 1,
    FA_SCHEDULE_PERSISTENT = 2
};
fa_status fa_set_schedule(int fwd_schedule, int bwd_order);

/*
 * Synchronises `stream`, then reads and clears the current device's error
 * word.  Returns FA_OK, FA_ERR_TIMEOUT (a kernel gave up a bounded wait and
 * returned without finishing) or FA_ERR_CUDA (the synchronisation failed).
 */
fa_status fa_get_device_error(fa_stream_t stream);

/*
 * Self-check of the failure detection behind FA_ERR_TIMEOUT ("FlashAttention:
 * Fast and Memory-Efficient Exact Attention with IO-Awareness" fixes no
 * failure model; this is the library's own).  Launches one CTA that waits,
 * with the same bounded waits as the attention kernels (a single-thread wait
 * and a warp-collective one), on an mbarrier that nothing arrives on.  After
 * the wait limit (2 s) both give up: the device error word becomes
 * FA_ERR_TIMEOUT and 2 is added to *gave_up (a device int, 4-byte aligned,
 * owned by the caller), and the kernel returns; the context stays usable.
 * Returns FA_ERR_INVALID_ARG for a null or misaligned pointer,
 * FA_ERR_UNSUPPORTED off sm_100, FA_ERR_CUDA if the launch fails.
 */
fa_status fa_check_bounded_wait(int* gave_up, fa_stream_t stream);

/* Static, NUL-terminated description of a status code. */
const char* fa_status_string(fa_status status);

/* Library version as major * 10000 + minor * 100 + patch. */
int fa_version(void);

#ifdef __cplusplus
}
#endif

#endif /* FA_B200_H */
