/*
 * loong_attn.h -- C ABI of the GB300 (sm_103a) LoongTrain 2D-Attention ring step.
 *
 * One process, one GPU.  Every emulated rank of the head-parallel x
 * context-parallel mesh lives on this device; a ring "exchange" is the choice
 * of which K/V chunk a rank reads at a step, so no bytes move between steps.
 *
 * Sources (page title, section):
 *   [G] "Guide to LoongTrain: 2D Head-Context Parallelism for LLMs"
 *   [A] "LoongTrain: Efficient Training of Long-Sequence LLMs with
 *       Head-Context Parallelism" (abstract page)
 *
 * Conventions shared by every entry point
 *   - Pointers named q, k, v, o, o_res, dout, dq, dk, dv, lse, ws, in, out,
 *     o_parts, lse_parts, o_out, lse_out, table, dtable, key_range, wq, wk, positions,
 *     q_out, k_out, v_out, dq_out, dk_out, dv_out, dwq, dwk are DEVICE pointers
 *     owned by the caller:
 *     memory of the current device, from cudaMalloc or managed.  A host
 *     pointer (pinned or not) or another device's memory is refused with
 *     LOONG_ERR_INVALID_ARG before any work is enqueued.  The
 *     library allocates no device memory, keeps no state between calls except a
 *     cached device query, which kernels have their launch attributes set, a
 *     loaded tensor-map encoder, one device error word and (STEPWISE_COPY) one
 *     side stream with its events per device, and synchronises only in
 *     loong_get_device_status.
 *   - All work is enqueued asynchronously on `stream` (0 = legacy default).
 *     Calls (or replays of captured ones) that may run at the same time need
 *     workspaces of their own.
 *   - Tensors are contiguous.  In the NATURAL layout Q, O, dO, dQ are bf16
 *     [B, S, Hq, d] and K, V, dK, dV bf16 [B, S, Hkv, d], natural token order.
 *     In the RANK_MAJOR layout (descriptor field `layout`) they are
 *     [B*cp, hp, S/cp, H/hp, d] with H = Hq or Hkv: ring rank c's S/cp tokens
 *     (its blocks in part order, as the placement assigns them) for head rank
 *     p's H/hp heads, which is what loong_headctx_pack (direction 0, gather 1
 *     for ZIGZAG, 2 for CONTIGUOUS) produces from the natural layout.  LSE is
 *     fp32 [B, Hq, S] in natural token order in both: the natural log of the
 *     softmax denominator of the scaled logits.
 *   - Base pointers must be 16-byte aligned.
 *   - Return value: LOONG_OK (0) or a negative loong_status.  No exception
 *     crosses the ABI; no call aborts the process or traps the GPU.
 */
#ifndef LOONG_ATTN_H
#define LOONG_ATTN_H

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define LOONG_API __attribute__((visibility("default")))
#else
#define LOONG_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

/* Same type as cudaStream_t; declared here so the header needs no CUDA headers. */
typedef struct CUstream_st* loong_stream_t;

typedef enum {
  LOONG_OK = 0,
  LOONG_ERR_INVALID_ARG = -1,     /* null, misaligned or non-device pointer,
                                     bad size or divisibility                 */
  LOONG_ERR_WORKSPACE = -2,       /* ws_bytes smaller than the workspace size */
  LOONG_ERR_UNSUPPORTED = -3,     /* valid but not built: head_dim, a mode /
                                     layout pairing, device is not compute
                                     capability 10.3                          */
  LOONG_ERR_CUDA = -4,            /* a CUDA call failed; see loong_last_cuda_error */
  LOONG_ERR_DEVICE_TIMEOUT = -5,  /* a kernel's bounded wait expired; the
                                     kernel stopped early and its outputs are
                                     undefined                                  */
  LOONG_ERR_DEVICE_CHECK = -6     /* libloong_attn_checked.so: a device
                                     address check failed and the access was
                                     skipped (or shared memory was misaligned);
                                     outputs are undefined                      */
} loong_status;

enum { LOONG_PLACEMENT_CONTIGUOUS = 0, LOONG_PLACEMENT_ZIGZAG = 1 };
enum { LOONG_MODE_STEPWISE = 0, LOONG_MODE_FUSED = 1, LOONG_MODE_STEPWISE_COPY = 2, LOONG_MODE_STEPWISE_COPY_AB = 3 };
enum { LOONG_LAYOUT_NATURAL = 0, LOONG_LAYOUT_RANK_MAJOR = 1 };

/*
 * Problem descriptor.  Follows the problem statement of [G] "1. 2D Mesh
 * Topology" (P = P_head x P_seq), "2. Paired-Block Allocation for Causal Load
 * Balancing" and [A] (Double-Ring-Attention).
 *   batch, seqlen     B and S (tokens per sequence).
 *   hq, hkv           query and key/value heads, hq % hkv == 0 (grouped-query
 *                     attention, [G] "The Scalability Limits of DeepSpeed
 *                     Ulysses").
 *   head_dim          d, 64 or 128.
 *   hp                head-parallel degree P_head: hq % hp == 0 and
 *                     hkv % hp == 0 (each head rank keeps whole kv heads).
 *   cp                context-parallel (ring) degree P_seq.
 *   ring_inner/outer  double-ring shape, inner * outer == cp.  At step
 *                     t = o*inner + i ring rank c holds the K/V of rank
 *                     ((c/inner - o) mod outer)*inner + ((c%inner - i) mod inner).
 *   causal            1: query i sees key j only for j <= i ([G] "The
 *                     Communication Overhead and Causal Imbalance of Ring
 *                     Attention"); 0: every key ([G] "Step 3", is_causal off).
 *   placement         LOONG_PLACEMENT_ZIGZAG: ring rank r owns blocks r and
 *                     2cp-1-r of length S/(2cp); CONTIGUOUS: block r of length
 *                     S/cp.  The block length must be a multiple of hp.
 *   mode              LOONG_MODE_FUSED: one launch walks all ring steps and
 *                     keeps the running softmax on chip; STEPWISE: one launch
 *                     per ring step, each merging its partial result into an
 *                     fp32 accumulator by log-sum-exp.  STEPWISE_COPY
 *                     (RANK_MAJOR layout only): STEPWISE with the ring's K/V
 *                     exchange made real ([G] "3. Double-Ring Asynchronous
 *                     Communication Pipeline"): before step t >= 1 every ring
 *                     rank's incoming chunk is copied (cudaMemcpyAsync, device
 *                     to device) into its receive buffer on a side stream the
 *                     library owns, double-buffered so that the copies of step
 *                     t overlap the kernel of step t-1, and the kernels read
 *                     K/V from the receive buffers.  dK, dV are added at their
 *                     owner's rows (their return trip is not copied).  The
 *                     side stream and its events are one per device: calls in
 *                     this mode on one device must not overlap.
 *                     STEPWISE_COPY_AB (ZIGZAG placement): the same with the
 *                     guide's two rings ([G] section 3): the block A and block
 *                     B halves of every chunk travel on two independent side
 *                     streams.  Results equal STEPWISE's.
 *   softmax_scale     <= 0 selects 1/sqrt(head_dim) ([G] "Step 3",
 *                     forward_local_attention).
 *   layout            LOONG_LAYOUT_NATURAL or LOONG_LAYOUT_RANK_MAJOR (the
 *                     per-rank layout after the Ulysses exchange, [G] "The
 *                     Scalability Limits of DeepSpeed Ulysses"; see above).
 *                     RANK_MAJOR needs batch * seqlen * hp < 2^31.
 */
typedef struct {
  int64_t batch, seqlen;
  int32_t hq, hkv, head_dim;
  int32_t hp, cp, ring_inner, ring_outer;
  int32_t causal;
  int32_t placement;
  int32_t mode;
  float softmax_scale;
  int32_t layout;
} loong_attn_desc;

/* Library version, (major << 16) | minor. */
LOONG_API int loong_version(void);

/* Human-readable text for a loong_status value (static storage). */
LOONG_API const char* loong_status_string(int status);

/* Text of the last CUDA error seen by this library in this thread (static). */
LOONG_API const char* loong_last_cuda_error(void);

/*
 * Check a descriptor without touching the GPU.  Returns LOONG_OK,
 * LOONG_ERR_INVALID_ARG or LOONG_ERR_UNSUPPORTED (see loong_attn_desc).
 */
LOONG_API int loong_attn_check(const loong_attn_desc* desc);

/*
 * Device workspace, in bytes, that loong_attn_fwd (pass 0) or loong_attn_bwd
 * (pass 1) needs for `desc`; 0 for an invalid descriptor.  Host-only.
 *   fwd: the fp16 copy of V that the P V product reads (B*S*Hkv*d values of
 *        2 bytes) and one word for max |V|; STEPWISE adds the fp32 O
 *        accumulator, B*S*Hq*d values.
 *   STEPWISE_COPY adds, to both passes, four 2-byte receive buffers of
 *        B*S*Hkv*d values each (K and V, two of each).
 *   bwd: fp32 dQ accumulator (B*S*Hq*d) + fp32 row statistics (LSE*log2 e
 *        and D = rowsum(dO*O)), 2 x B x Hq x (nblocks*roundup(blk,4) + 128)
 *        values, with nblocks = 2cp (ZIGZAG) or cp and blk = S/nblocks,
 *        + fp32 dK, dV accumulators, B*S*Hkv*d values each.
 *   Each part starts on a 256-byte boundary.
 */
LOONG_API size_t loong_attn_workspace_size(const loong_attn_desc* desc, int pass);

/*
 * The ring schedule as a host table: src[t * cp + c] = ring rank whose K/V
 * ring rank c holds at step t (double-ring reading above).  src must hold
 * inner*outer*inner*outer int32.  Host-only.
 */
LOONG_API int loong_ring_schedule(int32_t ring_inner, int32_t ring_outer, int32_t* src);

/*
 * Forward ring attention ([G] "Step 3", forward_local_attention per block
 * pair, merged over the ring steps).  For every emulated rank (ring rank c,
 * head rank h), every ring step t and every query head of head group h,
 * computes causal softmax attention of rank c's query blocks against the K/V
 * blocks of rank src(c, t) and merges the step's result into the running
 * result by log-sum-exp.  The result equals causal attention over the whole
 * sequence up to rounding.  The probabilities enter the P V product as fp16
 * (V as a scaled fp16 copy in the workspace) and accumulation is fp32, so the
 * unrounded O is within about 2^-12 of exact attention.
 *   q, k, v   inputs (layouts above), read only.
 *   o         bf16 output, the layout of q.
 *   lse       fp32 output [B,Hq,S].
 *   o_res     NULL, or a bf16 output in the layout of q: the rounding
 *             residual of O, bf16(O32 - bf16(O32)) with O32 the fp32 result,
 *             so that O + o_res holds O32 to about 16 bits.  Pass it to
 *             loong_attn_bwd, which then forms D = rowsum(dO * O) from
 *             O + o_res.
 *   ws        device workspace of at least loong_attn_workspace_size(desc,0)
 *             bytes; every descriptor needs one.
 */
LOONG_API int loong_attn_fwd(const loong_attn_desc* desc, const void* q, const void* k, const void* v,
                   void* o, float* lse, void* o_res, void* ws, size_t ws_bytes, loong_stream_t stream);

/*
 * loong_attn_fwd restricted to the query rows of ring ranks
 * [rank_begin, rank_end) (all heads, all sequences of the batch): the work of
 * those emulated ranks alone, so that one rank's share of the ring pass can be
 * timed ([G] section 2 gives every rank the same work under paired blocks).
 * Rows of other ranks in o and lse are left untouched; the rows written equal
 * those of loong_attn_fwd bit for bit.  FUSED mode only (STEPWISE returns
 * LOONG_ERR_UNSUPPORTED); ws as for loong_attn_fwd.  0 <= rank_begin <
 * rank_end <= cp.
 */
LOONG_API int loong_attn_fwd_ranks(const loong_attn_desc* desc, int32_t rank_begin, int32_t rank_end,
                                   const void* q, const void* k, const void* v, void* o, float* lse,
                                   void* ws, size_t ws_bytes, loong_stream_t stream);

/*
 * Backward of loong_attn_fwd: the exact gradient of causal softmax attention
 * (the pages give no backward; this is the plain chain rule through softmax).
 * Over the same schedule: P = exp(s - LSE), dV += P^T dO, dP = dO V^T,
 * dS = P * (dP - D) with D = rowsum(dO * O), dQ += scale dS K,
 * dK += scale dS^T Q; dK and dV sum over the query heads of a kv group.
 *   o, lse    the outputs of loong_attn_fwd for the same inputs.
 *   o_res     the forward's o_res output, or NULL.  D is formed in fp32 from
 *             O + o_res, else from the bf16 O alone.  The D term of dQ and dK
 *             is -scale * D * (probability-weighted keys or queries), so an
 *             error in D is amplified where a few large keys take the
 *             probability mass; with o_res, D carries the forward's own
 *             accuracy instead of bf16's 2^-9.
 *   dout      bf16 dO, the layout of q.
 *   dq        bf16, the layout of q; dk, dv bf16, the layout of k; written,
 *             not added to.
 *   ws        at least loong_attn_workspace_size(desc,1) bytes.
 */
LOONG_API int loong_attn_bwd(const loong_attn_desc* desc, const void* q, const void* k, const void* v,
                   const void* o, const void* o_res, const float* lse, const void* dout,
                   void* dq, void* dk, void* dv, void* ws, size_t ws_bytes,
                   loong_stream_t stream);

/*
 * Largest workspace, in bytes, that loong_attn_bwd_noalloc can serve: 32 MiB.
 * A problem fits when loong_attn_workspace_size(desc, 1) is at most this; in
 * FUSED and STEPWISE mode that size is at most 4*B*S*Hq*d + 8*B*S*Hkv*d +
 * 8*B*Hq*(S + 3*nblocks + 128) bytes plus 256 per part (four parts), with
 * nblocks = 2cp (ZIGZAG) or cp.  For example S = 4096 tokens, Hq = 8, Hkv = 1,
 * d = 128 needs about 20.3 MiB.
 */
#define LOONG_NOALLOC_SCRATCH_BYTES (32u << 20)

/*
 * loong_attn_bwd without a workspace argument, for callers that cannot
 * allocate device memory: a plugin inside a framework that owns the whole
 * device pool and hands it only inputs and outputs, or a latency-critical loop
 * that cannot take cudaMalloc's implicit device synchronisation.  The paper
 * has no counterpart; this is an interface convenience.
 *   Same arguments, layouts and results as loong_attn_bwd, minus ws/ws_bytes.
 *   The descriptor is checked first, then the device (LOONG_ERR_UNSUPPORTED
 *   on one that is not compute capability 10.3); a problem whose workspace
 *   exceeds the array gives LOONG_ERR_WORKSPACE.
 *   Scratch lives in one static device array of LOONG_NOALLOC_SCRATCH_BYTES
 *   that every GPU loading the library holds until the process exits.  The
 *   call allocates nothing: no cudaMalloc, cudaFree or allocating library
 *   routine.  Returns LOONG_ERR_WORKSPACE when
 *   loong_attn_workspace_size(desc, 1) exceeds LOONG_NOALLOC_SCRATCH_BYTES.
 *   The first call on a device looks up the array's device address
 *   (cudaGetSymbolAddress) with that device current; make that first call
 *   before any stream capture.  A failed lookup is not remembered: the next
 *   call tries again.
 *   Every call on a device shares the one array and it keeps the last call's
 *   contents (the parts that must start at zero are cleared by each call):
 *   calls whose work overlaps on the GPU (other streams, other host threads)
 *   race on it and must be serialised by the caller.
 */
LOONG_API int loong_attn_bwd_noalloc(const loong_attn_desc* desc, const void* q, const void* k,
                                     const void* v, const void* o, const void* o_res, const float* lse,
                                     const void* dout, void* dq, void* dk, void* dv, loong_stream_t stream);

/*
 * n-way log-sum-exp merge of partial attention results over disjoint key sets
 * (the pages leave the merge implicit; it is the rule under which softmax over
 * a union of key sets is recovered from the parts):
 *   L = ln sum_p exp(L_p),  O = sum_p exp(L_p - L) O_p.
 * A part with L_p = -inf is empty and has weight 0; if all parts are empty the
 * row gets L = -inf and O = 0.
 *   o_parts   fp32 [n_parts][rows][d];  lse_parts fp32 [n_parts][rows].
 *   o_out     fp32 [rows][d] (out_bf16 == 0) or bf16 [rows][d] (out_bf16 == 1).
 *   lse_out   fp32 [rows].
 * rows >= 0 (0 is a no-op), 1 <= d <= 1024 with d % 4 == 0, 1 <= n_parts <= 64.
 * Outputs must not overlap inputs.
 */
LOONG_API int loong_lse_merge(int64_t rows, int32_t d, int32_t n_parts,
                    const float* o_parts, const float* lse_parts,
                    void* o_out, float* lse_out, int out_bf16, loong_stream_t stream);

/*
 * Ulysses head-context repack ([G] "The Scalability Limits of DeepSpeed
 * Ulysses": all-to-all (S/P, H) -> (S, H/P) before attention and the inverse
 * after), for every ring rank's head-parallel group at once, as a bit copy of
 * 2-byte elements.
 *   direction 0:  out[n][p][q*s_local + t][h'][:] = in[n][q][t][p*H/P + h'][:]
 *   direction 1:  the inverse (out and in swap roles).
 * with n < batch*cp (group = ring rank of one sequence), p, q < P, t < s_local,
 * h' < H/P.  `gather` selects the layout of the (S/P, H) side:
 *   0  rank-major [batch*cp][P][s_local][H][d];
 *   1  natural token order [batch][S][H][d], S = cp*P*s_local, ring rank n
 *      owning the paired blocks n and 2cp-1-n ([G] section 2);
 *   2  natural token order with contiguous blocks.
 * The (S, H/P) side is always rank-major [batch*cp][P][P*s_local][H/P][d].
 * H % P == 0, d*2 bytes a multiple of 16, in and out must not overlap.
 */
LOONG_API int loong_headctx_pack(int64_t batch, int32_t cp, int32_t P, int64_t s_local, int32_t heads,
                       int32_t d, int direction, int gather, const void* in, void* out,
                       loong_stream_t stream);

/*
 * loong_headctx_pack over n tensors (1 <= n <= 4) in one launch: the same
 * batch, cp, P, s_local, d, direction and gather, their own head counts, as
 * the Q, K, V (and dO) of one pass, whose repacks are the one all-to-all the
 * guide describes.  Tensor t has heads[t] heads (each a multiple of P) and
 * moves from in[t] to out[t]; heads, in and out are host arrays of n entries.
 * The results equal n calls of loong_headctx_pack bit for bit.
 */
LOONG_API int loong_headctx_pack_n(int32_t n, int64_t batch, int32_t cp, int32_t P, int64_t s_local,
                                   const int32_t* heads, int32_t d, int direction, int gather,
                                   const void* const* in, void* const* out, loong_stream_t stream);

/*
 * Ring attention with a learned relative position bias in buckets: the logit
 * of query i and key j is softmax_scale * q_i.k_j + table[bucket(i - j)][head],
 * with i, j natural token positions.  The paper's attention has no bias; a
 * layer that learns its positions this way needs it inside the attention,
 * whose scores never reach memory.
 *   num_buckets  rows of the table, 1 .. 256.
 *   num_bounds   0 .. 255; the distances -inf .. inf are cut into num_bounds + 1
 *                intervals.
 *   bounds       HOST array of num_bounds strictly increasing distances: n lies
 *                in interval number #{bounds <= n}.  Causal descriptors only
 *                meet n >= 0, others both signs.
 *   bucket_of    HOST array of num_bounds + 1 buckets, one per interval
 *                (several intervals may share one), or NULL: interval i is
 *                bucket i.
 *   table        DEVICE bf16 [num_buckets][hq], 2-byte aligned.  A value of
 *                -2^20 or less (-1e9, the type's lowest and -inf included)
 *                masks: its keys get no weight.  A query that this leaves no
 *                key gets O = 0 and LSE = -inf, and adds nothing to any
 *                gradient.  Masked keys are still read and multiplied.  2^20 or
 *                more counts as +inf: like NaN, it makes the outputs NaN that
 *                it enters.  A bucket that no pair falls in adds to nothing, what
 *                ever it holds (a finite value there may decide how a logit next
 *                to it rounds).
 * The two host arrays are read during the call only.
 */
typedef struct {
  int32_t num_buckets, num_bounds;
  const int32_t* bounds;
  const int32_t* bucket_of;
  const void* table;
} loong_rel_bias;

/*
 * Check a descriptor and a bias without touching the GPU (the table pointer is
 * not looked at): as loong_attn_check, and LOONG_ERR_INVALID_ARG for a bias
 * out of the ranges above, LOONG_ERR_UNSUPPORTED for seqlen > 2^29 or a
 * softmax_scale in (0, 2^-24).
 */
LOONG_API int loong_rel_bias_check(const loong_attn_desc* desc, const loong_rel_bias* bias);

/*
 * Device workspace, in bytes, of loong_attn_bias_fwd (pass 0) or
 * loong_attn_bias_bwd (pass 1); 0 for invalid arguments.  Host-only.
 * loong_attn_workspace_size's, then the bias of every distance (fp32,
 * hq * (S + 384) values, hq * (2 S + 256) non-causal), its interval (bytes) and
 * two words on its surroundings; for the forward 1,216 words more; for the
 * backward the gradient's parts, 16 * (hq/hkv) * (num_bounds + 1) fp32 for every
 * (sequence, kv head, 128-key tile), a word for every head, and 64 sums of the
 * parts.
 */
LOONG_API size_t loong_attn_bias_workspace_size(const loong_attn_desc* desc, const loong_rel_bias* bias, int pass);

/*
 * loong_attn_fwd with the bias: same arguments, layouts, modes and accuracy.
 * ws needs loong_attn_bias_workspace_size(desc, bias, 0) bytes.
 */
LOONG_API int loong_attn_bias_fwd(const loong_attn_desc* desc, const loong_rel_bias* bias, const void* q,
                                  const void* k, const void* v, void* o, float* lse, void* o_res, void* ws,
                                  size_t ws_bytes, loong_stream_t stream);

/*
 * loong_attn_bwd with the bias, and the gradient of the table:
 *   dtable  bf16 [num_buckets][hq], written: the sum of dS (see loong_attn_bwd)
 *           over every pair of the bucket, summed in fp32 within a compute warp
 *           and in fp64 beyond, and rounded once; 0 for a bucket no pair falls
 *           in.  The sums do not depend on the order in which blocks run.  D
 *           carries the accuracy of o and o_res into it; without o_res it is as
 *           exact as bf16 O.
 * o, o_res and lse are loong_attn_bias_fwd's for the same bias.  ws needs
 * loong_attn_bias_workspace_size(desc, bias, 1) bytes.
 */
LOONG_API int loong_attn_bias_bwd(const loong_attn_desc* desc, const loong_rel_bias* bias, const void* q,
                                  const void* k, const void* v, const void* o, const void* o_res, const float* lse,
                                  const void* dout, void* dq, void* dk, void* dv, void* dtable, void* ws,
                                  size_t ws_bytes, loong_stream_t stream);

/*
 * Ring attention in which every query sees a range of keys of its own, with an
 * optional cap of the scores: the logit of query i and key j is
 * cap * tanh(softmax_scale * q_i.k_j / cap), over begin_i <= j < end_i.  Packed
 * documents, prefixes that see themselves whole, windows and padding are all
 * ranges.  The paper's attention is causal over one sequence; layers that train
 * on packed sequences or cap their scores need these inside it.
 *   key_range  DEVICE int32 [B][S][2], 8-byte aligned: begin and end of query i,
 *              in natural token positions of its sequence, or NULL: every key.
 *              Clipped to 0 .. S and, for causal descriptors, to keys j <= i.  A
 *              query that this leaves no key gets O = 0 and LSE = -inf, adds
 *              nothing to any gradient and gets dQ = 0.
 *   score_cap  0: none; else 2^-20 .. 2^20 (and softmax_scale, where given,
 *              2^-24 .. 2^24).
 * What a key or a query holds does not matter to those that do not see each
 * other: a value that is not finite reaches, as NaN, only what sees its row.
 * FUSED descriptors visit the tiles that some query of a tile sees in natural
 * order, the other modes those of every ring step.
 */
typedef struct {
  const int32_t* key_range;
  float score_cap;
} loong_attn_mask;

/*
 * Check a descriptor and a mask without touching the GPU (key_range is not
 * looked at): as loong_attn_check, and LOONG_ERR_INVALID_ARG for a negative or
 * not finite cap, LOONG_ERR_UNSUPPORTED for one out of range, seqlen > 2^30 or
 * more than 65535 sequences or query heads.
 */
LOONG_API int loong_attn_mask_check(const loong_attn_desc* desc, const loong_attn_mask* mask);

/*
 * Device workspace, in bytes, of loong_attn_mask_fwd (pass 0) or
 * loong_attn_mask_bwd (pass 1); 0 for invalid arguments.  Host-only.
 * loong_attn_workspace_size's, then 16 bytes for every 128-token query tile of a
 * block; for the forward 1,216 words and one word more, for the backward a byte
 * for every query tile and head.  Each part starts on a 256-byte boundary.  A FUSED
 * descriptor with the NATURAL layout counts as one of cp = hp = 1, one block.
 * Where a FUSED backward's key tiles of 128 (of all blocks, kv heads and sequences)
 * are 76 or fewer, the query heads of a group go to up to 152 / tiles blocks, each
 * with fp32 values for the whole of dK and dV.
 */
LOONG_API size_t loong_attn_mask_workspace_size(const loong_attn_desc* desc, const loong_attn_mask* mask, int pass);

/*
 * loong_attn_fwd with the mask: same arguments, layouts, modes and accuracy (a
 * capped logit is off by at most 2^-19 of itself more, or 2^-21 of a cap of up to 64).
 * ws needs loong_attn_mask_workspace_size(desc, mask, 0) bytes.
 */
LOONG_API int loong_attn_mask_fwd(const loong_attn_desc* desc, const loong_attn_mask* mask, const void* q,
                                  const void* k, const void* v, void* o, float* lse, void* o_res, void* ws,
                                  size_t ws_bytes, loong_stream_t stream);

/*
 * loong_attn_bwd with the mask: dS takes the factor 1 - tanh^2 of its score.
 * o, o_res and lse are loong_attn_mask_fwd's for the same mask.  ws needs
 * loong_attn_mask_workspace_size(desc, mask, 1) bytes.
 */
LOONG_API int loong_attn_mask_bwd(const loong_attn_desc* desc, const loong_attn_mask* mask, const void* q,
                                  const void* k, const void* v, const void* o, const void* o_res, const float* lse,
                                  const void* dout, void* dq, void* dk, void* dv, void* ws, size_t ws_bytes,
                                  loong_stream_t stream);

/*
 * What loong_qk_norm_rope_fwd does to Q and K.
 *   q/k/v_stride, elements from one token to the next of the projections q, k, v
 *   dq/dk/dv_stride  and of their gradients, so that either can be slices of
 *                 one fused [B, S, W] tensor: 0 = contiguous (heads *
 *                 head_dim), else at least that and a multiple of 8, at most
 *                 2^31.  A token's heads are contiguous; a sequence is seqlen
 *                 strides.
 *   norm          1: RMS norm of every head of Q and K (eps >= 0 finite, weight
 *                 w + w_offset, e.g. w_offset 1 for weights stored around 0);
 *                 0: none.
 *   rot_dim       the first rot_dim elements of a head rotate, a multiple of 16
 *                 from 0 (none) to head_dim, in pairs (i, i + rot_dim/2) or,
 *                 interleaved = 1, (2i, 2i + 1).  Pair i turns by position *
 *                 inv_freq[i] (HOST array of rot_dim/2 finite values, read
 *                 during the call) or, inv_freq == NULL, by position *
 *                 rot_base^(-2i/rot_dim), rot_base a positive normal
 *                 double.
 *   rot_scale     factor of every cosine and sine (1 for a plain rotation).
 *   pos_begin     position of token 0 of every sequence, where no positions are
 *                 given.
 * Angles are reduced in 64-bit fixed point: any 64-bit position turns by its
 * angle to 2^-23 + |position| (|inv_freq| 2^-52 + 2 pi 2^-64) of a radian.
 */
typedef struct {
  int64_t q_stride, k_stride, v_stride;
  int64_t dq_stride, dk_stride, dv_stride;
  int64_t pos_begin;
  double rot_base;
  const double* inv_freq;
  float eps, w_offset, rot_scale;
  int32_t norm, rot_dim, interleaved;
} loong_qk_opts;

/*
 * From a layer's projections to its attention's inputs in one pass: RMS norm
 * and rotation of every head of Q and K, and the descriptor's layout.  The
 * paper starts at the attention; this is the step in front of it, fused with
 * loong_headctx_pack (direction 0; gather 1 for ZIGZAG, 2 for CONTIGUOUS) when
 * the layout is RANK_MAJOR.  The descriptor's mode, causal flag and scale do
 * not matter.
 *   q, k, v          bf16 projections [B, S, heads, d], token-strided (above).
 *   wq, wk           fp32 [head_dim] norm weights, or NULL: all ones (w_offset
 *                    is then not added).
 *   positions        int64 [B, S], or NULL: pos_begin + token index.
 *   q_out, k_out,    bf16, the descriptor's layout, contiguous.  v_out is a copy
 *   v_out            of v; v and v_out may both be NULL.
 * Norm, rotation and weights are applied in fp32 and rounded to bf16 once.
 * Outputs must not overlap inputs.
 */
LOONG_API int loong_qk_norm_rope_fwd(const loong_attn_desc* desc, const loong_qk_opts* opts, const void* q,
                                     const void* k, const void* v, const float* wq, const float* wk,
                                     const int64_t* positions, void* q_out, void* k_out, void* v_out,
                                     loong_stream_t stream);

/*
 * Device workspace of loong_qk_norm_rope_bwd, in bytes (0 when opts.norm is 0,
 * or for invalid arguments).  Host-only.
 */
LOONG_API size_t loong_qk_norm_rope_bwd_workspace_size(const loong_attn_desc* desc, const loong_qk_opts* opts);

/*
 * Gradient of loong_qk_norm_rope_fwd.
 *   q, k               the forward's inputs (may be NULL when opts.norm is 0).
 *   dq_out, dk_out,    gradients of the forward's outputs, the descriptor's
 *   dv_out             layout.
 *   dq, dk, dv         gradients of the projections, token-strided (elements
 *                      between a token's heads and the next token are left as
 *                      they are).  dv_out and dv may both be NULL.
 *   dwq, dwk           fp32 [head_dim], written, or NULL where not wanted (both
 *                      NULL when opts.norm is 0).  Summed in a fixed order.
 *   ws                 needed when dwq or dwk is given.
 */
LOONG_API int loong_qk_norm_rope_bwd(const loong_attn_desc* desc, const loong_qk_opts* opts, const void* q,
                                     const void* k, const float* wq, const float* wk, const int64_t* positions,
                                     const void* dq_out, const void* dk_out, const void* dv_out, void* dq, void* dk,
                                     void* dv, float* dwq, float* dwk, void* ws, size_t ws_bytes,
                                     loong_stream_t stream);

/*
 * Attention of new tokens over a cache of pages, after writing their keys and
 * values into it: what a trained layer runs when it answers, from one new token
 * of many sequences to a chunk of a long prompt.  The paper trains only; query
 * heads, scores, cap and window are the attention's above.
 *   batch       sequences, 1 .. 4096.
 *   tokens      rows of q (and k, v): sequence b's new tokens are rows
 *               starts[b] .. starts[b + 1] - 1.  Rows from starts[batch] on are
 *               not looked at and their outputs left as they are.
 *   hq, hkv     hq % hkv == 0, at most 128 query heads to a kv head.
 *   head_dim    64 or 128.
 *   page_size   tokens of a page, a power of two from 8 to 1024.
 *   num_pages   pages of the pool; (num_pages + 1) * page_size <= 2^30.
 *   max_pages   pages of a row of the table; max_pages * page_size <= 2^30.
 *   window      0, or the number of keys that a token sees, itself included.
 *   softmax_scale  <= 0 selects 1/sqrt(head_dim).
 *   score_cap   0: none; else as in loong_attn_mask.
 *   q/k/v_stride  elements from one token's row to the next, 0 = contiguous
 *               (heads * head_dim), else at least that, a multiple of 8 and at
 *               most 2^31; a row's heads are contiguous.
 */
typedef struct {
  int32_t batch, tokens, hq, hkv, head_dim;
  int32_t page_size, num_pages, max_pages;
  int32_t window;
  float softmax_scale, score_cap;
  int64_t q_stride, k_stride, v_stride;
} loong_paged_desc;

/*
 * Check a paged descriptor without touching the GPU: LOONG_OK,
 * LOONG_ERR_INVALID_ARG or LOONG_ERR_UNSUPPORTED (ranges above; work whose units
 * of 128 rows by 128 keys may pass 2^31).
 */
LOONG_API int loong_paged_check(const loong_paged_desc* desc);

/* Device workspace of loong_paged_attn, in bytes; 0 for an invalid descriptor.  Host-only. */
LOONG_API size_t loong_paged_attn_workspace_size(const loong_paged_desc* desc);

/*
 *   q           bf16 [tokens][hq][head_dim], token-strided.
 *   k, v        bf16 [tokens][hkv][head_dim], token-strided: written to the new
 *               tokens' places before anything is read; both NULL: they are there
 *               already.
 *   k_pages,    bf16 [num_pages][page_size][hkv][head_dim], contiguous.  Places that
 *   v_pages     no sequence uses may hold anything.
 *   table       int32 [batch][max_pages]: sequence b's key j is row j % page_size of
 *               page table[b][j / page_size].  Entries past a sequence's length, or
 *               wholly before what its new tokens see, are not read.
 *   lens        int32 [batch]: lengths with the new tokens.  New token t of a
 *               sequence (t = 0 .. n - 1) stands at position lens[b] - n + t and sees
 *               the keys up to its own.
 *   starts      int32 [batch + 1], starting anywhere from 0, not falling.
 *   o, lse      bf16 [tokens][hq][head_dim] and fp32 [hq][tokens] (natural log of
 *               the softmax denominator), contiguous.  They must not overlap what
 *               is read, nor k and v the pages.
 * The arrays are read on the device, so a captured call may be replayed on other
 * lengths, tables and starts.  Pages that two new tokens share (the same place
 * written twice) hold either's row.  A page outside the pool is read as zeros and
 * not written, lengths and starts out of range are cut (tokens that stand before
 * position 0 see nothing: O = 0, LSE = -inf), and loong_get_device_status then
 * reports LOONG_ERR_DEVICE_CHECK.  No work with tokens == 0.
 * Results do not depend on the order in which blocks run.  P enters the P V
 * product as bf16 and O is divided by the sum of the rounded values; all else is
 * fp32.
 */
LOONG_API int loong_paged_attn(const loong_paged_desc* desc, const void* q, const void* k, const void* v,
                               void* k_pages, void* v_pages, const int32_t* table, const int32_t* lens,
                               const int32_t* starts, void* o, float* lse, void* ws, size_t ws_bytes,
                               loong_stream_t stream);

/*
 * Device workspace, in bytes, of loong_attn_2d_host for `desc`: pass 0 runs
 * the forward alone, pass 1 the forward and the backward; 0 for an invalid
 * descriptor.  Host-only.  It holds two sets of natural-layout inputs (the
 * slots), the natural-layout outputs and LSE, the forward's residual of O
 * (pass 1: the backward forms D from O and it), the rank-major tensors of the
 * pass (RANK_MAJOR) and the workspaces of loong_attn_fwd / loong_attn_bwd,
 * each part on a 256-byte boundary.
 */
LOONG_API size_t loong_attn_2d_host_workspace_size(const loong_attn_desc* desc, int pass);

/*
 * One whole 2D-attention pass from host memory to host memory: the inputs
 * travel to the device, the Ulysses repack moves them into every emulated
 * rank's layout ([G] "The Scalability Limits of DeepSpeed Ulysses"), the ring
 * forward (and backward) run on it, and the outputs are repacked and travel
 * back.  With a NATURAL descriptor the ring kernels read and write the
 * natural layout and there is no repack.
 *   q, k, v, dout   host inputs, natural layout [B,S,H,d] bf16.  dout == NULL
 *                   runs the forward alone (dq, dk, dv must then be NULL).
 *   o, lse          host outputs: bf16 [B,S,Hq,d] and fp32 [B,Hq,S].
 *   dq, dk, dv      host outputs, bf16, the layouts of q and k.
 *   slot            0 or 1: which of the workspace's two device input sets
 *                   this call fills.  Alternate it between consecutive calls
 *                   so that a call's inputs can arrive while the previous
 *                   call's kernels still read theirs.
 *   ws, ws_bytes    device workspace of loong_attn_2d_host_workspace_size
 *                   bytes (pass 1 when dout != NULL, else pass 0).
 *   done_event      a cudaEvent_t of the caller, or NULL.  Non-NULL: it is
 *                   recorded once every output has reached host memory, and
 *                   `stream` does not wait for the output copies, so the next
 *                   call's kernels overlap them.  NULL: `stream` waits for the
 *                   output copies before its later work.
 * Every copy runs on one of two library-owned copy streams (host to device,
 * device to host), ordered against the kernels on `stream` by events: a
 * call's input copies start when the call is made, once the slot's previous
 * inputs have been read; dO arrives while the forward runs, and O and LSE
 * leave while the backward runs.  Pinned host memory (cudaHostAlloc /
 * cudaHostRegister, or loong_host_alloc below, which also keeps the copies at
 * full speed when the device's translations of host pages have gone cold)
 * lets the copies overlap the kernels; pageable memory is accepted but
 * copies synchronously.  The caller must not change the inputs
 * or read the outputs before the call's work has finished (done_event, or
 * `stream` when done_event is NULL).  Calls on one device are serialised by
 * the library (one enqueue at a time).  Device pointers in the host
 * arguments, a slot other than 0 or 1 and null pointers give
 * LOONG_ERR_INVALID_ARG; a short workspace gives LOONG_ERR_WORKSPACE.
 */
LOONG_API int loong_attn_2d_host(const loong_attn_desc* desc, int32_t slot, const void* q, const void* k,
                                 const void* v, const void* dout, void* o, float* lse, void* dq, void* dk,
                                 void* dv, void* ws, size_t ws_bytes, loong_stream_t stream,
                                 void* done_event);

/*
 * Pinned host memory for the host arguments of loong_attn_2d_host (or any
 * host <-> device copy): `bytes` bytes at *ptr, registered with CUDA, in an
 * anonymous mapping aligned to the kernel's transparent huge page size and
 * advised to use huge pages (where the kernel offers none the buffer is
 * still pinned).  Why: the device translates every host page a copy touches,
 * and when those translations have gone cold (a few seconds without copies,
 * or after kernels that sweep much device memory) each page costs a miss.
 * Measured with 64 KB base pages, a 2.7 GB host-to-device copy then took
 * 360-380 ms from cudaHostAlloc memory and 12.7 ms from huge pages.  The
 * range is also asked to collapse into huge pages (MADV_COLLAPSE, where the
 * kernel has it).  On some hosts device writes into the buffer split part of
 * it back into base pages, and copies into it slow down again.
 *   bytes == 0 sets *ptr = NULL.  The caller owns the buffer and releases it
 *   with loong_host_free.  Returns LOONG_OK, LOONG_ERR_INVALID_ARG (null
 *   ptr), or LOONG_ERR_CUDA (mapping or registration failed; *ptr = NULL).
 */
LOONG_API int loong_host_alloc(size_t bytes, void** ptr);

/*
 * Unregister and unmap a buffer from loong_host_alloc.  NULL is a no-op; a
 * pointer that loong_host_alloc did not return gives LOONG_ERR_INVALID_ARG.
 * No copy may still use the buffer.
 */
LOONG_API int loong_host_free(void* ptr);

/*
 * Measurement aid.  When both are non-NULL, the calling thread's next
 * loong_attn_fwd / loong_attn_bwd calls record `start_event` on their stream
 * just before launching the main ring-attention kernel(s) and `stop_event`
 * just after the last of them, so the kernels' device time can be read with
 * cudaEventElapsedTime without counting the call's helper kernels.  The events
 * are cudaEvent_t handles owned by the caller; pass NULL, NULL to stop.
 */
LOONG_API int loong_set_timing_events(void* start_event, void* stop_event);

/*
 * Synchronise `stream` and report device-side failures of earlier calls:
 * LOONG_ERR_DEVICE_CHECK if an address check of the checked build failed or a
 * kernel found its shared memory misaligned, else LOONG_ERR_DEVICE_TIMEOUT if
 * a kernel's bounded wait expired (the error word is then cleared),
 * LOONG_ERR_CUDA if the stream reports a CUDA error, LOONG_OK otherwise.
 */
LOONG_API int loong_get_device_status(loong_stream_t stream);

/*
 * Self-test of the bounded-wait path (no counterpart on the pages): launches
 * one CTA on `stream` whose mbarrier wait, the same code every kernel's waits
 * use, has nothing to wait for.  It gives up after limit_us microseconds
 * (1 .. 1000000), raises the CTA's abort flag, sets the device error word and
 * returns, so the next loong_get_device_status reports
 * LOONG_ERR_DEVICE_TIMEOUT and clears the word; the context stays usable.
 * Returns LOONG_ERR_INVALID_ARG for a limit out of range (before any CUDA
 * call), else the launch status.
 */
LOONG_API int loong_selftest_wait_timeout(uint32_t limit_us, loong_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* LOONG_ATTN_H */
