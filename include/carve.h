/*
 * carve.h: C ABI of the CARVE chunk-parallel forward pass on MI355X (gfx950).
 *
 * The operation is the forward pass of the CARVE recurrent layer (arXiv
 * 2606.27229, "CARVE: Content-Aware Recurrent with Value Efficiency for
 * Chunk-Parallel Linear Attention"), as described in the gist.science
 * technical summaries:
 *   section 1 (problem statement)   per head a state S of shape d_v x d_k;
 *   section 2 (method)              every gate acts on the key axis only;
 *   section 2.1 (output reuse)      o_t = S_{t-1} q_t, chunk mean
 *                                   m_c = (1/L) sum o_t, erase gate
 *                                   b = sigmoid(b_x + U_b m), one chunk stale;
 *   section 2.2 (scalar write)      one write gate w per head and token,
 *                                   broadcast over the value channels;
 *   section 2.3 (key-axis decay)    exponential decay exp(g) on the key axis;
 *                                   the activation that turns the decay
 *                                   logits into g may run inside the kernel
 *                                   ("gate-in-kernel", CARVE_DECAY_LOGITS).
 * Per token (readings: b scales the retrieval key; decay precedes erase):
 *   o_t = S q_t;  S <- S diag(exp(g_t)) (I - (b_t * k_t) k_t^T) + w_t v_t k_t^T
 * with b_t = sigmoid(bx_t + U_up (U_down m_{c-1})) for every token of chunk c,
 * m_{-1} = mean_in (zero when absent), and m_c the mean of chunk c's outputs
 * over the tokens it holds (a last chunk may be partial).
 * The library computes this with the WY-form chunk solver (Theorem 11 in
 * section 3 of the same summaries: key-axis-only erase leaves one triangular
 * system per chunk).
 *
 * Conventions for every entry point:
 *   - No HIP types cross this header; `stream` is a hipStream_t passed as
 *     void* (NULL = the null stream).
 *   - All tensor pointers are device pointers owned by the caller. The library
 *     never allocates, frees or synchronises; work is queued on `stream` and
 *     the call returns before it finishes.
 *   - Tensors are dense, row-major, 16-byte aligned, no strides.
 *   - Every argument check runs before the first HIP call, so invalid
 *     arguments are reported (and testable) without a GPU.
 *   - The library keeps no state beyond a per-device record of the kernels'
 *     LDS limits it has raised; concurrent calls need distinct outputs.
 *   - Errors are returned as a carve_status code; nothing is thrown.
 */
#ifndef CARVE_H
#define CARVE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  CARVE_OK = 0,
  CARVE_EINVAL = 1,        /* NULL required pointer, negative size, unknown flag bit */
  CARVE_EUNSUPPORTED = 2,  /* d_k/d_v not in {64,128}, L not in {16,32,64,128}, d_k != d_v,
                              rank > 64, or a size past the kernels' 32-bit index range */
  CARVE_EALIGN = 3,        /* a pointer (or, where there are strides, a stride) is not 16-byte aligned */
  CARVE_EWORKSPACE = 4,    /* workspace smaller than the entry point's size function asks */
  CARVE_EHIP = 5           /* a HIP launch failed; carve_error_string(CARVE_EHIP) has the text */
} carve_status;

typedef enum { CARVE_F32 = 0, CARVE_BF16 = 1 } carve_dtype;

/* Bits of carve_config.flags.
 *   CARVE_DECAY_LOGITS  the g tensor holds raw decay logits a instead of the
 *                       log-decay, and the kernels form g = -softplus(a)
 *                       = -log(1 + e^a) themselves (the decay activation of
 *                       section 2.3 applied in-kernel), so the caller never
 *                       materialises the activated tensor. Any real a is
 *                       valid; exp(g) = sigmoid(-a) lies in (0, 1).
 *   CARVE_QK_L2NORM     q and k are raw: the kernels divide each token's q
 *                       and k by their L2 norms over dk (x / max(|x|, 1e-12))
 *                       before using them, so the caller need not normalise
 *                       them in a separate pass.
 *   CARVE_DETACH_MEAN   backward only (the forward and the step ignore it):
 *                       the chunk means that feed the content gate are taken
 *                       as constants, as when a training loop detaches them.
 *                       U_down and U_up still get their gradients through the
 *                       gate; no gradient reaches earlier outputs or mean_in
 *                       through it (d_mean_out still reaches the last chunk's
 *                       outputs). Without the bit the gradients are the exact
 *                       ones, through every stale mean. */
enum { CARVE_DECAY_LOGITS = 1, CARVE_QK_L2NORM = 2, CARVE_DETACH_MEAN = 4 };

/* Problem description. B batch, H heads, T tokens, dk key width, dv value
 * width, L chunk length of the content signal, rank of U_b (0 = no content
 * projection), dtype of every activation tensor and of U_down/U_up, flags a
 * bitwise OR of the bits above (0 for none; an unknown bit is CARVE_EINVAL). */
typedef struct {
  int32_t B, H, T, dk, dv, L, rank;
  int32_t dtype; /* carve_dtype */
  int32_t flags; /* a bitwise OR of the CARVE_* bits above, or 0 */
} carve_config;

/* Element counts of every tensor (not bytes), and the workspace size in bytes. */
typedef struct {
  int64_t q, k, v, g, bx, w;   /* inputs */
  int64_t ub_down, ub_up;      /* content projection factors (0 when rank == 0) */
  int64_t o;                   /* output */
  int64_t state, mean;         /* optional fp32 state_in/out and mean_in/out */
  int64_t workspace_bytes;     /* device scratch carve_chunk_fwd needs */
  int64_t bwd_workspace_bytes; /* device scratch carve_chunk_bwd needs */
} carve_shapes;

/* Validates `cfg` and fills `out` with the shape contract of the recurrence:
 *   q, k, g, bx : [B, T, H, dk]      v, o : [B, T, H, dv]      w : [B, T, H]
 *   ub_down     : [H, rank, dv]      ub_up : [H, dk, rank]
 *   state       : [B, H, dv, dk] fp32   mean : [B, H, dv] fp32
 * Returns CARVE_OK, CARVE_EINVAL or CARVE_EUNSUPPORTED. Makes no HIP call. */
int carve_recurrent_ref_shapes(const carve_config* cfg, carve_shapes* out);

/* Forward pass of the CARVE layer (see the header comment for the math).
 *   q, k       [B,T,H,dk] dtype   query and key (used as given: no scaling)
 *   v          [B,T,H,dv] dtype   value
 *   g          [B,T,H,dk] dtype   log-decay, expected <= 0; with
 *                                 CARVE_DECAY_LOGITS the raw decay logits
 *   bx         [B,T,H,dk] dtype   erase logit
 *   w          [B,T,H]    dtype   scalar write gate
 *   ub_down    [H,rank,dv] dtype, ub_up [H,dk,rank] dtype: U_b = ub_up @ ub_down
 *              per head. Ignored when rank == 0; required when rank > 0.
 *   state_in   [B,H,dv,dk] fp32 or NULL (zeros)
 *   mean_in    [B,H,dv] fp32 or NULL (zeros): the mean that gates chunk 0
 *   o          [B,T,H,dv] dtype   output; must not overlap any input
 *   state_out  [B,H,dv,dk] fp32 or NULL (not written); may equal state_in
 *   mean_out   [B,H,dv] fp32 or NULL (not written); may equal mean_in. It
 *              receives the mean of the last (possibly partial) chunk, or
 *              mean_in when T == 0.
 *   workspace  device scratch of at least shapes.workspace_bytes (may be NULL
 *              when that is 0)
 *   stream     hipStream_t as void*
 * B, H or T may be 0 (nothing to compute; with T == 0 the state and mean pass
 * through). T need not be a multiple of L.
 * The chunk-parallel state pass hands block states between the waves of a
 * workgroup through LDS with bounded waits. A wait that runs out (none has
 * ever been observed; it would take a hardware fault) writes NaN to the
 * affected output tiles, state and mean instead of hanging; the call still
 * returns CARVE_OK, since the kernels run after it returns. */
int carve_chunk_fwd(const carve_config* cfg,
                    const void* q, const void* k, const void* v,
                    const void* g, const void* bx, const void* w,
                    const void* ub_down, const void* ub_up,
                    const float* state_in, const float* mean_in,
                    void* o, float* state_out, float* mean_out,
                    void* workspace, size_t workspace_bytes, void* stream);

/* carve_chunk_fwd without a workspace argument, for callers that cannot
 * allocate device memory: code recorded under HIP graph capture, tight
 * serving loops, harnesses that forbid allocation. Arguments and results are
 * those of carve_chunk_fwd (bit for bit: the same kernels run). The library
 * allocates nothing for the call: where a schedule needs workspace (bf16 with
 * no content projection: the two-launch pair's block images), it uses a fixed
 * 64 MiB device array that every GPU the library runs on holds until the
 * process ends. A problem that needs more (shapes.workspace_bytes > 64 MiB,
 * e.g. more than 2048 (batch, head, 64-token block) triples at dk = dv = 64)
 * is CARVE_EWORKSPACE, before any HIP call. All calls on one GPU share that
 * array, so calls that overlap in time on one GPU (other streams, other host
 * threads) race and must be serialised by the caller. */
int carve_chunk_fwd_noalloc(const carve_config* cfg,
                            const void* q, const void* k, const void* v,
                            const void* g, const void* bx, const void* w,
                            const void* ub_down, const void* ub_up,
                            const float* state_in, const float* mean_in,
                            void* o, float* state_out, float* mean_out, void* stream);

/* Backward pass: gradients of a scalar loss with respect to every input of
 * carve_chunk_fwd, from its gradients with respect to the outputs. The pages
 * train the layer but give no backward pass; these are the exact derivatives
 * of the recurrence in the header comment through every path it has: the
 * stale chunk mean m_{c-1} that gates chunk c passes gradient back to chunk
 * c-1's outputs (and to mean_in for chunk 0), and U_down, U_up receive
 * theirs through the erase gate.
 *   cfg, q .. mean_in   exactly as given to carve_chunk_fwd (the forward pass
 *                       is recomputed; nothing from it is kept)
 *   d_o         [B,T,H,dv] dtype   gradient of o (required when B T H > 0)
 *   d_state_out [B,H,dv,dk] fp32 or NULL (zeros)
 *   d_mean_out  [B,H,dv] fp32 or NULL (zeros)
 *   dq, dk, dg, dbx [B,T,H,dk], dv [B,T,H,dv], dw [B,T,H]: dtype, written.
 *               With CARVE_DECAY_LOGITS, dg is the gradient of the raw logit.
 *   d_ub_down [H,rank,dv], d_ub_up [H,dk,rank]: fp32, written (summed over
 *               the batch); required when rank > 0 and H > 0
 *   d_state_in [B,H,dv,dk], d_mean_in [B,H,dv]: fp32 or NULL (not written).
 *               They may be the same buffers as d_state_out and d_mean_out.
 *   workspace   at least shapes.bwd_workspace_bytes of device scratch: the
 *               state at every chunk start and one chunk's recomputed states,
 *               4 (nc + L) dk dv bytes per (batch, head) at dk = 128 with a
 *               projection, 4 (nc + ceil(L / 8)) dk dv otherwise, plus small
 *               vectors;
 *               with rank == 0 also every token's per-slice column sums,
 *               4 T (dk / 16) (4 dk + 1) bytes per (batch, head); in bf16
 *               with rank == 0 and L a multiple of 64, also the forward
 *               pair's block images and an output, since the chunk-start
 *               states then come from the forward's chunk-parallel state pass;
 *               the chunks are then walked in up to 16 groups at once, which
 *               takes one chunk's recomputed states per group and the state
 *               gradient at every chunk end, 4 (G ceil(L / 8) + nc) dk dv
 *               bytes per (batch, head) in place of 4 ceil(L / 8) dk dv (the
 *               row-lane schedules keep the state at every 8-token sub-block
 *               start rather than at every token; 4 L dk dv at dk = 128 with
 *               a projection). In bf16 with rank == 0, dk = 64 and without
 *               CARVE_QK_L2NORM (any L), every 64-token block is
 *               differentiated at once from its start state and its
 *               end-of-block state gradient (dense products per block); the
 *               workspace then holds only those two per block and a row share
 *               of d_mean_out, 4 (2 nb dk dv + dv) bytes per (batch, head)
 *               with nb = ceil(T / 64), besides the forward pair's images and
 *               output
 * No output may overlap an input, another output or the workspace, except
 * for the two aliases above. Results are deterministic (no atomics).
 * Returns the status codes of carve_chunk_fwd. */
int carve_chunk_bwd(const carve_config* cfg,
                    const void* q, const void* k, const void* v,
                    const void* g, const void* bx, const void* w,
                    const void* ub_down, const void* ub_up,
                    const float* state_in, const float* mean_in,
                    const void* d_o, const float* d_state_out, const float* d_mean_out,
                    void* dq, void* dk, void* dv, void* dg, void* dbx, void* dw,
                    float* d_ub_down, float* d_ub_up, float* d_state_in, float* d_mean_in,
                    void* workspace, size_t workspace_bytes, void* stream);

/* One decode step: the token recurrence of the header comment for a single
 * token of every (batch, head), for serving loops that produce one token at a
 * time. The caller carries three fp32 tensors from step to step:
 *   state      [B,H,dv,dk]  S before this token; updated in place
 *   mean_prev  [B,H,dv]     the mean of the previous chunk's outputs, which
 *                           gates this token (section 2.1: one chunk stale);
 *                           replaced by this chunk's mean at its last position
 *   chunk_acc  [B,H,dv]     sum of this chunk's outputs before this token; the
 *                           token's output is added, and it restarts from zero
 *                           after the chunk's last position
 * and `pos`, the token's position within its chunk (0 <= pos < L). Stepping
 * tokens t = 0, 1, ... with pos = t mod L from (state_in, mean_in, zeros)
 * gives carve_chunk_fwd's outputs and final state; after a whole chunk,
 * mean_prev holds its mean (for a partial last chunk, carve_chunk_fwd's
 * mean_out is chunk_acc divided by the tokens it holds).
 *   cfg        B, H, dk, dv, L, rank, dtype as for carve_chunk_fwd; T must be 1
 *   q, k, g, bx [B,H,dk] dtype; v [B,H,dv] dtype; w [B,H] dtype: this token
 *              ([B,1,H,.] in the layout of carve_chunk_fwd)
 *   ub_down, ub_up as for carve_chunk_fwd
 *   o          [B,H,dv] dtype: this token's output
 * state, mean_prev and chunk_acc are required (when B H > 0); none of o,
 * state, mean_prev and chunk_acc may overlap each other or an input. Returns
 * CARVE_EINVAL for T != 1, pos outside [0, L), a missing pointer or an
 * overlap, and the status codes of carve_chunk_fwd otherwise. Needs no
 * workspace. */
int carve_recurrent_step(const carve_config* cfg, int32_t pos,
                         const void* q, const void* k, const void* v,
                         const void* g, const void* bx, const void* w,
                         const void* ub_down, const void* ub_up,
                         float* state, float* mean_prev, float* chunk_acc,
                         void* o, void* stream);

/* ---------------------------------------------------------------------------
 * The attention layer beside the mixer. The paper's hybrid model puts
 * sliding-window attention layers between CARVE layers; these entry points are
 * that layer's operators: the norm and rotation of queries and keys with their
 * gradients, a paged cache of keys and values, and attention of new tokens over
 * it. A prompt chunk and a single token are one call each, as chunk_fwd with a
 * carried state and recurrent_step are for the mixer.
 *
 * The conventions above hold, except that these tensors may have strides: the
 * d channels of a head are contiguous, a token's heads follow each other, and
 * the `*_row` fields give the elements from one token to the next (so q and k
 * can be parts of one projection's output). Every stride is a multiple of 16
 * bytes and below 2^31 elements. d is 64 or 128.
 * CARVE_EUNSUPPORTED also stands for calls larger than the launches take: more
 * than 2^26 - 4 tokens to norm, rotate or append, 2^31 rows (tokens x heads), or,
 * with few rows a sequence, 2^31 blocks of 128 keys over all heads and sequences
 * at the longest lengths that the table and window allow. */

/* Bits of carve_rope_config.flags and carve_paged_config.flags.
 *   CARVE_ROPE_INTERLEAVED  a rotated pair is channels (2i, 2i + 1); without it
 *                           (i, i + rot / 2)
 *   CARVE_ROPE_NORM         divide each row by its root mean square (and multiply
 *                           by the weights, where given) before the rotation
 *   CARVE_PAGED_STEP        every sequence has exactly one new token (N == S) and
 *                           `cu` is not read */
enum { CARVE_ROPE_INTERLEAVED = 1, CARVE_ROPE_NORM = 2, CARVE_PAGED_STEP = 4 };

typedef struct {
  int64_t N;                /* tokens */
  int64_t q_row, k_row;     /* q, k: elements from one token to the next */
  int64_t qo_row, ko_row;   /* q_out, k_out; in the backward d_q_out, d_k_out */
  int64_t dq_row, dk_row;   /* dq, dk (backward only) */
  int32_t T;                /* without positions, token n stands at n mod T */
  int32_t Hq, Hk, d;
  int32_t rot;              /* rotated channels: a multiple of 16 up to d, 0 for none */
  int32_t table_len;        /* rows of cos and sin */
  int32_t dtype, flags;
  float eps;                /* under the root; with CARVE_ROPE_NORM a normal number > 0 */
} carve_rope_config;

/* Norm and rotation of queries and keys in one pass. For each head x of each
 * token at position p:  y = R(p) (x / sqrt(mean(x^2) + eps) * weight), summed in
 * fp32 and rounded once.
 *   q [N,Hq,d], k [N,Hk,d] dtype, rows q_row and k_row apart
 *   q_weight, k_weight [d] dtype or NULL (ones); only with CARVE_ROPE_NORM
 *   cos, sin [table_len, rot/2] fp32: the angles' cosines and sines per position
 *   positions [N] int32 or NULL. A position outside [0, table_len) gives NaN in
 *               the rotated channels.
 *   q_out, k_out  dtype; each may be its input itself (same rows) */
int carve_qk_norm_rope_fwd(const carve_rope_config* cfg, const void* q, const void* k, const void* q_weight,
                           const void* k_weight, const float* cos, const float* sin, const int32_t* positions,
                           void* q_out, void* k_out, void* stream);

/* Bytes of workspace carve_qk_norm_rope_bwd needs (0 without weights; `weights`
 * says whether either weight is given). */
int carve_qk_norm_rope_workspace(const carve_rope_config* cfg, int32_t weights, int64_t* bytes);

/* Gradients of carve_qk_norm_rope_fwd's inputs. q, k and what follows them as
 * given to the forward pass; d_q_out, d_k_out the gradients of its outputs.
 *   dq, dk      dtype; each may be its d_*_out or its input itself (same rows)
 *   dq_weight, dk_weight [d] fp32, required with the weight, summed over tokens
 *               and heads in a fixed order (no atomics) */
int carve_qk_norm_rope_bwd(const carve_rope_config* cfg, const void* q, const void* k, const void* q_weight,
                           const void* k_weight, const float* cos, const float* sin, const int32_t* positions,
                           const void* d_q_out, const void* d_k_out, void* dq, void* dk, float* dq_weight,
                           float* dk_weight, void* workspace, size_t workspace_bytes, void* stream);

/* A paged cache and the sequences of one call.
 * Token t of sequence s is entry t mod page_size of page table[s][t / page_size]
 * of k_cache and v_cache; page, token and head strides are free (so one tensor
 * can hold both caches, heads may come before tokens, ...).
 * The N new tokens are packed: sequence s has the tokens cu[s] .. cu[s+1] - 1,
 * the last of its kv_lens[s] tokens (the length counts the new ones, a negative
 * one is 0). cu does not decrease and starts at 0; tokens from cu[S] on belong to
 * no sequence and their outputs are left as they were. Lengths and pages are read
 * on the device, so a captured graph follows them. */
typedef struct {
  int32_t N, S;                      /* new tokens, sequences */
  int32_t Hq, Hk, d;                 /* Hq = G Hk; query head h reads head h / G (append: Hq = 0 without q) */
  int32_t page_size, pages, width;   /* page_size a power of two; table [S, width], width * page_size <= 2^30 */
  int32_t rot, table_len;            /* append: as in carve_rope_config */
  int32_t window;                    /* attention: keys a token sees, itself included; 0 for all before it */
  int32_t dtype, flags;
  float eps;                         /* append, with CARVE_ROPE_NORM */
  float scale;                       /* attention: 0 < scale <= 16 */
  int64_t q_row, k_row, v_row;       /* elements from one new token to the next */
  int64_t o_row;                     /* of attention's o and of append's q_out */
  int64_t table_row;                 /* entries from one sequence's table row to the next's */
  int64_t kc_page, kc_tok, kc_head;  /* strides of k_cache in elements */
  int64_t vc_page, vc_tok, vc_head;  /* strides of v_cache */
} carve_paged_config;

/* Stores the new tokens' keys and values in the cache; the keys (and q, where
 * given) are normed and rotated on the way as by carve_qk_norm_rope_fwd at the
 * tokens' positions kv_lens[s] - n_s + i.
 *   k, v [N,Hk,d], q [N,Hq,d] or NULL (Hq = 0); q_out may be q itself
 * A token whose position is negative or lies past the table, or whose page
 * number is outside [0, pages), is not stored. No page may be shared by two
 * sequences that store to it, and no two entries of the caches may overlap
 * (refused, between the two caches only where their strides are the same). */
int carve_paged_append(const carve_paged_config* cfg, const void* k, const void* v, const void* q,
                       const void* q_weight, const void* k_weight, const float* cos, const float* sin,
                       const int32_t* cu, const int32_t* kv_lens, const int32_t* table, void* k_cache, void* v_cache,
                       void* q_out, void* stream);

/* Bytes of workspace carve_paged_attention needs for this configuration. */
int carve_paged_workspace(const carve_paged_config* cfg, int64_t* bytes);

/* Attention of the new tokens over the cache (which holds them already): a token
 * at position p sees the keys j <= p with j > p - window.
 *   o = softmax(scale q k^T) v,   lse = log sum exp(scale q k^T)
 *   q [N,Hq,d], o [N,Hq,d] dtype (o overlaps no input); lse [N,Hq] fp32 or NULL;
 *   the caches have at least one page
 * Softmax statistics and sums are fp32; in bf16 the weights enter the product with
 * v as one bf16 number (off by at most 2^-8 of each), or as two (2^-16) where the
 * call has few rows (tokens x grouped heads) per sequence. A token that sees no key
 * (a negative position) has o = 0 and lse = -inf. Keys whose page number is outside
 * [0, pages) or past the table are not seen, and neither is a key whose score q k is
 * -inf; a finite score counts, however large. What is not seen does not matter,
 * infinities and NaN included.
 * The workspace may be shared by calls that do not overlap in time. Results are
 * deterministic (no atomics): a call with the same sizes and inputs gives the same
 * bits. The kernel is chosen for the whole call from its sizes, so a sequence's last
 * bits, and in bf16 the rounding of its weights, may depend on what it is batched
 * with; single tokens and a long prompt chunk are faster in calls of their own. */
int carve_paged_attention(const carve_paged_config* cfg, const void* q, const void* k_cache, const void* v_cache,
                          const int32_t* cu, const int32_t* kv_lens, const int32_t* table, void* o, float* lse,
                          void* workspace, size_t workspace_bytes, void* stream);

/* ---------------------------------------------------------------------------
 * A paged cache in 4 bits. The attention layers hold the only state of a hybrid
 * that grows with the context; held in 4 bits it takes 17/64 of the bf16 cache's
 * bytes, and a decode step reads that much less. Sequences, lengths and block
 * tables are those of the calls above.
 *
 * A head's d channels are d / 32 blocks of 32. A block is 32 codes of 4 bits (a sign,
 * two bits of exponent, one of mantissa: 0, 0.5, 1, 1.5, 2, 3, 4, 6), two to a byte
 * with the even channel in the low half, and one byte e, its scale 2^(e - 127); 255
 * makes every value of the block NaN. With 2 <= e <= 252, all that is ever stored, a value
 * is a normal number or 0 and exact in bf16; what other bytes give is not defined.
 *   codes   uint8 [pages, page_size, Hk, d / 2]
 *   scales  uint8 [pages, page_size, Hk, d / 32]
 * for keys and for values; a head's bytes are contiguous, page, token and head strides
 * free. Reading is fastest where a head's tokens of a page follow each other. */

/* carve_paged_config with kc_* and vc_* in bytes of the codes (multiples of 16, below
 * 2^31), and the scales' strides in bytes (multiples of d / 32, below 2^31). `dtype` is
 * that of q, k, v and o. Codes are 16-byte aligned, scales 4-byte aligned. */
typedef struct {
  carve_paged_config paged;
  int64_t ks_page, ks_tok, ks_head;
  int64_t vs_page, vs_tok, vs_head;
} carve_fp4_config;

/* carve_paged_append into such a cache. A block takes the smallest scale 2^e with
 * max |x| <= 7 2^e, -125 <= e <= 125; a value becomes the nearest code, the even one of
 * two, at most 6: it is off by at most 2^e (by more only where |x| > 7 2^125), and by at
 * most 2^e / 4 where |x| <= 2^(e+1). A block with an infinity or NaN is stored as NaN
 * (codes 0). The keys are normed and rotated on the way where that is asked for, rounded to
 * `dtype` as by carve_qk_norm_rope_fwd, and that is what is stored in 4 bits. The same refusals hold;
 * codes and scales of keys and values may share one allocation. */
int carve_paged_append_fp4(const carve_fp4_config* cfg, const void* k, const void* v, const void* q,
                           const void* q_weight, const void* k_weight, const float* cos, const float* sin,
                           const int32_t* cu, const int32_t* kv_lens, const int32_t* table, uint8_t* k_codes,
                           uint8_t* k_scales, uint8_t* v_codes, uint8_t* v_scales, void* q_out, void* stream);

/* The values that cache entries stand for: row n of k and v [N,Hk,d] dtype (rows
 * paged.k_row and paged.v_row apart) from entry slots[n] % page_size of page
 * slots[n] / page_size. A slot outside [0, pages page_size) gives zeros. Either of k
 * and v may be NULL with its codes and scales. Of paged N, Hk, d, page_size, pages,
 * dtype, k_row, v_row and the caches' strides say what is read; the other fields are
 * checked as by the calls above, so 0 in them is right, and CARVE_PAGED_STEP with
 * another S than N is refused. N at most 2^26 - 4, k and v together at most 2^38 - 2^14
 * bytes (CARVE_EUNSUPPORTED beyond). */
int carve_paged_read_fp4(const carve_fp4_config* cfg, const uint8_t* k_codes, const uint8_t* k_scales,
                         const uint8_t* v_codes, const uint8_t* v_scales, const int64_t* slots, void* k, void* v,
                         void* stream);

/* Bytes of workspace carve_paged_attention_fp4 needs for this configuration. */
int carve_paged_workspace_fp4(const carve_fp4_config* cfg, int64_t* bytes);

/* carve_paged_attention over such a cache: what that call says holds, its results those
 * over the values that the codes stand for (the products take them as they are, bf16
 * with fp32 sums, or fp32). */
int carve_paged_attention_fp4(const carve_fp4_config* cfg, const void* q, const uint8_t* k_codes,
                              const uint8_t* k_scales, const uint8_t* v_codes, const uint8_t* v_scales,
                              const int32_t* cu, const int32_t* kv_lens, const int32_t* table, void* o, float* lse,
                              void* workspace, size_t workspace_bytes, void* stream);

/* Room in a paged cache, of either kind, for the next tokens of S requests: block table,
 * lengths, offsets, positions and slots, all worked out on the device, so that a captured
 * step goes on from the last one's results.
 *   old_s = 0 where the request has ended (done[s] != 0), else kv_lens[s]
 *   kv_lens_out[s] = old_s + new_lens[s];  cu[s + 1] = cu[s] + new_lens[s], cu[0] = 0
 * Negative lengths count as 0, sums stop at 2^31 - 1.
 *   free_pages [capacity]  a stack: entries [0, free_count[0]) are pages nobody holds
 *   free_count [2]         pages free; pages that were lacking so far
 * First the pages of ended requests (the table entries >= 0 of their kv_lens[s] tokens)
 * go on top of the stack, in the order of requests and entries; what would pass its
 * capacity is lost. Then every request takes from the top what it needs for its tokens
 * beyond ceil(old_s / page_size) pages, in the same order, and its table entries are
 * written (entries past the table's width are not, and take nothing). Where the stack is
 * empty the entry is -1 and free_count_out[1] counts one more; such tokens have no slot
 * and neither are they stored or seen. A page that several requests hold is the caller's
 * to keep out of ended ones. Table entries past ceil(old_s / page_size) are taken for
 * empty and written over: a caller that sets a length back (tokens that were drafted and
 * rejected) first puts the pages past it on the stack itself, or they are lost.
 *   positions [N]  of token cu[s] + i: old_s + i; 0 behind cu[S]
 *   slots [N]      page page_size + position mod page_size, or -1 without a page and
 *                  behind cu[S]
 * Either of the two may be NULL. kv_lens_out may be kv_lens and free_count_out
 * free_count; no other output overlaps anything. */
typedef struct {
  int32_t S, N;
  int32_t page_size, width;          /* page_size a power of two; width * page_size <= 2^30, S * width < 2^31 */
  int64_t table_row;                 /* entries from one request's table row to the next's */
  int64_t capacity;                  /* of free_pages, below 2^31 */
} carve_assign_config;
int carve_paged_assign(const carve_assign_config* cfg, const int32_t* kv_lens, const int32_t* new_lens,
                       const int32_t* done, int32_t* table, int32_t* free_pages, const int32_t* free_count,
                       int32_t* kv_lens_out, int32_t* cu, int32_t* positions, int64_t* slots, int32_t* free_count_out,
                       void* stream);

/* Static text for a status code. For CARVE_EHIP it returns the HIP error text
 * of the most recent failure on the calling thread. */
const char* carve_error_string(int code);

#ifdef __cplusplus
}
#endif
#endif /* CARVE_H */
