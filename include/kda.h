/*
 * kda.h - C ABI of the GB300 Kimi Delta Attention (KDA) library.
 *
 * KDA is the gated delta-rule recurrence, per sequence n and head h, over tokens t:
 *
 *   log a_t = -5 * sigmoid(exp(A_h) * z_t)       (a vector over d_k; bounded decay,
 *                                                 'From Linear Attention to KDA', §5.4)
 *   beta_t  = sigmoid(b_t)                       (a scalar; same page, §5.3)
 *   S_t     = (I - beta_t k_t k_t^T) Diag(a_t) S_{t-1} + beta_t k_t v_t^T
 *   o_t     = S_t^T q_t                          (same page, §5.2; 'Kimi K3 attention deep
 *                                                 dive', §2.1; 'Kimi K3', section
 *                                                 "Kimi Delta Attention")
 *
 * S is a d_k x d_v fp32 matrix (row index = key channel). The library supports
 * d_k = d_v = 128 only. Inputs arrive already projected: q and k L2-normalised by the
 * caller, z and b the raw pre-activations of the decay and write-strength gates.
 * No 1/sqrt(d_k) scale is applied to q.
 *
 * Conventions for every entry point
 *   - Pointers named "device" are CUDA device pointers owned by the caller. The library
 *     allocates nothing and keeps no pointer after the call returns.
 *   - bf16 tensors are passed as uint16_t bit patterns (IEEE bfloat16).
 *   - Layouts are dense row-major with the last dimension contiguous.
 *   - 'stream' is a cudaStream_t (NULL = the legacy default stream). Work is enqueued
 *     asynchronously; a return of KDA_OK means the arguments were valid and the
 *     kernels were launched, not that they have finished.
 *   - The compute entry points only enqueue kernels on 'stream' (no allocation, copy or
 *     synchronisation), so they can be captured into a CUDA graph and replayed; a
 *     replay gives the bits of the same call made directly. The first call of a process
 *     sets kernel attributes and reads the device's properties: make one call before the
 *     first capture. kda_workspace_status synchronises and cannot be captured.
 *   - Errors are returned as kda_status codes; nothing is thrown across the ABI and no
 *     kernel traps. A failed argument check launches nothing and writes nothing.
 *   - Every pointer must be 16-byte aligned (the kernels use 128-bit accesses);
 *     the prefill workspace must be 256-byte aligned.
 */
#ifndef KDA_H_
#define KDA_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    KDA_OK = 0,
    KDA_ERR_NULL = -1,        /* a required pointer is NULL */
    KDA_ERR_SHAPE = -2,       /* a size is negative or inconsistent, or beyond the launch
                                 limits: num_seqs x num_heads >= 2^31, num_heads > 65535, or
                                 (prefill) chunk slots x num_heads >= 2^31 */
    KDA_ERR_UNSUPPORTED = -3, /* d_k or d_v other than 128, or an unknown output dtype */
    KDA_ERR_SEQLENS = -4,     /* cu_seqlens not rising from 0 to the token count */
    KDA_ERR_ALIGN = -5,       /* a pointer is not 16-byte (workspace: 256-byte) aligned */
    KDA_ERR_WORKSPACE = -6,   /* workspace smaller than kda_chunk_prefill_workspace_size() */
    KDA_ERR_CUDA = -7,        /* a CUDA launch or API call failed */
    KDA_ERR_DEVICE = -8,      /* the device lacks what the kernels need (sm_103a, smem) */
    KDA_ERR_PAGES = -9        /* a page id outside the cache or the pool */
} kda_status;

/* Output element type of the prefill. */
typedef enum {
    KDA_OUT_BF16 = 0, /* o rounded to bf16 (round to nearest even) */
    KDA_OUT_F32 = 1   /* o kept in fp32 */
} kda_out_dtype;

/* Short English text for a status code (static storage; never NULL). */
const char *kda_status_string(int status);

/* Library version, major * 10000 + minor * 100 + patch. */
int kda_version(void);

/*
 * Test hook for the state walk's failure path (no counterpart on the pages). On the
 * current device, every later kda_chunk_prefill call leaves out the MMA-completion signal
 * of chunk slot skip_commit_chunk in its state walks (-1: none; -2 - j: that of map j of
 * the map chain that a segmented walk's output walks run first, j = 0 the first), and
 * every wait of the walk gives up after wait_limit_ns nanoseconds of the GPU clock
 * (default 2e9). A walk
 * whose wait gives up skips the rest of its work, writes NaN into its final state and
 * sets the workspace status word to KDA_ERR_CUDA (see kda_workspace_status); no GPU fault
 * is involved and the context stays usable. Restore with (-1, 2000000000) before normal
 * use. The setting is global to the device and the process and not synchronised with
 * work in flight: call it with the device idle.
 *
 * Returns KDA_OK, KDA_ERR_SHAPE for wait_limit_ns == 0, or KDA_ERR_CUDA.
 */
int kda_debug_walk_fault(int32_t skip_commit_chunk, uint64_t wait_limit_ns);

/*
 * Test hook for the segmented walk's long end segments (no counterpart on the pages).
 * When a kda_chunk_prefill call takes the segmented walk with a combine kernel (walk
 * form 2, see kda_chunk_prefill_walk_form), a sequence of at least (2 E + 1) P chunks
 * (P the segment length the sizes give) is cut into a first and a last segment of E P
 * chunks and segments of P chunks between them; the sizes choose E themselves (1 = every segment P chunks), and
 * end_factor > 0 forces E = end_factor on every later call in this process (0 restores
 * the sizes' choice). The segment length, the workspace size and the launch count do not
 * change; only the cut of each sequence does, so the results agree with E = 1 up to
 * rounding. Process-global and not synchronised with calls in flight.
 *
 * Returns KDA_OK, or KDA_ERR_SHAPE for end_factor outside [0, 64].
 */
int kda_debug_segment_ends(int32_t end_factor);

/*
 * Bytes of device workspace kda_chunk_prefill() needs for a batch of total_tokens
 * tokens in num_seqs sequences and num_heads heads. The size is an upper bound that
 * depends only on these three numbers, so one buffer serves every batch up to them.
 * Returns 0 for negative arguments.
 */
size_t kda_chunk_prefill_workspace_size(int64_t total_tokens, int32_t num_seqs, int32_t num_heads);

/*
 * Number of kernels one kda_chunk_prefill() call with these sizes launches on its
 * stream: 0 when num_seqs is 0, 3 (plan, intra-chunk, state walk) when every
 * (sequence, head) chain walks its chunks in one pass, 5 when the chains are too few to
 * fill the GPU and the walk is split into segments: plan, intra-chunk, segment-map walk,
 * then either a second intra-chunk launch beside the map walk (the chained form, see
 * kda_chunk_prefill_walk_form) or a combine kernel, and the output walk. Depends only on
 * the three sizes, like the workspace. Returns -1 for negative arguments.
 */
int32_t kda_chunk_prefill_launch_count(int64_t total_tokens, int32_t num_seqs, int32_t num_heads);

/*
 * How a kda_chunk_prefill() call with these sizes walks the state: 0 in one pass per
 * (sequence, head) chain; 1 in segments whose output walks first chain the segment maps
 * before them on the tensor cores (every output walk fits in one wave of the GPU); 2 in
 * segments whose input states a combine kernel chains. In form 1 the intra-chunk items
 * past a whole number of rounds of the GPU's SMs that belong to the last segment of a
 * dense batch's last sequence run in a second intra-chunk launch beside the map walk.
 * Depends only on the three sizes. Returns -1 for negative arguments, 0 when num_seqs is 0.
 */
int32_t kda_chunk_prefill_walk_form(int64_t total_tokens, int32_t num_seqs, int32_t num_heads);

/*
 * kda_chunk_prefill - chunkwise-parallel KDA over whole sequences.
 *
 * Computes, for every sequence and head, all outputs o_t and the final state S_T of the
 * recurrence above, starting from initial_state. The work is the chunkwise form of
 * 'From Linear Attention to KDA', §7 (chunks of 64 tokens: per-chunk decayed K K^T and
 * Q K^T matrices, the UT/WY triangular solve that turns the chain of delta updates
 * into dense products, then a serial pass that carries S from chunk to chunk), with
 * the 16-token tiles of §8 inside each chunk. The gate and beta are computed from
 * z, A, b inside the kernels.
 *
 * Batch layouts (tokens packed row by row):
 *   dense   : cu_seqlens == NULL. batch sequences of seq_len tokens each; num_seqs must
 *             equal batch. Token (i, t) is row i * seq_len + t.
 *   varlen  : cu_seqlens != NULL. batch must be 1; seq_len is the total token count;
 *             sequence n owns rows cu_seqlens[n] .. cu_seqlens[n+1]-1. Empty sequences
 *             are allowed (their final state equals their initial state).
 *
 * Arguments (T_total = batch * seq_len rows, H = num_heads):
 *   q, k        device bf16 [T_total, H, 128]   queries, L2-normalised keys
 *   v           device bf16 [T_total, H, 128]   values
 *   z           device fp32 [T_total, H, 128]   decay pre-activation
 *   A           device fp32 [H]                 per-head log scale of the decay gate
 *   b           device fp32 [T_total, H]        write-strength pre-activation
 *   initial_state device fp32 [num_seqs, H, 128, 128] or NULL (zeros)
 *   cu_seqlens  device int32 [num_seqs + 1] or NULL (dense layout)
 *   cu_seqlens_host  host int32 [num_seqs + 1] or NULL. When given it must hold the same
 *               values as cu_seqlens; it is validated on the host before anything is
 *               launched (KDA_ERR_SEQLENS). Without it, cu_seqlens is validated on the
 *               device: a bad table makes the kernels fill final_state with NaN, leave o
 *               untouched, and record KDA_ERR_SEQLENS for kda_workspace_status().
 *   o           device [T_total, H, 128], bf16 or fp32 per o_dtype (written)
 *   final_state device fp32 [num_seqs, H, 128, 128] (written). May alias initial_state.
 *   workspace   device scratch of at least kda_chunk_prefill_workspace_size() bytes,
 *               256-byte aligned. Its contents need no initialisation and are dead after
 *               the kernels finish, except the status word read by kda_workspace_status().
 *   stream      cudaStream_t
 *
 * Calls that share a workspace must be ordered on one stream.
 */
int kda_chunk_prefill(const uint16_t *q, const uint16_t *k, const uint16_t *v,
                      const float *z, const float *A, const float *b,
                      const float *initial_state,
                      const int32_t *cu_seqlens, const int32_t *cu_seqlens_host,
                      int32_t batch, int64_t seq_len, int32_t num_seqs, int32_t num_heads,
                      int32_t d_k, int32_t d_v,
                      void *o, int32_t o_dtype, float *final_state,
                      void *workspace, size_t workspace_bytes, void *stream);

/*
 * Status recorded on the device by the last kda_chunk_prefill() that used this
 * workspace. Synchronises 'stream'. Returns
 *   KDA_OK           the kernels ran to the end;
 *   KDA_ERR_SEQLENS  the device-side cu_seqlens check failed (final_state is NaN);
 *   KDA_ERR_CUDA     a bounded wait inside the state walk gave up (a copy or a tensor-core
 *                    group did not complete in time); the final states of the affected
 *                    (sequence, head) pairs are NaN and their outputs are not valid;
 *   or KDA_ERR_CUDA if the copy of the status word itself fails.
 */
int kda_workspace_status(const void *workspace, void *stream);

/*
 * kda_chunk_prefill_noalloc - the same prefill, for callers that cannot allocate.
 *
 * The pages have no counterpart to this entry point; it exists for callers that cannot
 * provide the device workspace kda_chunk_prefill() asks for: a plugin running inside an
 * engine that owns all device memory and passes it only the call's tensors, or code on
 * a latency-critical path where cudaMalloc, which may synchronise the whole device, is
 * not allowed. Instead of a workspace it uses a scratch area of
 * KDA_NOALLOC_SCRATCH_BYTES compiled into the library: a static device array that exists
 * on every GPU that loads the library, from load until process exit. The library still
 * allocates nothing at call time. Arguments, results and error codes are those of
 * kda_chunk_prefill() without the two workspace arguments; inputs and outputs are still
 * the caller's.
 *
 *   - A batch whose workspace (kda_chunk_prefill_workspace_size(total_tokens, num_seqs,
 *     num_heads)) exceeds KDA_NOALLOC_SCRATCH_BYTES is refused with KDA_ERR_WORKSPACE
 *     before anything is launched. 64 MiB holds, for example, 3072 tokens x 8 heads or
 *     2048 tokens x 12 heads.
 *   - The first call on a device looks up the scratch's device address on that device
 *     (cudaGetSymbolAddress, with the device current); make that first call before any
 *     stream capture. The address is kept for the life of the process, so do not use
 *     this entry point after cudaDeviceReset() on that device: the reset unloads the
 *     library's device code and the kept address no longer names the scratch.
 *   - All calls share the one scratch area and it keeps the last call's contents. The
 *     kernels need nothing in it to start at zero, but calls whose GPU work overlaps in
 *     time (different streams, or threads without ordering) race on it: order them.
 *   - The device-side cu_seqlens check still fills final_state with NaN on a bad table;
 *     there is no workspace to pass to kda_workspace_status(), so pass cu_seqlens_host
 *     to have the table checked on the host instead.
 */
#define KDA_NOALLOC_SCRATCH_BYTES ((size_t)64 << 20)
int kda_chunk_prefill_noalloc(const uint16_t *q, const uint16_t *k, const uint16_t *v,
                              const float *z, const float *A, const float *b,
                              const float *initial_state,
                              const int32_t *cu_seqlens, const int32_t *cu_seqlens_host,
                              int32_t batch, int64_t seq_len, int32_t num_seqs, int32_t num_heads,
                              int32_t d_k, int32_t d_v,
                              void *o, int32_t o_dtype, float *final_state, void *stream);

/*
 * kda_recurrent_decode - one token per sequence, the recurrence applied in place.
 *
 * For every sequence n and head h: read S = state[n, h], apply
 *   S' = Diag(a) S;  p = S'^T k;  S = S' + beta k (v - p)^T;  o = S^T q
 * (the three-step diagonal-plus-low-rank update of 'Kimi K3 attention deep dive', §2.2;
 * the error form of 'Kimi K3', section "Kimi Delta Attention"), write S back and o out.
 * All arithmetic is fp32.
 *
 * Arguments (N = num_seqs, H = num_heads):
 *   q, k, v   device bf16 [N, H, 128]
 *   z         device fp32 [N, H, 128]
 *   A         device fp32 [H]
 *   b         device fp32 [N, H]
 *   state     device fp32 [N, H, 128, 128], read and overwritten in place
 *   o         device fp32 [N, H, 128] (written)
 *   stream    cudaStream_t
 */
int kda_recurrent_decode(const uint16_t *q, const uint16_t *k, const uint16_t *v,
                         const float *z, const float *A, const float *b,
                         float *state, float *o,
                         int32_t num_seqs, int32_t num_heads, int32_t d_k, int32_t d_v,
                         void *stream);

/* Most draft tokens one kda_recurrent_verify() or kda_replay_fold() call takes. */
#define KDA_MAX_REPLAY_TOKENS 16

/*
 * kda_recurrent_verify - several tokens per sequence from a checkpoint state, with the
 * gate values logged for a later replay (ReplaySSM, 'Kimi K3 attention deep dive', §6.2).
 *
 * For every sequence n and head h, starting from S = state[n, h], the decode update of
 * kda_recurrent_decode() is applied to the m tokens of the sequence in order, and each
 * token's output o = S^T q (after its own write) is written. The checkpoint `state` is
 * only read. With state_out = state this is multi-token decode in place.
 *
 * Token t of sequence n is row n * m + t of the token-major inputs (m = num_tokens):
 *   q, k, v   device bf16 [N * m, H, 128]
 *   z         device fp32 [N * m, H, 128]
 *   A         device fp32 [H]
 *   b         device fp32 [N * m, H]
 *   state     device fp32 [N, H, 128, 128], read only
 *   state_out device fp32 [N, H, 128, 128] or NULL: the state after all m tokens
 *             (may be `state` itself)
 *   o         device fp32 [N * m, H, 128] (written)
 *   gk_log    device fp32 [N * m, H, 128] or NULL: each token's log a = -5 sigmoid(e^A z)
 *   beta_log  device fp32 [N * m, H] or NULL: each token's beta = sigmoid(b)
 *   num_tokens 0 .. KDA_MAX_REPLAY_TOKENS (larger: KDA_ERR_UNSUPPORTED)
 *
 * The per-element arithmetic, the column split and the order of the reductions are
 * those of kda_recurrent_decode() for the same num_seqs and num_heads, so o of token t
 * equals, bit for bit, the output of the (t+1)-th of m kda_recurrent_decode() calls on
 * a copy of the checkpoint, and state_out equals the state after the m-th call. That
 * (the ReplaySSM requirement) holds on one device for one (num_seqs, num_heads).
 * Pointers need 16-byte alignment (A, b, beta_log: 4). Stream-ordered, asynchronous.
 */
int kda_recurrent_verify(const uint16_t *q, const uint16_t *k, const uint16_t *v,
                         const float *z, const float *A, const float *b,
                         const float *state, float *state_out, float *o,
                         float *gk_log, float *beta_log,
                         int32_t num_seqs, int32_t num_heads, int32_t num_tokens,
                         int32_t d_k, int32_t d_v, void *stream);

/*
 * kda_replay_fold - commit the accepted prefix of a verified draft window to the state.
 *
 * For every sequence n, the first a_n = clamp(num_accepted[n], 0, m) tokens of the
 * window are replayed, in order, on state[n, :] in place, from the caller's k, v and
 * the gate values that kda_recurrent_verify() logged (the fused fold of 'Kimi K3
 * attention deep dive', §6.2). The state must be the checkpoint the window was verified
 * from. No output is produced, and a sequence with a_n = 0 is not touched.
 *
 *   k, v          device bf16 [N * m, H, 128], the window's tokens as given to verify
 *   gk_log        device fp32 [N * m, H, 128] from kda_recurrent_verify()
 *   beta_log      device fp32 [N * m, H]      from kda_recurrent_verify()
 *   num_accepted  device int32 [N]
 *   state         device fp32 [N, H, 128, 128], updated in place
 *   num_tokens    the window length m, 0 .. KDA_MAX_REPLAY_TOKENS
 *
 * The result equals, bit for bit, a_n kda_recurrent_decode() calls with the same
 * (num_seqs, num_heads) on that sequence's tokens. Alignment: 16 bytes (beta_log and
 * num_accepted: 4).
 */
int kda_replay_fold(const uint16_t *k, const uint16_t *v, const float *gk_log, const float *beta_log,
                    const int32_t *num_accepted, float *state,
                    int32_t num_seqs, int32_t num_heads, int32_t num_tokens,
                    int32_t d_k, int32_t d_v, void *stream);

/*
 * kda_fused_decode - one decode token of the whole KDA layer step between the
 * projections: causal conv -> recurrent update -> gated RMSNorm in one launch ('Kimi K3
 * attention deep dive', §6.3), with the activations of the same page's §2.3:
 *
 *   q = L2Norm(Swish(ShortConv(x_q))),  k = L2Norm(Swish(ShortConv(x_k))),
 *   v = Swish(ShortConv(x_v))
 *   then the update of kda_recurrent_decode() on state[n, h] (in place), o = S^T q
 *   y = o / sqrt(mean(o^2) + eps_rms) * norm_w * sigmoid(g)
 *
 * ShortConv is depthwise and causal with 4 taps: output channel c is
 *   conv_w[s, h, c, 0] x_{t-3} + conv_w[s, h, c, 1] x_{t-2} + conv_w[s, h, c, 2] x_{t-1}
 *   + conv_w[s, h, c, 3] x_t,
 * with x_{t-3..t-1} read from the conv state, which afterwards holds x_{t-2}, x_{t-1}, x_t
 * (a new sequence starts from zeros). L2Norm(x) = x / sqrt(sum(x^2) + eps_l2) over the
 * head's 128 channels; Swish(x) = x sigmoid(x). There is no 1/sqrt(d) scale on q.
 *
 * Arguments (N = num_seqs, H = num_heads; all device pointers, caller-owned):
 *   x_q, x_k, x_v  bf16 [N, H, 128]      the projections before the convolution
 *   conv_state     bf16 [N, 3, 3, H, 128] per stream (q, k, v) the last three inputs,
 *                  oldest first; read and updated in place
 *   conv_w         fp32 [3, H, 128, 4]    taps per stream, head, channel, oldest first
 *   z, A, b        as kda_recurrent_decode()
 *   g              fp32 [N, H, 128]       output-gate pre-activation
 *   norm_w         fp32 [128]             RMSNorm weight (shared by the heads)
 *   eps_l2, eps_rms  >= 0 (negative or NaN: KDA_ERR_UNSUPPORTED)
 *   state          fp32 [N, H, 128, 128]  read and overwritten in place
 *   y              fp32 [N, H, 128]       written
 * Alignment: 16 bytes (A, b: 4). All arithmetic is fp32. Stream-ordered, asynchronous.
 */
int kda_fused_decode(const uint16_t *x_q, const uint16_t *x_k, const uint16_t *x_v,
                     uint16_t *conv_state, const float *conv_w,
                     const float *z, const float *A, const float *b,
                     const float *g, const float *norm_w, float eps_l2, float eps_rms,
                     float *state, float *y,
                     int32_t num_seqs, int32_t num_heads, int32_t d_k, int32_t d_v, void *stream);

/* ---------------------------------------------------------------------------------
 * Latent attention over a paged cache, for the layers that stand between KDA layers (24
 * of them beside 69 KDA layers in the pages' model).
 *
 * A token keeps one row of KDA_MLA_ROW = 576 bf16 values: the normalised latent c (512)
 * and the positional key p (64), both shared by all heads. With W_K, W_V the head's
 * up-projections, the head's key is (W_K c, p) and its value W_V c:
 *
 *   expanded   s = scale (q_nope . (W_K c) + q_pe . p),   o = sum_j softmax(s)_j (W_V c_j)
 *   absorbed   s = scale ((W_K^T q_nope) . c + q_pe . p),  o = W_V (sum_j softmax(s)_j c_j)
 *
 * The expanded form (kda_mla_prefill) costs 2 (192 + 128) operations a query, key and
 * head and reads keys and values that the caller has expanded; the absorbed form
 * (kda_mla_decode) costs 2 (576 + 512) and reads the cached rows alone, so it is the one
 * for few queries. The four projections stay with the caller.
 *
 * The cache of one layer is num_pages pages of page_size rows; row r of page p starts at
 * element p * page_stride + r * 576, so pages of several layers may interleave.
 * page_size is a multiple of 16 (at most 65536); page_stride is a multiple of 8 and at
 * least page_size * 576. Row i of sequence n is row i % page_size of page
 * page_table[n * max_pages + i / page_size]. Entries past a sequence's rows are not read.
 *
 * 'status' is a device int32 or NULL. The caller sets it to 0 once; a call whose device
 * tables turn out bad stores a kda_status there (KDA_ERR_SEQLENS for a length or offset,
 * KDA_ERR_PAGES for a page id, KDA_ERR_CUDA for a bounded wait that gave up: that call's
 * outputs are not to be used), and no call clears it. No bad table makes a kernel read or
 * write outside the tensors it was given. kda_workspace_status(status, stream) reads it.
 * Outputs overlap no input unless a call says so.
 * --------------------------------------------------------------------------------- */
#define KDA_MLA_LATENT 512 /* values of the latent */
#define KDA_MLA_POS 64     /* values of the positional key */
#define KDA_MLA_ROW 576    /* a cached row */
#define KDA_MLA_NOPE 128   /* expanded key without position, and value, of one head */
#define KDA_MLA_QK 192     /* expanded query of one head */

/*
 * kda_mla_append - normalise new tokens' latents, rotate their positional keys, and write
 * both into the pages; rotate their queries' positional part in the same launch.
 *
 *   row = ( c / sqrt(mean(c^2) + eps) * norm_w ,  R(pos) k_pe ),   q_out = R(pos) q_pe
 *
 * in fp32, rounded once to bf16. R(pos) turns 32 pairs of values by the angles of the
 * token's position: (a, b) -> (a cos - b sin, b cos + a sin), the pairs being (i, i + 32),
 * or (2 i, 2 i + 1) with rope_interleaved. Without 'rope' nothing is rotated (the layers of
 * the pages carry no position), and k_pe is copied.
 *
 * The new tokens of sequence n are rows cu_seqlens[n] .. cu_seqlens[n+1]-1; they are its
 * last ones: row cu_seqlens[n+1] - 1 has position cache_lens[n] - 1. cache_lens thus
 * counts the new tokens already, as kda_mla_decode() wants it. cu_seqlens == NULL: every
 * sequence has total_tokens / num_seqs (a whole number) tokens. Rows outside every
 * sequence's range are left alone.
 *
 *   c         device bf16, row t at c + t * c_stride (512 values)
 *   k_pe      device bf16, row t at k_pe + t * k_pe_stride (64 values)
 *   norm_w    device fp32 [512] or NULL (no normalisation: c is copied)
 *   rope      device fp32 [rope_len, 64], 32 cosines then 32 sines a position, or NULL
 *   q_pe, q_out  device bf16, head h of token t at t * q_token_stride + h * q_head_stride
 *             (q_out: its own strides; 64 values), or both NULL. q_out may be q_pe itself
 *             with the same strides. Only with 'rope'.
 *   cu_seqlens device int32 [num_seqs + 1] or NULL; cache_lens device int32 [num_seqs];
 *   page_table device int32 [num_seqs, max_pages]; cache device bf16, written
 * Strides count elements and are multiples of 8; pointers are 16-byte aligned (tables: 4).
 * The rows written by one call must be distinct. A token whose position or page is bad
 * (position negative, past the page table, or past rope_len) writes no row and NaN into
 * q_out, and sets 'status'.
 */
int kda_mla_append(const uint16_t *c, int64_t c_stride, const uint16_t *k_pe, int64_t k_pe_stride,
                   const float *norm_w, float eps, const float *rope, int32_t rope_len, int32_t rope_interleaved,
                   const uint16_t *q_pe, int64_t q_token_stride, int64_t q_head_stride,
                   uint16_t *q_out, int64_t q_out_token_stride, int64_t q_out_head_stride, int32_t num_heads,
                   const int32_t *cu_seqlens, const int32_t *cache_lens, const int32_t *page_table, int32_t max_pages,
                   uint16_t *cache, int64_t page_stride, int32_t num_pages, int32_t page_size,
                   int64_t total_tokens, int32_t num_seqs, int32_t *status, void *stream);

/*
 * kda_mla_gather - cached rows of a batch as dense rows, for the expanded form: out row
 * cu_seqlens[n] + i is row i of sequence n.
 *
 *   cu_seqlens device int32 [num_seqs + 1]; page_table device int32 [num_seqs, max_pages];
 *   out       device bf16 [total_rows, 576]
 * Rows of out outside every sequence's range are left as they were; a row whose page is
 * bad becomes NaN and sets 'status'.
 */
int kda_mla_gather(const uint16_t *cache, int64_t page_stride, int32_t num_pages, int32_t page_size,
                   const int32_t *cu_seqlens, const int32_t *page_table, int32_t max_pages, uint16_t *out,
                   int64_t total_rows, int32_t num_seqs, int32_t *status, void *stream);

/*
 * kda_mla_prefill - attention in the expanded form over packed sequences.
 *
 * Query row i of sequence n (n_q rows) attends to its n_k keys: all of them, or with
 * 'causal' keys 0 .. n_k - n_q + i (the queries are the last tokens; n_k > n_q when a
 * prefix is cached). A row that sees no key gets o = 0 and lse = -inf.
 *
 *   q         device bf16 [total_q, H, 192]   128 values without position, then 64 with it
 *   kv        device bf16 [total_k, H, 256]   a head's key without position (128), then its
 *             value (128), as one up-projection of the latents gives them
 *   k_pe      device bf16, row j at k_pe + j * k_pe_stride (64 values): the positional keys
 *   cu_seqlens_q, cu_seqlens_k  device int32 [num_seqs + 1], rising from 0 or more to
 *             total_q and total_k at most
 *   scale     finite and > 0 (KDA_ERR_UNSUPPORTED otherwise)
 *   o         device bf16 [total_q, H, 128] (written)
 *   lse       device fp32 [total_q, H] or NULL: log sum_j exp(s_j)
 * k_pe_stride is a multiple of 8 and at least 64. Rows of o and lse outside every sequence's range are
 * left as they were. Scores, statistics and sums are fp32 (a sum of values is within about 2^-11 of
 * itself, however many keys); the probabilities are rounded to bf16 for the product with the
 * values. Hidden scores count for nothing whatever they are,
 * but a NaN or infinite value row inside a sequence can reach rows that do not see it (its
 * probability there is 0); rows outside the sequence never do. A sequence whose offsets fall
 * or leave the tensors, or whose queries begin before an earlier one's end (offsets fell between
 * them), is not computed and sets 'status' to KDA_ERR_SEQLENS; its rows are
 * left as they were. Pointers are 16-byte aligned (tables, lse and status: 4).
 */
int kda_mla_prefill(const uint16_t *q, const uint16_t *kv, const uint16_t *k_pe, int64_t k_pe_stride,
                    const int32_t *cu_seqlens_q, const int32_t *cu_seqlens_k, int64_t total_q, int64_t total_k,
                    int32_t num_seqs, int32_t num_heads, int32_t causal, float scale,
                    uint16_t *o, float *lse, int32_t *status, void *stream);

/* Bytes of device workspace for kda_mla_decode() with these sizes (a bound that depends
 * on them alone); 0 for a negative argument. */
size_t kda_mla_decode_workspace_size(int32_t num_seqs, int32_t num_heads, int32_t num_tokens);

/*
 * kda_mla_decode - attention in the absorbed form over the paged rows, for one token a
 * sequence or a window of up to KDA_MAX_REPLAY_TOKENS draft tokens.
 *
 * Sequence n has cache_lens[n] rows in the cache, its num_tokens new ones last. Token t of
 * the window is row n * num_tokens + t and attends to rows 0 .. cache_lens[n] - num_tokens
 * + t; where that leaves none, o = 0 and lse = -inf.
 *
 *   q_lat     device bf16 [N * m, H, 512]   queries carried into the latent space
 *   q_pe      device bf16 [N * m, H, 64]    their positional part
 *   cache, page_stride, num_pages, page_size, page_table, max_pages: as above
 *   cache_lens device int32 [N]
 *   scale     finite and > 0 (KDA_ERR_UNSUPPORTED otherwise)
 *   o         device bf16 [N * m, H, 512] (written): sum_j softmax(s)_j c_j
 *   lse       device fp32 [N * m, H] or NULL
 *   workspace device scratch, kda_mla_decode_workspace_size() bytes, 256-byte aligned; its
 *             contents need no initialisation and are dead after the call
 * Pointers are 16-byte aligned (tables, lse and status: 4). Calls that share a workspace must be
 * ordered on one stream. Scores, statistics, sums and partial outputs are fp32 (a sum is within about
 * 2^-11 of itself, however many rows); the probabilities are rounded to bf16 for the product with the
 * rows. A NaN or infinite row of a sequence can reach window tokens that do
 * not see it; rows outside the sequence never do. A sequence with a negative length, one past
 * its page table, or a bad page id gets NaN in o and lse and sets 'status'.
 */
int kda_mla_decode(const uint16_t *q_lat, const uint16_t *q_pe, const uint16_t *cache, int64_t page_stride,
                   int32_t num_pages, int32_t page_size, const int32_t *page_table, int32_t max_pages,
                   const int32_t *cache_lens, int32_t num_seqs, int32_t num_heads, int32_t num_tokens, float scale,
                   uint16_t *o, float *lse, void *workspace, size_t workspace_bytes, int32_t *status, void *stream);

/* ---------------------------------------------------------------------------------
 * The same cache in 8 bits: 644 bytes a token instead of 1152.
 *
 * A token's row is KDA_MLA_ROW_FP8 = 640 bytes: its 512 latent values in e4m3, then its 64
 * positional ones in bf16, both in units of the row's own scale s = 2^e (fp32): e is the least
 * integer of -40 .. 40 for which the row's largest |latent| is at most 448 s, the largest value
 * of the type (0 for a row of zeros). Each latent is rounded once, from fp32 to the nearest
 * e4m3; the scale being a power of two, the positional key is its bf16 rounding, and reading
 * a row back is exact. The scale is a token's own, since tokens are written one at a time:
 * a larger one that comes later leaves the written ones as they are.
 *
 * A page of page_size rows (a multiple of 16, at most 65536) is page_size * 640 bytes of rows,
 * then page_size fp32 scales: page_size * KDA_MLA_TOKEN_FP8 bytes, a multiple of 16, at byte
 * p * page_stride; page_stride counts bytes, is a multiple of 16 and at least that. Page
 * tables, lengths, 'status' and bad tables are as above, and kda_pages_copy() moves these pages
 * like any others.
 * --------------------------------------------------------------------------------- */
#define KDA_MLA_ROW_FP8 640   /* bytes of a row, its scale apart */
#define KDA_MLA_TOKEN_FP8 644 /* bytes of a token */

/*
 * kda_mla_append_fp8 - kda_mla_append() into the 8-bit cache: the same normalisation and
 * rotation in fp32, then the row's scale and its rounding as above. Arguments as there, but
 * for cache: device bytes, written.
 *
 * Latents past 448 * 2^40 are held as that; a NaN stays one (and counts for nothing in the
 * scale); a positional value past bf16's range in units of s becomes infinite.
 */
int kda_mla_append_fp8(const uint16_t *c, int64_t c_stride, const uint16_t *k_pe, int64_t k_pe_stride,
                       const float *norm_w, float eps, const float *rope, int32_t rope_len, int32_t rope_interleaved,
                       const uint16_t *q_pe, int64_t q_token_stride, int64_t q_head_stride,
                       uint16_t *q_out, int64_t q_out_token_stride, int64_t q_out_head_stride, int32_t num_heads,
                       const int32_t *cu_seqlens, const int32_t *cache_lens, const int32_t *page_table, int32_t max_pages,
                       uint8_t *cache, int64_t page_stride, int32_t num_pages, int32_t page_size,
                       int64_t total_tokens, int32_t num_seqs, int32_t *status, void *stream);

/*
 * kda_mla_gather_fp8 - rows of the 8-bit cache as dense bf16 rows, the values that they stand
 * for: out row cu_seqlens[n] + i is row starts[n] + i of sequence n.
 *
 *   cu_seqlens device int32 [num_seqs + 1]; starts device int32 [num_seqs], the first row to
 *             read of each sequence, or NULL for 0 (a long prefix is expanded a window at a time)
 *   page_table device int32 [num_seqs, max_pages]; out device bf16 [total_rows, 576]
 * Rows of out outside every sequence's range are left as they were; a row that is negative, past
 * the page table or in a bad page becomes NaN and sets 'status'.
 */
int kda_mla_gather_fp8(const uint8_t *cache, int64_t page_stride, int32_t num_pages, int32_t page_size,
                       const int32_t *cu_seqlens, const int32_t *starts, const int32_t *page_table, int32_t max_pages,
                       uint16_t *out, int64_t total_rows, int32_t num_seqs, int32_t *status, void *stream);

/* Bytes of device workspace for kda_mla_decode_fp8() with these sizes (a bound that depends
 * on them alone); 0 for a negative argument. */
size_t kda_mla_decode_fp8_workspace_size(int32_t num_seqs, int32_t num_heads, int32_t num_tokens);

/*
 * kda_mla_decode_fp8 - kda_mla_decode() over the 8-bit cache:
 *
 *   s_rj = scale s_j (q_lat_r . c_j + q_pe_r . p_j),   o_r = sum_j softmax(s_r)_j s_j c_j
 *
 * with c_j, p_j the stored values and s_j their scale. Arguments, windows, empty rows, bad tables
 * and the order of calls that share a workspace are as there, but for
 *   cache     device bytes; the scales are the powers of two that kda_mla_append_fp8() writes
 *   workspace kda_mla_decode_fp8_workspace_size() bytes, 256-byte aligned
 *
 * The cached values enter the products as they lie. The other operands are two 8-bit numbers each: a
 * query row's latents keep every bf16 bit down to 2^-17.8 of the row's largest; a weight (a probability times s_j) is
 * off by at most 2^-7.8 of itself (a bf16's rounding is 2^-8), or, where that is more, 2^-13.9 of a unit, and by 2^-53 of
 * the row's largest weight besides. With the cached rows in tiles of 64 the unit is at most the larger of 2^-2.5 of the largest
 * weight in the 9 tiles that end with its own and 1/8 of the largest sum of four tiles in a row among them, the weights
 * of the sequence's first 8 rows counting 2^-6.2 of theirs.
 * Scores, statistics, sums and partial outputs are fp32. A query row with an infinity or a NaN gives NaN in
 * its own row of o and lse. How the rows are cut, and with that the last bits, depends on the lengths, on
 * num_seqs, num_heads and num_tokens and on max_pages; a call repeated gives the same bits.
 */
int kda_mla_decode_fp8(const uint16_t *q_lat, const uint16_t *q_pe, const uint8_t *cache, int64_t page_stride,
                       int32_t num_pages, int32_t page_size, const int32_t *page_table, int32_t max_pages,
                       const int32_t *cache_lens, int32_t num_seqs, int32_t num_heads, int32_t num_tokens, float scale,
                       uint16_t *o, float *lse, void *workspace, size_t workspace_bytes, int32_t *status, void *stream);

/*
 * kda_pages_copy - copy pages of a pool in every layer: the device side of forking a
 * sequence (its last page, and its KDA state slot) and of compacting a cache.
 *
 * Page p of layer l is the page_bytes bytes at pool + l * layer_stride + p * page_stride
 * (strides in bytes). For i = 0 .. num_pairs - 1 in order, page dst[i] becomes a copy of
 * page src[i] in all num_layers layers; a later pair sees what an earlier one wrote.
 *
 *   pool      device; src, dst  HOST int32 [num_pairs], read before the call returns (a
 *             captured call keeps the lists of its capture)
 * page_bytes, page_stride, layer_stride and the pool's address are multiples of 16; the
 * pages of all layers are disjoint (KDA_ERR_SHAPE otherwise). A page id outside
 * [0, num_pages) is refused with KDA_ERR_PAGES before anything is launched.
 */
int kda_pages_copy(void *pool, int64_t page_stride, int64_t page_bytes, int32_t num_pages, int64_t layer_stride,
                   int32_t num_layers, const int32_t *src, const int32_t *dst, int32_t num_pairs, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* KDA_H_ */
