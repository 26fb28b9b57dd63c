/*
 * kda.h -- C ABI of the GB300 (sm_103a) Kimi Delta Attention hot path.
 *
 * The operator (page "Kimi Delta Attention" deep dive, section 03, the
 * recurrence as written in the Kimi Linear report; section 02 for the read):
 *
 *     S_t = (I - beta_t k_t k_t^T) Diag(alpha_t) S_{t-1} + beta_t k_t v_t^T
 *     o_t = S_t^T q_t
 *
 * per sequence and head, with a fixed d_k x d_v state S (rows are key
 * channels), alpha_t in (0,1]^{d_k} a per-channel decay and beta_t a scalar.
 * It runs in the two modes of section 06 of the same page: a chunk-parallel
 * prefill over a packed batch of variable-length sequences, and a one-token
 * recurrent decode step that updates the state in place.  Section 07 gives the
 * state hand-off: the final state of a prefill is the checkpoint another
 * prefill or the decode step continues from.
 *
 * Conventions shared by every entry point
 * ----------------------------------------
 *  - Every pointer argument is a DEVICE pointer (CUDA global memory of the
 *    current device), row-major and densely packed.  Alignment: q, k, v,
 *    log_alpha, out, cu_seqlens and the prefill states 16 bytes; the decode
 *    state 32 bytes; beta its element size; the workspace 256 bytes.
 *  - Layouts: q, k, log_alpha [T_tot, H, d_k]; v, out [T_tot, H, d_v];
 *    beta [T_tot, H]; cu_seqlens int32 [N+1]; states fp32 [N, H, d_k, d_v]
 *    (d_v contiguous).  The decode step uses the same layouts with T_tot = N.
 *    With KDA_FLAG_SCALAR_GATE, log_alpha is [T_tot, H] instead.
 *  - dtype (KDA_F32 or KDA_BF16) applies to q, k, v, log_alpha, beta and out;
 *    states are always fp32; all accumulation is fp32.
 *  - alpha = exp(log_alpha) is formed inside the kernels; beta is taken as
 *    given (already through its sigmoid).  Scaling and normalising q and k is
 *    the caller's business.
 *  - Supported head sizes: d_k == d_v, 64 or 128 (else KDA_ERR_UNSUPPORTED).
 *  - The caller owns all memory.  The library never allocates or frees
 *    device memory and never synchronises, except kda_get_device_status,
 *    which synchronises the stream it is given.  Work is enqueued on
 *    `stream` (NULL = the legacy default stream); buffers must stay alive
 *    until that work completes.  Calls are re-entrant; concurrent calls on
 *    different streams need different workspaces.
 *  - Return codes are synchronous and report what the host can see (bad
 *    arguments, launch failures).  Problems only the device can detect
 *    (a malformed cu_seqlens) are written to a status word inside the
 *    workspace and read back with kda_get_device_status.  Nothing is thrown
 *    across the ABI.
 */
#ifndef KDA_GB300_H
#define KDA_GB300_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#if defined(__GNUC__)
#define KDA_API __attribute__((visibility("default")))
#else
#define KDA_API
#endif

/* Same type as cudaStream_t. */
typedef struct CUstream_st *kda_stream_t;

typedef enum {
    KDA_OK = 0,
    KDA_ERR_INVALID_ARGUMENT = 1, /* null / misaligned pointer, bad size, aliasing out with an input */
    KDA_ERR_UNSUPPORTED = 2,      /* head size or dtype outside what the kernels implement */
    KDA_ERR_CUDA = 3,             /* a CUDA launch or API call failed (see kda_last_cuda_error) */
    KDA_ERR_TIMEOUT = 4,          /* a bounded on-device wait gave up (device status only) */
    KDA_ERR_BAD_SEQLENS = 5,      /* cu_seqlens not 0 = c_0 <= c_1 <= ... <= c_N = T_tot (device status) */
    KDA_ERR_WORKSPACE = 6,        /* workspace missing or smaller than kda_prefill_workspace_bytes */
    KDA_ERR_BAD_SNAPSHOT = 7,     /* a snapshot request off its sequence, off a chunk boundary, or
                                     repeated (device status, kda_prefill_snapshots) */
    KDA_ERR_BAD_PAGE = 8          /* a page number outside the cache (device status, kda_latent_decode) */
} kda_status;

typedef enum { KDA_F32 = 0, KDA_BF16 = 1 } kda_dtype;

/* kda_desc.flags bits. */
enum {
    /* Run the prefill (and kda_prefill_backward) on CUDA cores in fp32 even
       where the tensor-core path applies (bf16, head size 128).  Slower; meant
       for cross-checking. */
    KDA_FLAG_CUDA_CORE_PREFILL = 1,
    /* Scalar gate: log_alpha holds ONE value per (token, head) -- layout
       [T_tot, H] for the prefill, [N, H] for the decode step, aligned to its
       element size like beta -- and every key channel of the head decays by
       that same alpha.  This is the Gated DeltaNet gate that KDA refines into
       a per-channel one (deep dive, section 03: Gated DeltaNet multiplies a
       head's state by a scalar alpha, KDA by Diag(alpha)); the result equals
       the per-channel operator with log_alpha broadcast over d_k. */
    KDA_FLAG_SCALAR_GATE = 2
};

/* Problem description.  Not retained by the library after a call returns. */
typedef struct kda_desc {
    int32_t num_seqs;       /* N >= 0 sequences (decode: sequences advanced by one token) */
    int32_t num_heads;      /* H >= 1 */
    int32_t d_k;            /* key/query head size: 64 or 128 */
    int32_t d_v;            /* value head size: must equal d_k */
    int64_t total_tokens;   /* T_tot = cu_seqlens[N] (decode: must equal N) */
    int32_t dtype;          /* kda_dtype of q, k, v, log_alpha, beta, out */
    int32_t flags;          /* OR of KDA_FLAG_* bits (0: tensor cores where they apply, per-channel gate) */
    void *workspace;        /* device scratch owned by the caller (prefill only), 256-byte aligned */
    size_t workspace_bytes; /* its size in bytes */
    void **phase_events;    /* optional timing hook (NULL: none): kda_prefill records
                               phase_events[0] before the intra-chunk kernel,
                               phase_events[1] between it and the inter-chunk kernel and
                               phase_events[2] after that, each a cudaEvent_t created by
                               the caller, on `stream` */
} kda_desc;

/*
 * Bytes of device workspace kda_prefill needs for this description (0 for an
 * invalid one).  The bound depends only on N, H, d and T_tot, never on the
 * contents of cu_seqlens, so it can be sized before the lengths are known on
 * the host.  The workspace is scratch: its contents on entry are ignored, and
 * on exit it holds intermediate chunk data plus the device status word.
 */
KDA_API size_t kda_prefill_workspace_bytes(const kda_desc *desc);

/*
 * Chunk-parallel prefill over a packed batch (deep dive section 06, "chunk-
 * parallel KDA"; variable-length batching per the FlashKDA update there).
 *
 *   q, k, log_alpha  [T_tot, H, d_k]   inputs, dtype `desc->dtype`
 *                    (log_alpha [T_tot, H] with KDA_FLAG_SCALAR_GATE)
 *   v                [T_tot, H, d_v]
 *   beta             [T_tot, H]
 *   cu_seqlens       int32 [N+1], device; sequence n is packed tokens
 *                    [cu_seqlens[n], cu_seqlens[n+1]).  NULL means one
 *                    sequence of all T_tot tokens (then N must be 1).
 *   initial_state    fp32 [N, H, d_k, d_v] or NULL (zero state).
 *   out              [T_tot, H, d_v], written; must not overlap any input.
 *   final_state      fp32 [N, H, d_k, d_v] or NULL (not written).  May be the
 *                    same pointer as initial_state (in-place continuation).
 *                    A sequence of length 0 returns its initial state.
 *   stream           CUDA stream for all work.
 *
 * Returns KDA_OK once the work is enqueued.  A malformed cu_seqlens is not
 * seen by the host: the kernels then skip all work, leave out/final_state
 * unspecified and record KDA_ERR_BAD_SEQLENS in the device status word.
 */
KDA_API int kda_prefill(const kda_desc *desc,
                const void *q, const void *k, const void *v,
                const void *log_alpha, const void *beta,
                const int32_t *cu_seqlens, const float *initial_state,
                void *out, float *final_state, kda_stream_t stream);

/*
 * kda_prefill that also saves the recurrent state at interior positions: the
 * prefix checkpoints of deep dive section 07 (a cached prefix is the state
 * after it; restoring that state and feeding the rest of the sequence
 * continues exactly), taken in the same pass instead of one call per prefix.
 *
 *   num_snapshots  M >= 0 requests.
 *   snapshot_at    int32 [M][2], device, 4-byte aligned: (sequence n, prefix
 *                  length p) pairs, 0 <= n < N, 0 <= p <= L_n, where p is a
 *                  multiple of 64 (the prefill's chunk size) or p = L_n.
 *                  p = 0 gives the initial state.  No pair may repeat.
 *   snapshots      fp32 [M, H, d_k, d_v], device, 16-byte aligned, written:
 *                  snapshot m is the state of sequence n after its first p
 *                  tokens (what kda_prefill over those tokens would return as
 *                  final_state).  Must not overlap any other buffer.
 *
 * Every other argument is that of kda_prefill.  A request that breaks the
 * rules above is seen on the device only: all work is skipped and the status
 * word holds KDA_ERR_BAD_SNAPSHOT.  M = 0 is plain kda_prefill.
 */
KDA_API int kda_prefill_snapshots(const kda_desc *desc,
                                  const void *q, const void *k, const void *v,
                                  const void *log_alpha, const void *beta,
                                  const int32_t *cu_seqlens, const float *initial_state,
                                  void *out, float *final_state,
                                  int32_t num_snapshots, const int32_t *snapshot_at, float *snapshots,
                                  kda_stream_t stream);

/*
 * Reverse mode of kda_prefill: the gradients of a scalar loss with respect to
 * every input, given its gradients with respect to the outputs and the final
 * state.  The deep dive (section 06) names prefill and training as the uses
 * of the chunked form; this entry point supplies the training half by the
 * chain rule through each token's step of the section 03 recurrence.
 *
 *   q, k, v, log_alpha, beta, cu_seqlens, initial_state: as for kda_prefill
 *                    (the same call's inputs).
 *   d_out            [T_tot, H, d_v], dtype `desc->dtype`: dLoss/dout.
 *   d_final_state    fp32 [N, H, d_k, d_v] or NULL (zero): dLoss/dfinal_state.
 *   dq, dk           fp32 [T_tot, H, d_k], written.
 *   dv               fp32 [T_tot, H, d_v], written.
 *   dlog_alpha       fp32 [T_tot, H, d_k] ([T_tot, H] with the scalar gate).
 *   dbeta            fp32 [T_tot, H].
 *   d_initial_state  fp32 [N, H, d_k, d_v] or NULL (not written).
 * Gradients are 4-byte aligned, the states 16-byte aligned; no output may
 * overlap an input or another output.  desc->workspace must hold
 * kda_backward_workspace_bytes(desc) bytes (about 4 * H * d_k * d_v bytes
 * per 8 tokens of kept states plus 4 * (3 d_k + 1) * H * d_v / 32 bytes per
 * token of partial sums, which also covers the tensor-core path's scratch).
 *
 * bf16 inputs with head size 128 run on the tensor cores: the forward is
 * recomputed saving every 64-token chunk's end state, a reverse walk over the
 * chunks gives each chunk's end-state gradient, and one kernel per (chunk,
 * head) forms the gradients (bf16 operands, fp32 accumulation: gradients
 * within about 1e-2 relative L2 of exact arithmetic).  A call in which some
 * chunk's cumulative decay exceeds 2^100 in a channel (log alpha summed over
 * the chunk below -69) runs instead on the fp32 CUDA-core path, decided on
 * the device.  fp32 inputs, head size 64, or KDA_FLAG_CUDA_CORE_PREFILL take
 * the fp32 CUDA-core path (about 1e-4).  Results do not depend on scheduling
 * (no atomics).  Errors as for kda_prefill.
 */
KDA_API size_t kda_backward_workspace_bytes(const kda_desc *desc);
KDA_API int kda_prefill_backward(const kda_desc *desc,
                                 const void *q, const void *k, const void *v,
                                 const void *log_alpha, const void *beta,
                                 const int32_t *cu_seqlens, const float *initial_state,
                                 const void *d_out, const float *d_final_state,
                                 float *dq, float *dk, float *dv, float *dlog_alpha, float *dbeta,
                                 float *d_initial_state, kda_stream_t stream);

/*
 * One recurrent decode step for N independent sequences (deep dive section
 * 06, "fused recurrent KDA": decay, correct and write the state in place,
 * reading a fixed amount of memory per head).  Inputs are [N, H, *] (one
 * token per sequence, desc->total_tokens == N); state_inout fp32
 * [N, H, d_k, d_v] is read and overwritten in place; out [N, H, d_v].
 * No workspace is used (desc->workspace may be NULL).
 */
KDA_API int kda_decode_step(const kda_desc *desc,
                    const void *q, const void *k, const void *v,
                    const void *log_alpha, const void *beta,
                    float *state_inout, void *out, kda_stream_t stream);

/*
 * Synchronises `stream`, then returns the device status word that the last
 * kda_prefill on this workspace recorded: KDA_OK, KDA_ERR_BAD_SEQLENS,
 * KDA_ERR_BAD_SNAPSHOT or KDA_ERR_TIMEOUT (KDA_ERR_CUDA if the
 * synchronisation itself failed).
 */
KDA_API int kda_get_device_status(const kda_desc *desc, kda_stream_t stream);

/*
 * Size of the fixed scratch area kda_prefill_noalloc uses: 64 MiB.
 */
#define KDA_PREFILL_NOALLOC_SCRATCH_BYTES (64u * 1024u * 1024u)

/*
 * kda_prefill without a workspace, for callers that cannot allocate device
 * memory: code that gets all its buffers from someone else's pool, plugins
 * given only their inputs and outputs, or code where a cudaMalloc would
 * synchronise the device at the wrong moment.  The pages have no counterpart
 * to this call; it is a convenience of this library.
 *
 * Same arguments, layouts and results as kda_prefill; desc->workspace and
 * desc->workspace_bytes are ignored.  Instead the library's own static
 * device array of KDA_PREFILL_NOALLOC_SCRATCH_BYTES is used.  The runtime
 * reserves it on each device where this call is first used and holds it until
 * the process exits; no call allocates or frees anything.
 *  - Problems needing more scratch than that (kda_prefill_workspace_bytes
 *    larger than KDA_PREFILL_NOALLOC_SCRATCH_BYTES, for example more than about
 *    800 chunk-heads of 64 tokens on the bf16 head-size-128 path) are rejected
 *    with KDA_ERR_WORKSPACE before any GPU work.
 *  - Every call looks up the array's device address (cudaGetSymbolAddress,
 *    host-side, no stream work) with the caller's device current, so a
 *    context that was reset and re-created gets the new address.  The first
 *    call in a context may make the runtime load the library's kernels
 *    there: make it before any stream capture.
 *  - All calls on a device share the one array, which keeps the last call's
 *    contents (nothing in it needs to start at zero).  Calls whose GPU work
 *    may overlap -- different streams, or host threads without ordering --
 *    race on it and must be serialised by the caller.
 *  - The device status word lives in that array too; kda_get_device_status
 *    cannot read it.
 */
KDA_API int kda_prefill_noalloc(const kda_desc *desc,
                                const void *q, const void *k, const void *v,
                                const void *log_alpha, const void *beta,
                                const int32_t *cu_seqlens, const float *initial_state,
                                void *out, float *final_state, kda_stream_t stream);

/*
 * Diagnostic for the failure path: launches one CTA that waits on an mbarrier
 * no one ever arrives on, with the same bounded wait the prefill kernels use,
 * limited to timeout_ns (0 .. 1e9).  When the limit runs out the kernel stores
 * KDA_ERR_TIMEOUT in the device status word of desc->workspace and returns, so
 * kda_get_device_status then reports it.  Needs only desc->workspace (at least
 * 256 bytes); returns KDA_ERR_INVALID_ARGUMENT for a limit outside the range.
 */
KDA_API int kda_selftest_wait_timeout(const kda_desc *desc, int64_t timeout_ns, kda_stream_t stream);

/* ===========================================================================
 * Operators around the recurrent layers: the norm and the 8-bit products of
 * their projections, and the attention over shared latents of the layers of
 * full attention that a KDA stack alternates with (deep dive, section 04).
 *
 * They keep the conventions above (device pointers, caller-owned memory, no
 * allocation, no synchronisation, synchronous return codes) with these
 * differences: rows may be strided where a desc has a stride for them (in
 * elements, the last dimension always dense), and pointers need the alignment
 * of their element only (wider alignment selects wider accesses).
 * ======================================================================== */

/* Root-mean-square norm of rows, with the residual's addition before it and
 * an 8-bit output behind it:
 *
 *     h = x + residual                       (x alone when residual is NULL)
 *     y = h / sqrt(mean(h^2) + eps) * weight
 *     scales[b] = max(max |y| over block b, 1e-12) / 448
 *     quantized = e4m3(y / scales[b])        (to nearest even, saturating)
 *
 * with blocks of 128 consecutive elements of a row, the last one short where
 * dim is no multiple of 128.  h, the mean and y are fp32; the mean is taken of
 * the unrounded h.  A row that holds an infinity or a NaN has unspecified
 * values of y, scales and quantized; other rows are not affected. */
typedef struct kda_norm_desc {
    int64_t rows;            /* >= 0 */
    int32_t dim;             /* elements of a row, >= 1 */
    int32_t dtype;           /* kda_dtype of x, weight, residual, residual_out, normed */
    int64_t x_stride;        /* elements between rows of x, >= dim */
    int64_t residual_stride; /* elements between rows of residual, >= dim */
    float eps;               /* >= 0 */
} kda_norm_desc;

/* weight [dim] or NULL (ones); residual [rows, dim] or NULL.  Written, each
 * unless NULL, dense: residual_out = h in dtype, normed = y in dtype,
 * quantized (e4m3 bytes) with scales fp32 [rows, ceil(dim / 128)] (both or
 * neither).  residual_out may be x or residual itself if that is dense; no
 * other output may overlap an input or another output. */
KDA_API int kda_rms_norm(const kda_norm_desc *desc, const void *x, const void *weight, const void *residual,
                         void *residual_out, void *normed, uint8_t *quantized, float *scales,
                         kda_stream_t stream);

/* Product of e4m3 matrices with scales:
 *
 *     c[m, n] = sum over k of a[m, k] a_scale[m, k / 128] b[n, k] b_scale[n / 128, k / 128]
 *
 * Products of one k block are summed in fp32 by the tensor cores and scaled and
 * added in fp32 after that. */
typedef struct kda_matmul_desc {
    int64_t m;               /* rows of a and c, >= 0 */
    int32_t n, k;            /* rows of b; length of the sum; n >= 0, k >= 1 */
    int64_t a_stride;        /* elements between rows of a, >= k */
    int64_t b_stride;        /* elements between rows of b, >= k */
    int64_t c_stride;        /* elements between rows of c, >= n */
    int32_t dtype;           /* kda_dtype of c */
    int32_t flags;           /* 0 or KDA_FLAG_CUDA_CORE_PREFILL (fp32 CUDA cores, for cross-checking) */
} kda_matmul_desc;

/* a [m, k], b [n, k] e4m3 bytes; a_scale fp32 [m, ceil(k / 128)], b_scale fp32
 * [ceil(n / 128), ceil(k / 128)], both dense; c [m, n] written, overlapping no
 * input.  a and b with 16-byte aligned rows (address and stride) run on the
 * tensor cores, others on CUDA cores. */
KDA_API int kda_matmul_fp8(const kda_matmul_desc *desc, const uint8_t *a, const float *a_scale, const uint8_t *b,
                           const float *b_scale, void *c, kda_stream_t stream);

/* kda_latent_desc.flags bits, beside KDA_FLAG_CUDA_CORE_PREFILL. */
enum {
    /* kda_latent_prefill: every key of its sequence is visible to a query. */
    KDA_FLAG_NO_CAUSAL = 4,
    /* kda_latent_decode: the cache is one that kda_latent_cache_write fills (8-bit codes, see there); page_stride is in
       bytes, cache and page_stride are multiples of 16. */
    KDA_FLAG_CACHE_8 = 64
};

/* Attention whose keys and values come from one latent vector c_s and one
 * rotary key r_s a token, both shared by all heads.  Expanded form (prompts):
 * keys [k_s,h | r_s] and values v_s,h, the up-projections of c_s, are given.
 * Absorbed form (decoding): the up-projections are folded into the queries and
 * the output, keys are [c_s | r_s] and values c_s.  bf16 with the sizes (d_k,
 * d_rope, d_v) = (128, 64, 128) expanded and rank 512, d_rope 64 absorbed runs
 * on the tensor cores; fp32, KDA_FLAG_CUDA_CORE_PREFILL, other sizes up to the
 * limits below, and strides or addresses that are no multiple of 16 bytes run
 * on CUDA cores in fp32.
 *
 * On the tensor cores the softmax weights are rounded to bf16 (by at most 2^-8
 * of each) for their product with the values; their sum is taken in fp32 before
 * that.  Outputs are off by up to a third more than with weights in fp32, where
 * their own rounding to bf16 decides (relative, against 64 bits: 0.0020 and
 * 0.0015 for a prompt of 8192 tokens).  fp32 inputs and
 * KDA_FLAG_CUDA_CORE_PREFILL keep the weights in fp32.
 *
 * A score that is NaN or +infinity makes its row NaN; one of -infinity hides its
 * key.  Keys that a row does not see do not reach it, whatever they hold.  Nor
 * do values behind the end of a sequence.  Values that a row does not see inside
 * its sequence (behind the causal limit) may: on the tensor cores they are
 * multiplied by 0, so an infinity or NaN in one makes rows NaN that see keys of
 * the same 128 (not so with KDA_FLAG_CACHE_8, where no value does that its row
 * does not see). */
typedef struct kda_latent_desc {
    int32_t num_seqs;        /* N >= 0 */
    int32_t num_heads;       /* H >= 1 */
    int32_t dtype;           /* kda_dtype of everything but lse */
    int32_t flags;
    float scale;             /* factor of the scores before the softmax, finite and > 0 */
    int32_t d_k;             /* expanded: per-head key channels; absorbed: rank of the latent */
    int32_t d_rope;          /* shared rotary key channels, >= 0; d_k + d_rope <= 256 / 640 */
    int32_t d_v;             /* expanded: value channels <= 256; absorbed: must equal d_k <= 512 */
    /* expanded form */
    int64_t total_q, total_k;                /* cu_seqlens_q[N], cu_seqlens_k[N] */
    int64_t q_token_stride, q_head_stride;   /* both forms (absorbed: a token is one (sequence, query)) */
    int64_t k_token_stride, k_head_stride, v_token_stride, v_head_stride, rope_token_stride;
    /* absorbed form */
    int32_t num_queries;     /* queries a sequence, >= 1 */
    int32_t page_size;       /* tokens of a page, >= 1 */
    int32_t num_pages;       /* pages of the cache */
    int32_t max_pages;       /* row length of the page table, >= 1 */
    int64_t page_stride;     /* elements between pages; tokens of a page are dense, d_k + d_rope apart (KDA_FLAG_CACHE_8:
                                bytes between pages) */
    void *workspace;         /* 256-byte aligned device scratch */
    size_t workspace_bytes;
} kda_latent_desc;

/* Bytes of device workspace for each form (0 for an invalid desc).  They do not
 * depend on the contents of any device array. */
KDA_API size_t kda_latent_prefill_workspace_bytes(const kda_latent_desc *desc);
KDA_API size_t kda_latent_decode_workspace_bytes(const kda_latent_desc *desc);

/* Expanded form over a packed batch: query i of a sequence with Lq queries and
 * Lk keys sees keys 0 .. Lk - Lq + i (all with KDA_FLAG_NO_CAUSAL).
 *
 *   q        [total_q, H, d_k + d_rope]     k_nope [total_k, H, d_k]
 *   k_rope   [total_k, d_rope] (NULL iff d_rope = 0)    v [total_k, H, d_v]
 *   cu_seqlens_q, cu_seqlens_k  int32 [N+1], device; NULL for one sequence.
 *   out      [total_q, H, d_v] dense, written; lse fp32 [total_q, H] or NULL:
 *            log of the sum of exp(score).  A query that sees no key gets a zero
 *            row and lse = -infinity.
 *
 * A malformed cu_seqlens is recorded as KDA_ERR_BAD_SEQLENS in the device
 * status word (kda_latent_status); out is then unspecified. */
KDA_API int kda_latent_prefill(const kda_latent_desc *desc, const void *q, const void *k_nope, const void *k_rope,
                               const void *v, const int32_t *cu_seqlens_q, const int32_t *cu_seqlens_k, void *out,
                               float *lse, kda_stream_t stream);

/* Absorbed form for the last num_queries (Lq) tokens of each sequence over a
 * paged cache: query i of a sequence of length L sees cached tokens 0 ..
 * L - Lq + i.
 *
 *   q          [N, Lq, H, d_k + d_rope]
 *   cache      [num_pages, page_size, d_k + d_rope]
 *   page_table int32 [N, max_pages], device: token t of sequence n is row
 *              t % page_size of page page_table[n, t / page_size]; entries
 *              behind a sequence's length are not read
 *   lengths    int32 [N], device, 0 <= lengths[n] <= max_pages * page_size
 *   out        [N, Lq, H, d_k] dense, written; lse fp32 [N, Lq, H] or NULL, as above
 *
 * A page number outside the cache (KDA_ERR_BAD_PAGE) or a length outside its
 * range (KDA_ERR_BAD_SEQLENS) is recorded in the device status word and never
 * dereferenced; the outputs of that sequence are then unspecified.
 *
 * With KDA_FLAG_CACHE_8, keys are [2^e code | rope] and values 2^e code of the
 * quantised cache below, each exactly.  bf16 queries, rank 512 and d_rope 64 run
 * on the tensor cores, on the codes themselves: there a query is the sum of two
 * e4m3 values under one power of two for its row (exact down to 2^-22 of its
 * largest channel; infinite ones count as NaN) and a softmax weight times its
 * token's 2^e the sum of three e5m2 values (off by 2^-8.6 of it at most, or by
 * 2^-26 of the row's largest such product, whichever is more).  Sums are fp32; a
 * weight may be missing from its row's if it is below 2^(x - 99) of another one's,
 * 2^x the row's largest scale.  Everything else, and fp32 queries, run on CUDA
 * cores in fp32. */
KDA_API int kda_latent_decode(const kda_latent_desc *desc, const void *q, const void *cache,
                              const int32_t *page_table, const int32_t *lengths, void *out, float *lse,
                              kda_stream_t stream);

/* The quantised cache of latents.  A page holds page_size rows of rank e4m3
 * codes and d_rope bf16 rotary channels, then a byte e + 127 for each of its
 * tokens, and is padded to 128 bytes:
 *
 *     byte t * (rank + 2 d_rope) + c             code c of the page's token t
 *     byte t * (rank + 2 d_rope) + rank + 2 c    its rotary channel c
 *     byte page_size * (rank + 2 d_rope) + t     its scale, e + 127
 *
 * A latent channel is worth 2^e code.  e is the smallest integer with
 * max |latent| <= 448 2^e, within -100 .. 120 (448: e4m3's largest value; the
 * maximum is over the token's finite channels), so that no code saturates and the
 * values are exact in bf16.  One scale a token does: behind a channel's own
 * exponent of four bits, scales of shorter groups would change only values below
 * 2^-14 of the token's largest.  Channels that are infinite or NaN become NaN.
 * Memory need not be cleared before it is written.  Pages of zeros hold tokens of
 * zeros. */
typedef struct kda_latent_cache_desc {
    int32_t num_seqs;        /* N >= 0 */
    int32_t dtype;           /* kda_dtype of latents and rope */
    int64_t total_tokens;    /* T >= 0 rows of latents and rope */
    int32_t rank;            /* a multiple of 16, 16 .. 512 */
    int32_t d_rope;          /* a multiple of 8, 0 .. 128 */
    int32_t page_size;       /* tokens of a page, >= 1 */
    int32_t num_pages;       /* pages of the cache */
    int32_t max_pages;       /* row length of the page table, >= 1 */
    int32_t flags;           /* 0 */
    int64_t page_stride;     /* bytes between pages, a multiple of 16, >= kda_latent_cache_page_bytes */
    int64_t latent_stride;   /* elements between rows of latents, >= rank */
    int64_t rope_stride;     /* elements between rows of rope, >= d_rope */
    void *workspace;         /* 256-byte aligned device memory for the status word, or NULL: none is recorded */
    size_t workspace_bytes;  /* >= 256 with a workspace */
} kda_latent_cache_desc;

/* Bytes of a page (0 for sizes that are not supported). */
KDA_API size_t kda_latent_cache_page_bytes(int32_t page_size, int32_t rank, int32_t d_rope);

/* Quantises the last tokens of each sequence into its pages, and reads tokens
 * back as rows.
 *
 *   latents    [T, rank], rope [T, d_rope] (NULL iff d_rope = 0): rows of the
 *              sequences, packed; read by _write, written by _read
 *   cu_seqlens int32 [N+1], device: rows cu_seqlens[n] .. cu_seqlens[n+1] - 1 are
 *              sequence n's; NULL: T / N rows each (N divides T).  cu_seqlens[N]
 *              may be less than T: rows behind it are not written to the cache, or
 *              left as they were
 *   page_table int32 [N, max_pages], lengths int32 [N] as for kda_latent_decode:
 *              row i of the L rows of sequence n is its cached token
 *              lengths[n] - L + i (lengths count the new tokens).  Rows whose
 *              place is negative are left out (a sequence padded into a batch has
 *              length 0)
 *   cache      [num_pages] pages, 16-byte aligned
 *
 * A malformed cu_seqlens or a length outside 0 .. max_pages * page_size
 * (KDA_ERR_BAD_SEQLENS) and page numbers outside the cache (KDA_ERR_BAD_PAGE)
 * are recorded in the status word (kda_latent_status), if there is one.  Left out,
 * and never dereferenced, are the rows of a sequence with such a length or with
 * bounds that are not 0 <= c_n <= c_n+1 <= T (c_0 = 0), and the rows of a page with
 * such a number; rows that several sequences claim are one's of them.  Two rows of
 * one call in the same place of the cache leave that place unspecified. */
KDA_API int kda_latent_cache_write(const kda_latent_cache_desc *desc, const void *latents, const void *rope,
                                   const int32_t *cu_seqlens, const int32_t *page_table, const int32_t *lengths,
                                   uint8_t *cache, kda_stream_t stream);
KDA_API int kda_latent_cache_read(const kda_latent_cache_desc *desc, const uint8_t *cache, const int32_t *page_table,
                                  const int32_t *lengths, const int32_t *cu_seqlens, void *latents, void *rope,
                                  kda_stream_t stream);

/* Rotary positions.  Of each row (token and head) of `width` channels, `dim`
 * from `offset` on are pairs (a_i, b_i), i < dim / 2: channels i and i + dim / 2
 * of them, or 2 i and 2 i + 1 with KDA_FLAG_INTERLEAVED.  With
 * theta = positions[t] * frequencies[i],
 *
 *     a_i' = scale (a_i cos theta - b_i sin theta)
 *     b_i' = scale (b_i cos theta + a_i sin theta)
 *
 * and the other channels as they are.  KDA_FLAG_INVERSE turns by -theta, which
 * makes the gradient of the inputs from that of the outputs.  theta is taken
 * modulo a turn in 64 bits, whatever the position; the rest is fp32, rounded once. */
enum {
    KDA_FLAG_INTERLEAVED = 8,
    KDA_FLAG_INVERSE = 16,
    KDA_FLAG_POSITIONS_64 = 32   /* positions are int64, else int32 */
};
typedef struct kda_rotary_part {
    int32_t heads;               /* >= 1, <= 65535 */
    int32_t width;               /* channels of a row, <= 4096 */
    int32_t offset;              /* the first one that is turned, offset + dim <= width */
    int32_t reserved;            /* 0 */
    int64_t token_stride, head_stride;           /* elements, of the input */
    int64_t out_token_stride, out_head_stride;   /* of the output, whose rows do not overlap */
} kda_rotary_part;
typedef struct kda_rotary_desc {
    int64_t tokens;              /* >= 0 */
    int32_t dim;                 /* even, 2 .. 1024 */
    int32_t dtype;               /* kda_dtype of x, key and the outputs */
    int32_t flags;
    float scale;                 /* finite */
    kda_rotary_part x, key;      /* key is not looked at without one */
} kda_rotary_desc;

/* x, and key or NULL (the keys of the same tokens, in the same launch), to out
 * and key_out.  An output may be its own input, with the same strides, and
 * overlaps nothing else (rows of both inside one wider row, like queries and keys
 * of one projection, a token's or each head's side by side, do not overlap).
 * positions int32 or int64 [tokens], frequencies fp64 [dim / 2] (radians a
 * position), device; the pairs of one that is infinite or NaN become NaN. */
KDA_API int kda_rotary(const kda_rotary_desc *desc, const void *x, const void *key, const void *positions,
                       const double *frequencies, void *out, void *key_out, kda_stream_t stream);

/* Frequencies base^(-2 i / dim), and their scalings for contexts `factor` times
 * as long as `original_length`, the trained one.  HOST memory, no CUDA work. */
typedef enum {
    KDA_ROTARY_PLAIN = 0,
    KDA_ROTARY_LINEAR = 1,       /* all divided by factor */
    KDA_ROTARY_BASE = 2,         /* with base * factor^(dim / (dim - 2)): the slowest divided by factor, the fastest kept */
    KDA_ROTARY_BY_PARTS = 3      /* f (w + (1 - w) / factor), w = (turns - slow) / (fast - slow) within 0 .. 1, of the
                                    turns original_length f / (2 pi) that a pair made in training.  (w goes by the turns;
                                    frequencies whose w goes by the pair's index i between those of `fast` and `slow`
                                    turns are others, to be made by the caller) */
} kda_rotary_method;
KDA_API int kda_rotary_frequencies(int32_t dim, double base, int32_t method, double factor, double original_length,
                                   double slow, double fast, double *frequencies);

/* Synchronises `stream`, then returns the status word that the last
 * kda_latent_* call on this workspace recorded, be it one without queries or
 * sequences (which may do without a workspace).  KDA_ERR_TIMEOUT, of a wait on
 * the device that gave up, comes before the others and leaves every output
 * unspecified. */
KDA_API int kda_latent_status(const kda_latent_desc *desc, kda_stream_t stream);

/* A test of the limits of waits: later calls of the process on the tensor cores
 * wait for something that never comes, so their waits give up (2 s each, up to
 * some seconds a call) and KDA_ERR_TIMEOUT is recorded, or NaN written
 * (kda_matmul_fp8).  which: 1 the copies, 2 the first products, 3 the second
 * ones, 4 the softmax weights, 5 what a block is to work on (the zeros behind a
 * length, kda_latent_decode); 0 ends it.  kda_matmul_fp8 has 1 and 2. */
KDA_API int kda_selftest_drop_arrival(int32_t which);

/* Static, human-readable name of a status code. */
KDA_API const char *kda_status_string(int status);

/* The cudaError_t of the last failing CUDA call made by this thread (0 if none). */
KDA_API int kda_last_cuda_error(void);

/* ABI version: major * 10000 + minor * 100 + patch. */
KDA_API int kda_version(void);

#ifdef __cplusplus
}
#endif

#endif /* KDA_GB300_H */
