/*
 * kda.h -- C ABI of the KDA (Kimi Delta Attention) recurrence library for
 * NVIDIA GB300 (sm_103a).  libkda.so exports exactly the functions below.
 *
 * The operation (source: "[논문 리뷰] Kimi K3 Technical Report",
 * jw9603.github.io, section 3.2 "KDA의 핵심 상태 업데이트"; delta form in
 * section 3.3; alpha = exp(g) in section 3.5).  Per sequence and head, with a
 * state S in R^{d_k x d_v} whose rows are key channels:
 *
 *     S_t = (I - beta_t k_t k_t^T) Diag(alpha_t) S_{t-1} + beta_t k_t v_t^T
 *     o_t = S_t^T q_t                  (read after token t's write)
 *     alpha_t = exp(log_alpha_t)       (per key channel), beta_t a scalar.
 *
 * Conventions shared by every call:
 *  - All pointers are DEVICE pointers unless stated otherwise (only
 *    kda_prefill_host takes host buffers); the caller owns every buffer.  The
 *    library allocates nothing and keeps no state between calls other than
 *    cached device attributes.
 *  - Work is enqueued on `stream`; no call synchronises the host.  Argument
 *    errors are returned synchronously before anything is launched; a launch
 *    failure returns KDA_ERR_CUDA.  Nothing is thrown across the ABI.
 *  - Tensors are dense, row-major, with the last index fastest:
 *      q, k, log_alpha : [T_tot, H, d_k]
 *      v, o            : [T_tot, H, d_v]
 *      beta            : [T_tot, H]
 *      states          : [N, H, d_k, d_v]   fp32
 *    q, k, v share one dtype and o has the output dtype (kda_dtype_t);
 *    log_alpha, beta and states are always fp32.  Base pointers must be
 *    16-byte aligned.
 *  - Preconditions that are documented, not checked on the device:
 *    -5 <= log_alpha <= 0 (the lower-bounded decay of section 3.5); k is
 *    L2-normalised and q pre-scaled by the caller (the op uses them as given);
 *    beta is any finite value (beta up to 2 gives a reflection, "Kimi 모델
 *    분석", rlaope.github.io, section "반사가 계층을 바꿈"); inputs finite.
 *    On the tensor-core path (bf16 q/k/v with d_k = d_v = 128, see
 *    kda_prefill's Paths) v, the states (S0 and every state the recurrence
 *    passes through) and the chunk products formed from them enter the
 *    tensor cores as fp16, so |v| and every state entry must stay below
 *    65504, the largest finite fp16 value; beyond it the results are not
 *    finite.  The fp32 CUDA-core path has no such limit: a caller whose
 *    values may exceed it passes fp32 inputs (KDA_FP32).
 *  - Supported shapes: every dtype code with d_k = d_v in {16, 32, 64, 128}.
 *    Anything else returns KDA_ERR_UNSUPPORTED.
 */
#ifndef KDA_H
#define KDA_H

#include <stddef.h>
#include <stdint.h>

#include <cuda_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    KDA_OK = 0,
    KDA_ERR_INVALID_ARG = 1,   /* null required pointer, bad count, misalignment */
    KDA_ERR_UNSUPPORTED = 2,   /* dtype / head size not implemented */
    KDA_ERR_WORKSPACE = 3,     /* workspace missing, misaligned or too small */
    KDA_ERR_CUDA = 4           /* a kernel launch failed (cudaGetLastError) */
} kda_status_t;

typedef enum {
    KDA_BF16 = 0,              /* q, k, v, o are bfloat16 */
    KDA_FP32 = 1,              /* q, k, v, o are float32  */
    KDA_BF16_F32OUT = 2        /* q, k, v are bfloat16, o is float32 */
} kda_dtype_t;

/* Bytes of device workspace kda_prefill needs for num_seqs sequences of H
 * heads.  The workspace always holds the varlen work list (sequences ordered
 * longest first, counters, an error word).  When d_k = d_v = 128 and the
 * num_seqs x H (sequence, head) units fill at most half of the current
 * device's SMs (and num_seqs <= 128), the value also covers the operand ring
 * of the producer / consumer prefill kernel (tens of MB at most; the size
 * depends on the SM count).  Returns 0 when num_seqs < 1. */
size_t kda_prefill_workspace_bytes(int32_t num_seqs, int32_t H, int32_t d_k,
                                   int32_t d_v);

/* Chunked prefill over packed variable-length sequences.
 *
 * Computes o_t for every token of every sequence and, optionally, the state
 * after each sequence's last token.  The chunkwise-parallel form used on the
 * GPU ("Kimi 모델 분석", section "순환을 GPU에 올리기": chunks of 64 tokens,
 * intra-chunk matrix products, inter-chunk state carry) gives the same result
 * as the token-by-token recurrence up to rounding.
 *
 *   q, k, v       [T_tot, H, d] in the input dtype of `dtype`
 *   log_alpha     [T_tot, H, d_k] fp32, g = ln(alpha)
 *   beta          [T_tot, H] fp32
 *   S0            [N, H, d_k, d_v] fp32 initial states, or NULL for zeros
 *   cu_seqlens    device int32 [N+1]: cu[0] = 0, non-decreasing,
 *                 cu[N] = total_tokens; sequence n owns tokens
 *                 cu[n] .. cu[n+1]-1.  NULL means one sequence (N must be 1).
 *                 Empty sequences are allowed (their S_final = S0).
 *   num_seqs      N >= 1;  total_tokens >= 0;  H >= 1
 *   o             [T_tot, H, d_v] in the output dtype of `dtype` (written)
 *   S_final       [N, H, d_k, d_v] fp32, or NULL when not wanted.  May alias
 *                 S0 exactly (in-place resume); any other overlap is an error
 *                 the library cannot detect.
 *   workspace     device buffer of at least 256 + 256 * ceil(N / 64) bytes
 *                 (the work list), 256-byte aligned; its contents on entry do
 *                 not matter and are overwritten.  It must not be shared by
 *                 calls that may run concurrently.  A workspace of
 *                 kda_prefill_workspace_bytes(...) bytes lets the call use the
 *                 producer / consumer kernel where it applies (see Paths); a
 *                 smaller one selects the single-CTA kernel, with the same
 *                 results.
 *
 * If cu_seqlens violates its contract the kernels write nothing and set the
 * 32-bit word at byte offset 4 of the workspace to a nonzero value (it is
 * cleared to zero by every call that finds cu_seqlens valid).  The 32-bit word
 * at byte offset 8 gets bit 1 set if a wait inside the tensor-core kernel gave
 * up after two seconds (which means a library fault; the kernel then stops
 * early and its outputs are incomplete); the library never clears it, so a
 * caller who wants to watch it zeroes it first.  Both are device-side flags:
 * reading them needs a synchronisation by the caller.
 *
 * Paths: bf16 inputs with d_k = d_v = 128 run on the tensor cores (tcgen05,
 * chunks of 64 tokens).  With few (sequence, head) units (at most half the
 * SM count) and a full-size workspace, one cooperative launch of one CTA per
 * SM splits each chunk's work: producer CTAs compute the parts that do not
 * depend on the state and hand them, through the workspace, to one consumer
 * CTA per unit that carries the state; otherwise one CTA per unit does both.
 * Every other supported shape, and every call made while the environment
 * variable KDA_FORCE_SIMT is set, runs the fp32 CUDA-core path (chunks of 16
 * tokens).  All paths compute the same result up to rounding (the two
 * tensor-core kernels bit for bit).
 */
kda_status_t kda_prefill(const void *q, const void *k, const void *v,
                         const float *log_alpha, const float *beta,
                         const float *S0, const int32_t *cu_seqlens,
                         int32_t num_seqs, int64_t total_tokens, int32_t H,
                         int32_t d_k, int32_t d_v, kda_dtype_t dtype, void *o,
                         float *S_final, void *workspace,
                         size_t workspace_bytes, cudaStream_t stream);

/* kda_prefill that also records prefix states ("snapshots") for a prefix
 * cache: the state of each sequence after every `interval` tokens, which a
 * serving stack stores and later restores with S0 to resume from that prefix
 * ("[논문 리뷰] Kimi K3 Technical Report", section 13, the KDA-aware prefix
 * cache; "Kimi 모델 분석", section "요약본 저장 위치").
 *
 * Arguments, layouts and results are those of kda_prefill, plus:
 *   interval      a positive multiple of 64 (so that every snapshot falls on
 *                 a chunk boundary of every path); else KDA_ERR_INVALID_ARG.
 *   snap_offsets  device int32 [N+1] with snap_offsets[0] = 0 and
 *                 snap_offsets[n+1] - snap_offsets[n] = floor(len_n / interval);
 *                 required when cu_seqlens is given, ignored (offset 0)
 *                 otherwise.  Checked on the device: a mismatch is reported
 *                 like an invalid cu_seqlens (workspace word at byte 4, nothing
 *                 written).
 *   snapshots     device fp32 [snap_offsets[N], H, d_k, d_v] (written).
 *                 Snapshot j of sequence n, at snap_offsets[n] + j, is the
 *                 state after that sequence's first (j + 1) * interval tokens;
 *                 when interval divides the length, the last one equals the
 *                 sequence's S_final.  Must not overlap the other buffers.
 * The outputs o and S_final are those kda_prefill computes, bit for bit. */
kda_status_t kda_prefill_snapshots(const void *q, const void *k, const void *v,
                                   const float *log_alpha, const float *beta,
                                   const float *S0, const int32_t *cu_seqlens,
                                   int32_t num_seqs, int64_t total_tokens,
                                   int32_t H, int32_t d_k, int32_t d_v,
                                   kda_dtype_t dtype, void *o, float *S_final,
                                   int32_t interval, const int32_t *snap_offsets,
                                   float *snapshots, void *workspace,
                                   size_t workspace_bytes, cudaStream_t stream);

/* kda_prefill with the steps in front of the recurrence fused into the
 * kernels ("Kimi 모델 분석", section "커널 최적화": one kernel for the KDA
 * layer): the lower-bounded decay of "[논문 리뷰] Kimi K3 Technical Report",
 * section 3.5,
 *     g = -5 Sigmoid(e^A z),   alpha = exp(g) in (e^-5, 1),
 * and the L2 normalisation of q and k over the key channels (q then
 * multiplied by q_scale, typically d_k^-1/2).
 *
 * Arguments and results are those of kda_prefill, except:
 *   q, k   raw (not normalised) in the input dtype; each row of d_k values
 *          must be nonzero
 *   z      [T_tot, H, d_k] fp32, the gate pre-activation (in place of
 *          log_alpha)
 *   A      [H, d_k] fp32, 16-byte aligned (a per-head A is its value repeated
 *          over the channels); NULL is KDA_ERR_INVALID_ARG
 *   q_scale  the factor applied to the normalised q
 * Normalised q and k enter the products in fp32 before any rounding to the
 * operand precision, so the result is at least as accurate as calling
 * kda_prefill on q, k normalised and rounded by the caller. */
kda_status_t kda_prefill_fused(const void *q, const void *k, const void *v,
                               const float *z, const float *A, const float *beta,
                               const float *S0, const int32_t *cu_seqlens,
                               int32_t num_seqs, int64_t total_tokens, int32_t H,
                               int32_t d_k, int32_t d_v, kda_dtype_t dtype,
                               float q_scale, void *o, float *S_final,
                               void *workspace, size_t workspace_bytes,
                               cudaStream_t stream);

/* Bytes of device workspace kda_prefill_segmented needs for one sequence of
 * total_tokens tokens and H heads cut into `segments` segments (<= 0: the
 * number the call would choose).  When the call would not cut the sequence
 * (see below) this is kda_prefill_workspace_bytes(1, H, d_k, d_v).  The
 * workspace holds, besides kda_prefill's, two fp32 copies of the outputs
 * (8 * total_tokens * H * d_v bytes) and 3 * segments states per head. */
size_t kda_prefill_segmented_workspace_bytes(int64_t total_tokens, int32_t H,
                                             int32_t d_k, int32_t d_v,
                                             int32_t segments);

/* kda_prefill of ONE sequence with its chunks cut into `segments` groups
 * that run at once (chunk-group parallel prefill): the form for a short
 * prompt whose chunk chain, not the amount of work, sets the time.
 *
 * The recurrence carries only the state from chunk to chunk ("Kimi 모델
 * 분석", section "순환을 GPU에 올리기") and is linear in (S, v), so each
 * segment g >= 1 runs twice on the same chunk operands: from S = 0 (its local
 * outputs and final state L_g) and, with v = 0, from S = I (the product
 * Phi_g of its token transitions and, per token, Phi_t^T q_t).  A scan then
 * gives the state entering each segment, S_1 = L_0, S_{g+1} = Phi_g S_g +
 * L_g, and a fix-up adds S_g^T Phi_t^T q_t to the local outputs.  This is the
 * one-GPU form of what "[논문 리뷰] Kimi K3 Technical Report", section 13,
 * calls KDA context parallelism.  The result equals kda_prefill's up to
 * rounding.
 *
 * Arguments and layouts are those of kda_prefill with N = 1 (no cu_seqlens),
 * plus:
 *   segments   the number of segments, >= 2 (used when every segment has a
 *              chunk and the 2 * segments - 1 chains of each head fill at
 *              most half of the SMs), or <= 0 to let the library choose: the
 *              most segments for which those chains fill about a third of
 *              the SMs and every segment has at least 32 chunks (one GB300:
 *              2 at H = 16, 3 at H = 8, 6 at H = 4; none at H >= 24 or below
 *              4,096 tokens, where cutting does not pay).
 *   workspace  kda_prefill_segmented_workspace_bytes(...) bytes, 256-byte
 *              aligned, not shared with concurrent calls.
 * When the shape cannot be cut (not bf16 inputs with d_k = d_v = 128, too
 * many heads for two segments, a single chunk) or the workspace is smaller
 * than that size, the call is kda_prefill, with the same results.  The
 * device-side status words are those of kda_prefill (workspace bytes 4 and
 * 8).  Launches: the work list, the cut prefill, the scan and the fix-up. */
kda_status_t kda_prefill_segmented(const void *q, const void *k, const void *v,
                                   const float *log_alpha, const float *beta,
                                   const float *S0, int64_t total_tokens,
                                   int32_t H, int32_t d_k, int32_t d_v,
                                   kda_dtype_t dtype, void *o, float *S_final,
                                   int32_t segments, void *workspace,
                                   size_t workspace_bytes, cudaStream_t stream);

/* Device staging bytes kda_prefill_host needs for segments of
 * segment_tokens tokens (a multiple of 64): two input and two output segment
 * buffers, two state buffers and a prefill workspace.  0 for bad arguments. */
size_t kda_prefill_host_staging_bytes(int32_t H, int32_t d_k, int32_t d_v,
                                      kda_dtype_t dtype, int64_t segment_tokens);

/* kda_prefill of ONE sequence whose token inputs and output live in HOST
 * memory (a long prompt that arrives from the host).  The sequence is cut into
 * segments of segment_tokens tokens (a positive multiple of 64) that flow
 * through a pipeline: copies in on `h2d`, kda_prefill on `compute` (the state
 * carried from segment to segment, "Kimi 모델 분석", section "순환을 GPU에
 * 올리기": only the state passes between chunks), copies out on `d2h`, so that
 * the three overlap.  The result equals kda_prefill over the whole sequence
 * bit for bit.
 *
 *   q, k, v, log_alpha, beta, o   HOST pointers, layouts of kda_prefill with
 *                 N = 1 (page-locked memory for full copy bandwidth; pageable
 *                 memory works, with slower copies).  Page-locked pages that
 *                 the CPU has never written are mapped for the GPU on first
 *                 access, and the first passes over them copy at a fraction of
 *                 the link rate; buffers the host filled run at full rate.
 *   S0, S_final   DEVICE [H, d_k, d_v] fp32 or NULL, as in kda_prefill
 *   staging       DEVICE buffer of kda_prefill_host_staging_bytes(...) bytes,
 *                 256-byte aligned, not shared with concurrent calls
 *   compute, h2d, d2h  three streams (distinct for overlap).  When `compute`
 *                 is complete, so is everything the call enqueued.  The first
 *                 copy in waits for the work already on `compute` (a previous
 *                 call on the same staging area, the producer of S0).
 * The pipeline fills and drains over one segment, so shorter segments bound
 * the overhead; 16384 tokens keep each segment's launches well above their
 * fixed cost.
 * The call creates six CUDA events and releases them before it returns; it
 * allocates no memory and does not synchronise the host.  Argument errors are
 * returned before anything is enqueued. */
kda_status_t kda_prefill_host(const void *q, const void *k, const void *v,
                              const float *log_alpha, const float *beta,
                              const float *S0, int64_t total_tokens, int32_t H,
                              int32_t d_k, int32_t d_v, kda_dtype_t dtype,
                              void *o, float *S_final, void *staging,
                              size_t staging_bytes, int64_t segment_tokens,
                              cudaStream_t compute, cudaStream_t h2d,
                              cudaStream_t d2h);

/* One decode step for N independent sequences (one new token each): the
 * recurrence above applied once per (sequence, head), state updated in place.
 * Decode reads and writes a fixed 2 * 4 * d_k * d_v bytes of fp32 state per
 * (sequence, head) whatever the context length ("Kimi 모델 분석", section
 * "Decoding이 왜 느린가"); it is memory-bound.
 *
 *   q, k          [N, H, d_k], v: [N, H, d_v], in the input dtype of `dtype`
 *   log_alpha     [N, H, d_k] fp32;  beta: [N, H] fp32
 *   S_inout       [N, H, d_k, d_v] fp32, read and overwritten with S_t
 *   o             [N, H, d_v] in the output dtype of `dtype` (written); must
 *                 not overlap S_inout
 */
kda_status_t kda_decode_step(const void *q, const void *k, const void *v,
                             const float *log_alpha, const float *beta,
                             float *S_inout, int32_t N, int32_t H, int32_t d_k,
                             int32_t d_v, kda_dtype_t dtype, void *o,
                             cudaStream_t stream);

/* kda_decode_step with the gate prologue fused (see kda_prefill_fused): z
 * [N, H, d_k] fp32 in place of log_alpha, A [H, d_k] fp32, raw q and k
 * (nonzero rows), q_scale. */
kda_status_t kda_decode_step_fused(const void *q, const void *k, const void *v,
                                   const float *z, const float *A,
                                   const float *beta, float *S_inout, int32_t N,
                                   int32_t H, int32_t d_k, int32_t d_v,
                                   kda_dtype_t dtype, float q_scale, void *o,
                                   cudaStream_t stream);

/* Several decode tokens per sequence, keeping the state after every token:
 * the verification step of speculative decoding, which must be able to
 * return to the state after any accepted prefix of the draft, since the state
 * is overwritten in place and cannot be truncated ("[논문 리뷰] Kimi K3
 * Technical Report", section 13, speculative decoding replay; "Kimi 모델
 * 분석", section "Dspark 투기적 디코딩").  Token t of each sequence is one
 * decode step (the recurrence above) from the state after token t - 1.
 *
 *   q, k, log_alpha [N, Ts, H, d_k]; v [N, Ts, H, d_v]; beta [N, Ts, H]
 *                   in the dtypes of kda_decode_step
 *   S_in            [N, H, d_k, d_v] fp32, the state before the first token
 *                   (read only)
 *   o               [N, Ts, H, d_v] in the output dtype (written)
 *   states          [N, Ts, H, d_k, d_v] fp32: states[n, t] is the state after
 *                   token t of sequence n (written)
 * No two of S_in, o and states may overlap.  The launch reads S_in once and
 * writes Ts states: 4 (1 + Ts) d_k d_v bytes per (sequence, head). */
kda_status_t kda_decode_multi(const void *q, const void *k, const void *v,
                              const float *log_alpha, const float *beta,
                              const float *S_in, int32_t N, int32_t Ts,
                              int32_t H, int32_t d_k, int32_t d_v,
                              kda_dtype_t dtype, void *o, float *states,
                              cudaStream_t stream);

/* After verification: the state of each sequence after its accepted prefix.
 * S_out[n] = states[n, accept[n] - 1] when accept[n] > 0, else S_in[n]
 * (all heads).  accept: device int32 [N] in [0, Ts] (values outside are
 * clamped).  S_out may be S_in itself (in-place update of the cache) and must
 * not overlap `states`. */
kda_status_t kda_state_gather(const float *states, const float *S_in,
                              const int32_t *accept, int32_t N, int32_t Ts,
                              int32_t H, int32_t d_k, int32_t d_v, float *S_out,
                              cudaStream_t stream);

/* kda_prefill for callers that cannot allocate device memory.
 *
 * The pages have no counterpart to this entry point: it exists for callers
 * that cannot call cudaMalloc, such as an inference engine that plans all of
 * its device memory once at start-up and forbids allocation afterwards, or a
 * plugin host that passes a library only the operation's inputs and outputs.
 *
 * Same arguments, layouts and results as kda_prefill, without the workspace:
 * the work list lives in a fixed scratch array inside the library's device
 * image (about 16 KiB, room for at most 4096 sequences; every GPU that loads
 * the library keeps it until the process exits).  num_seqs above 4096
 * returns KDA_ERR_WORKSPACE.  The first call on each device, with that device
 * current, looks the array's device address up (cudaGetSymbolAddress, which
 * may load the library's device code), so make that first call before any
 * stream capture; the address is looked up again only when the device's
 * current context changes (after cudaDeviceReset, for example).  All calls on
 * a device share the array: calls that may overlap on the GPU race on it and
 * must be ordered by the caller.  Nothing is allocated and nothing in the
 * array needs clearing between calls.  KDA_ERR_CUDA is returned if the
 * device or the array's address cannot be determined.
 *
 * What differs from kda_prefill:
 *  - The device-side status words (invalid cu_seqlens, a wait that gave up)
 *    live in the private array and cannot be read by the caller.  An invalid
 *    cu_seqlens therefore still returns KDA_OK, with o and S_final not
 *    written; a caller that cannot vouch for its cu_seqlens validates it
 *    before the call, or calls kda_prefill.
 *  - The array has room for the work list only, never for the operand ring
 *    of the producer / consumer kernel, so every call takes the one-CTA-per-
 *    (sequence, head) kernel.  The results are the same, but a batch with few
 *    units (one long sequence of 32 heads, say) keeps only that many SMs
 *    busy: several times slower than kda_prefill with a full workspace. */
kda_status_t kda_prefill_noalloc(const void *q, const void *k, const void *v,
                                 const float *log_alpha, const float *beta,
                                 const float *S0, const int32_t *cu_seqlens,
                                 int32_t num_seqs, int64_t total_tokens,
                                 int32_t H, int32_t d_k, int32_t d_v,
                                 kda_dtype_t dtype, void *o, float *S_final,
                                 cudaStream_t stream);

/* ---- Verifying a tree of drafted tokens --------------------------------
 *
 * The KDA layers of a model stand beside layers of softmax attention over a
 * cache ("[논문 리뷰] Kimi K3 Technical Report", section 1: 69 of 93 layers are
 * KDA), and a drafter may propose a tree instead of a chain.  (The other layers of
 * that model are MLA, whose cache is one latent row for all heads: these calls do
 * not read it.  They serve models whose softmax layers keep keys and values per
 * cache head, of 16 to 128 channels.)  One verification
 * step is then: kda_decode_tree in the KDA layers, kda_tree_attention in the
 * others, kda_token_logprobs on the logits; and after the caller has chosen
 * the accepted path, kda_state_gather (with accept[n] = last accepted node + 1)
 * and kda_cache_commit.
 *
 * A tree is given as parent[n][t] (device int32 [N, Ts], Ts <= 64, more is
 * KDA_ERR_UNSUPPORTED): the node that node t follows, an earlier one (< t), or
 * -1 when t follows the context directly.  A node with any other parent, or
 * with an unused parent, is unused: it takes no part and its output is 0, so
 * sequences with fewer nodes fill their rows with -2.  A NULL parent is the
 * chain parent[t] = t - 1.
 *
 * A cache is a pool of num_pages pages of page_size rows of Hkv heads,
 * [num_pages, page_size, Hkv, d], dense within a page, page p starting
 * page_stride elements after page p - 1 (page_stride >= page_size * Hkv * d,
 * a multiple of 16 bytes; ignored for one page).  page_table [N, max_pages] (device int32) names the
 * pages of each sequence in order: position i of sequence n is row i %
 * page_size of page page_table[n][i / page_size].  Entries that no position
 * needs are never read; one that names no page (outside [0, num_pages)) hides
 * its positions from attention and drops rows written to it.  Any page_size
 * >= 1 will do; max_pages * page_size must fit 31 bits. */

/* Bytes of device workspace kda_tree_attention needs (partial results of
 * sequences whose keys are spread over several CTAs; it depends on the SM
 * count, not on N or the lengths).  0 for arguments that kda_tree_attention
 * refuses; Ts * Hq is at most 2^20. */
size_t kda_tree_attention_workspace_bytes(int32_t N, int32_t Ts, int32_t Hq,
                                          int32_t Hkv, int32_t d,
                                          kda_dtype_t dtype);

/* Softmax attention of drafted nodes: node t of sequence n, query head h sees
 * the lengths[n] rows of its sequence in the cache and, among the drafted
 * nodes, its ancestors and itself, all in cache head g = h / (Hq / Hkv):
 *     o = sum_j softmax_j(scale q . k_j) v_j.
 * Ts = 1 is the attention of ordinary decode; a NULL parent a causal block.
 *
 *   q, o          [N, Ts, Hq, d];  k, v: [N, Ts, Hkv, d], the drafted nodes'
 *                 own keys and values (the cache is only read); Hkv divides Hq
 *   parent        see above
 *   k_cache, v_cache, page_table, num_pages, page_size, max_pages, page_stride
 *                 see above; in q's dtype.  May be NULL when num_pages or
 *                 max_pages is 0 (no context).  Rows past lengths[n] are never
 *                 read, whatever they hold.
 *   lengths       device int32 [N], context rows (values outside [0, max_pages
 *                 * page_size] are clamped)
 *   workspace     kda_tree_attention_workspace_bytes(...) bytes, 256-byte
 *                 aligned, not shared with concurrent calls; contents on entry
 *                 do not matter
 * dtype is that of q, k, v and the cache, and of o.  KDA_BF16 with d = 64 or 128
 * and scale > 0 runs on the tensor cores, with probabilities rounded to bf16 for
 * the second product; everything else, and everything when the environment
 * variable KDA_FORCE_SIMT is set, on the CUDA cores in fp32.  The waits of the
 * tensor-core kernel are bounded: one that gives up (after some two seconds) sets
 * the int32 at byte 8 of the workspace, which no call clears, and the rows of o
 * that depended on it are NaN.  An infinity or NaN in a
 * node's k or v reaches the nodes that see it and no others.  The result does
 * not depend on timing (no atomics on values); it may differ in rounding
 * between GPUs with different SM counts. */
kda_status_t kda_tree_attention(const void *q, const void *k, const void *v,
                                const int32_t *parent, const void *k_cache,
                                const void *v_cache, const int32_t *page_table,
                                const int32_t *lengths, int32_t N, int32_t Ts,
                                int32_t Hq, int32_t Hkv, int32_t d,
                                int32_t num_pages, int32_t page_size,
                                int32_t max_pages, int64_t page_stride,
                                kda_dtype_t dtype, float scale, void *o,
                                void *workspace, size_t workspace_bytes,
                                cudaStream_t stream);

/* kda_decode_multi over a tree: node t is one decode step from the state after
 * its parent node (parent -1: from S_in).  Arguments are those of
 * kda_decode_multi, plus parent (see above; NULL is kda_decode_multi itself).
 * states[n, t] of an unused node is not written; its o is 0.  o and states must
 * overlap neither each other nor any input, with a NULL parent too. */
kda_status_t kda_decode_tree(const void *q, const void *k, const void *v,
                             const float *log_alpha, const float *beta,
                             const float *S_in, const int32_t *parent, int32_t N,
                             int32_t Ts, int32_t H, int32_t d_k, int32_t d_v,
                             kda_dtype_t dtype, void *o, float *states,
                             cudaStream_t stream);

/* For each row of logits x, with lse = log sum_i e^{x_i}: the log
 * probabilities x_i - lse of given tokens, the entropy -sum p log p, and the K
 * most probable tokens.
 *
 *   logits        [T, V] in rows of row_stride elements (>= V, any), base
 *                 16-byte aligned; bf16 (KDA_BF16_F32OUT) or fp32 (KDA_FP32)
 *   tokens        device int32 [T, J], J >= 0 (none: NULL)
 *   logprobs      [T, J] fp32 (written); -inf for a token outside [0, V), in
 *                 any row
 *   entropy       [T] fp32 (written) or NULL
 *   top_ids, top_logprobs   [T, K] int32 and fp32 (written), 0 <= K <= min(V,
 *                 32) (more than 32 is KDA_ERR_UNSUPPORTED), most probable
 *                 first, equal logits by the lower index; NULL when K is 0
 * A logit of -inf is a masked token.  A row of nothing but -inf gives -inf log
 * probabilities and entropy 0.  A NaN or +inf logit makes the log
 * probabilities of its row's tokens and its entropy NaN; in the order of top_ids NaN counts as -inf. */
kda_status_t kda_token_logprobs(const void *logits, int64_t row_stride,
                                const int32_t *tokens, int32_t T, int32_t V,
                                int32_t J, int32_t K, kda_dtype_t dtype,
                                float *logprobs, float *entropy,
                                int32_t *top_ids, float *top_logprobs,
                                cudaStream_t stream);

/* The accepted nodes' rows into the cache, for all layers at once: row
 * path[n][i] of k and v goes to position lengths[n] + i of sequence n, for
 * i < count[n].
 *
 *   k, v          [layers, N, Ts, Hkv, d], any dtype code (o's part of it does
 *                 not matter); Ts may be any size
 *   path          device int32 [N, Ts] or NULL (path[i] = i); entries outside
 *                 [0, Ts) are skipped (their position is not written)
 *   count         device int32 [N] or NULL (all Ts), clamped to [0, Ts]
 *   lengths       device int32 [N], rows already there
 *   k_cache, v_cache, page_table, ...   see above; layer l starts layer_stride
 *                 elements after layer l - 1 (>= page_size * Hkv * d, a multiple
 *                 of 16 bytes; ignored for one layer).  Rows past the table or
 *                 to entries that name no page are dropped.  Two sequences must
 *                 not write one row.
 *   new_lengths   [N] (written: lengths + count) or NULL; must not overlap
 *                 lengths, count, path, cu_seqlens (kda_cache_append) or
 *                 page_table, which other CTAs still read
 * k and v must not overlap the cache. */
kda_status_t kda_cache_commit(const void *k, const void *v, const int32_t *path,
                              const int32_t *count, const int32_t *page_table,
                              const int32_t *lengths, int32_t layers, int32_t N,
                              int32_t Ts, int32_t Hkv, int32_t d,
                              int32_t num_pages, int32_t page_size,
                              int32_t max_pages, int64_t page_stride,
                              int64_t layer_stride, kda_dtype_t dtype,
                              void *k_cache, void *v_cache, int32_t *new_lengths,
                              cudaStream_t stream);

/* The same for a packed batch (a prefill): k, v [layers, total_tokens, Hkv, d],
 * sequence n owning rows cu_seqlens[n] .. cu_seqlens[n+1] - 1 (device int32
 * [N+1], as in kda_prefill), which go to positions lengths[n], lengths[n] + 1,
 * and so on.  Rows that cu_seqlens gives to no sequence are dropped; rows before 0
 * or from total_tokens on do not exist and a sequence that ends before it begins
 * has none, in new_lengths too.  (Of sequences that claim the same row one gets
 * it, which is not defined.) */
kda_status_t kda_cache_append(const void *k, const void *v,
                              const int32_t *cu_seqlens, int64_t total_tokens,
                              const int32_t *page_table, const int32_t *lengths,
                              int32_t layers, int32_t N, int32_t Hkv, int32_t d,
                              int32_t num_pages, int32_t page_size,
                              int32_t max_pages, int64_t page_stride,
                              int64_t layer_stride, kda_dtype_t dtype,
                              void *k_cache, void *v_cache, int32_t *new_lengths,
                              cudaStream_t stream);

/* ---- A prompt and its answer in the softmax layers ------------------------
 *
 * What the softmax layers of such a hybrid do beside kda_prefill and
 * kda_decode_step: kda_cache_append_rotary turns a batch's queries and keys to
 * their positions and puts keys and values into the cache's pages, in the model's
 * type or in 8 bits; kda_prompt_attention is the attention of the prompt itself;
 * kda_cache_attention_e4m3 that of later tokens to a cache of 8 bits
 * (kda_tree_attention reads one in the model's type).
 *
 * A token of q has Hq heads of d channels, dense, one of k and v Hkv; from token to
 * token they lie q_stride, k_stride, v_stride elements apart (at least a token's
 * own, a multiple of 16 bytes; ignored for one token), so that they may be views of
 * one projection's output.  d is 16, 32, 64 or 128 and Hkv divides Hq: query head h
 * goes with key head h / (Hq / Hkv).
 *
 * A cache of 8 bits is a pool as above of e4m3 values, with fp32 scales
 * [num_pages, page_size / block, Hkv] for keys and for values: the value is scale *
 * e4m3.  A block of `block` rows (of one page, position i of a sequence being row i
 * % page_size) and head has the scale 2^e with the smallest e >= -126 for which 448
 * * 2^e reaches its largest magnitude, 0 when it has only zeros, NaN (and bytes 0 for
 * the rows that are written then and later) when it has an infinity or NaN.
 * (kda_cache_attention_e4m3 takes any scales that are not negative.)  page_stride
 * counts bytes here. */

/* Bytes of device workspace kda_prompt_attention needs; 0 for arguments that it
 * refuses. */
size_t kda_prompt_attention_workspace_bytes(int32_t num_seqs, int32_t Hq,
                                            int32_t Hkv, int32_t d,
                                            kda_dtype_t dtype);

/* Causal softmax attention over packed sequences: with Lq and Lk rows of queries
 * and keys in a sequence, query i sees its keys 0 .. i + Lk - Lq, so that the
 * queries are the sequence's last (Lk = Lq: a whole prompt; Lk > Lq: its rest
 * behind a prefix).  One that sees no key (Lk < Lq) gives 0.
 *
 *   q, o          [total_tokens, Hq, d] (o dense);  k, v [total_keys, Hkv, d]
 *   cu_seqlens    device int32 [num_seqs + 1], as in kda_prefill, or NULL for one
 *                 sequence of all rows
 *   cu_seqlens_k  the same for k and v; NULL: cu_seqlens is used for them too, and
 *                 total_keys is total_tokens
 *   o             (written) rows that cu_seqlens gives to no sequence keep what they
 *                 hold; must not overlap the inputs.  Rows before 0 or past the last
 *                 do not exist; where offsets fall, so that sequences claim the same
 *                 rows, it is not defined which rows of theirs are written, and from
 *                 which of them.
 *   workspace     kda_prompt_attention_workspace_bytes(...) bytes, 256-byte aligned,
 *                 over none of the above, not shared with concurrent calls; contents on
 *                 entry do not matter.
 *                 Bit 1 of the int32 at byte 8 is set when a wait of the tcgen05
 *                 kernel has given up (after some two seconds), which no call
 *                 clears; the rows of o that depended on it are NaN.
 * dtype is that of q, k, v, and of o.  KDA_BF16 with d = 64 or 128, scale > 0,
 * Hq / Hkv <= 128, Hq <= 2^16 and total_tokens, total_keys <= 2^27 runs on tcgen05,
 * with probabilities rounded to bf16 for the second product; everything else in
 * products of fp16 pairs.  Of a row of q, k or v these hold bf16 values exactly down to
 * 2^-31 of the row's largest, and 22 bits of fp32 ones down to 2^-28; of the
 * probabilities (each times its value row's magnitude) 11 bits for a bf16 output and 22
 * for an fp32 one, down to 2^-20 of a query's largest, and smaller ones to 2^-32 and
 * 2^-43 of that.  Sums are fp32.  When the environment variable KDA_FORCE_SIMT is set
 * everything runs on the CUDA cores in fp32.  An infinity or NaN in a row of k or v
 * reaches the queries that see it and no others.  The result does not depend on
 * timing. */
kda_status_t kda_prompt_attention(const void *q, const void *k, const void *v,
                                  int64_t q_stride, int64_t k_stride,
                                  int64_t v_stride, const int32_t *cu_seqlens,
                                  const int32_t *cu_seqlens_k, int32_t num_seqs,
                                  int64_t total_tokens, int64_t total_keys,
                                  int32_t Hq, int32_t Hkv, int32_t d,
                                  kda_dtype_t dtype, float scale, void *o,
                                  void *workspace, size_t workspace_bytes,
                                  cudaStream_t stream);

/* Rows of a packed batch (a prefill, or one token per sequence) turned to their
 * positions and into a cache: row i of sequence n has position p = lengths[n] + i.
 * Each pair (x, y) of the first rot_dim channels of q and k becomes
 *     (x cos a - y sin a, x sin a + y cos a),  a = p * inv_freq[j],
 * the j-th pair being channels j and j + rot_dim / 2, or 2 j and 2 j + 1
 * (interleaved != 0); the other channels, and v, stay.  The angle is off by 2^-26 of a
 * turn and p |inv_freq[j]| 2^-54 more at most (as much again for a frequency of 1 at position
 * 2^28).
 *
 *   q, q_out      [total_tokens, Hq, d]; Hq = 0 and NULL: k and v only
 *   k, v          [total_tokens, Hkv, d]
 *   k_out         [total_tokens, Hkv, d] (the turned keys) or NULL
 *   q_out, k_out  in dtype, q_out_stride, k_out_stride elements from token to token;
 *                 may be q and k themselves (same stride), must overlap nothing else
 *   cu_seqlens, lengths, page_table, k_cache, v_cache, new_lengths   as in
 *                 kda_cache_append, for one layer (k_cache [num_pages, page_size,
 *                 Hkv, d]).  Rows without a place in the cache are dropped there,
 *                 but turned; those of no sequence, or of one with a negative
 *                 length, are left as they were.
 *   inv_freq      device fp32 [rot_dim / 2], finite; rot_dim is a multiple of 16, 16 .. d
 *   block         0: the cache is in k's dtype, page_stride in elements, and
 *                 the scales are not used.  Else the cache has 8 bits, a scale for
 *                 each `block` rows (1 .. 128, more is KDA_ERR_UNSUPPORTED; it divides
 *                 page_size): see above.
 *                 A block that the sequence has already begun keeps its rows: when
 *                 the new ones need a larger scale they are rounded to it.  Scales of
 *                 such blocks must be those that this call wrote (or other powers
 *                 of two).  Two sequences must not write one block.
 *   new_lengths   [N] (written) or NULL; must overlap no input
 * dtype is that of q, k, v, q_out and k_out (KDA_BF16_F32OUT is KDA_BF16 here); all
 * arithmetic is fp32. */
kda_status_t kda_cache_append_rotary(
    const void *q, const void *k, const void *v, int64_t q_stride,
    int64_t k_stride, int64_t v_stride, const int32_t *cu_seqlens,
    int64_t total_tokens, const float *inv_freq, int32_t rot_dim,
    int32_t interleaved, const int32_t *page_table, const int32_t *lengths,
    int32_t N, int32_t Hq, int32_t Hkv, int32_t d, int32_t num_pages,
    int32_t page_size, int32_t max_pages, int64_t page_stride, int32_t block,
    kda_dtype_t dtype, void *q_out, int64_t q_out_stride, void *k_out,
    int64_t k_out_stride, void *k_cache, void *v_cache, float *k_scales,
    float *v_scales, int32_t *new_lengths, cudaStream_t stream);

/* Bytes of device workspace kda_cache_attention_e4m3 needs; 0 for arguments that
 * it refuses.  It depends on the SM count, not on N or the lengths. */
size_t kda_cache_attention_e4m3_workspace_bytes(int32_t N, int32_t Ts,
                                                int32_t Hq, int32_t Hkv,
                                                int32_t d, kda_dtype_t dtype);

/* Softmax attention of the Ts newest tokens of each sequence (one, or a chain of
 * drafted ones) to a cache of 8 bits that holds them already: token t of sequence
 * n sees rows 0 .. lengths[n] - Ts + t.  One before the first row gives 0, so that
 * a sequence with fewer tokens has them in its last rows.
 *
 *   q, o          [N, Ts, Hq, d], dense; o must not overlap the inputs
 *   k_cache, v_cache, k_scales, v_scales, page_table, num_pages, page_size,
 *   max_pages, page_stride, block   see above; page_size at most 65536 (more is
 *                 KDA_ERR_UNSUPPORTED).  Positions whose table entry names no page are
 *                 hidden.  Rows past lengths[n] do not count, whatever they hold.
 *   lengths       device int32 [N], rows with those of the Ts tokens (values outside
 *                 [0, max_pages * page_size] are clamped)
 *   workspace     kda_cache_attention_e4m3_workspace_bytes(...) bytes, 256-byte
 *                 aligned, not shared with concurrent calls; contents on entry do
 *                 not matter.  Bit 1 of the int32 at byte 8 is set when a wait of the
 *                 kernel has given up (after some two seconds), which no call clears;
 *                 the rows of o that depended on it are NaN.
 * dtype is that of q and of o.  Products are of fp16 pairs: of q's head they hold bf16
 * values exactly down to 2^-31 of its largest, and 22 bits of fp32 ones down to 2^-28; of
 * the probabilities (each times its value's scale) 11 bits for a bf16 output and 22 for
 * an fp32 one, down to 2^-20 of a token's largest, and smaller ones to 2^-32 and 2^-43 of
 * that.  Sums are fp32.
 * A scale of NaN makes the tokens that see a row of its block NaN and no others;
 * an e4m3 code of NaN, which kda_cache_append_rotary never writes, may reach all
 * tokens of its sequence; an infinity or NaN in q makes that head's output NaN.  No
 * atomics: the result does not depend on timing; it may differ in rounding between GPUs
 * with different SM counts, and with the other sequences of the call. */
kda_status_t kda_cache_attention_e4m3(
    const void *q, const void *k_cache, const void *v_cache,
    const float *k_scales, const float *v_scales, const int32_t *page_table,
    const int32_t *lengths, int32_t N, int32_t Ts, int32_t Hq, int32_t Hkv,
    int32_t d, int32_t num_pages, int32_t page_size, int32_t max_pages,
    int64_t page_stride, int32_t block, kda_dtype_t dtype, float scale, void *o,
    void *workspace, size_t workspace_bytes, cudaStream_t stream);

/* A static, human-readable name for a status code (never NULL). */
const char *kda_status_string(kda_status_t status);

#ifdef __cplusplus
}
#endif

#endif /* KDA_H */
