/*
 * kda.h -- C ABI of the MI355X (gfx950) gated delta-rule library, libkda.so.
 *
 * The operator is the diagonal-plus-rank-one recurrence of Kimi Delta
 * Attention and its extensions, as described in "Complex KDA: Understanding
 * and Enhancing the Expressivity of Kimi Delta Attention" (summary page,
 * background "diagonal-plus-rank-one transitions" and core method):
 *
 *   S_t = (I - beta_t k_t k_t^T) Diag(alpha_t) S_{t-1} + beta_t k_t v_t^T
 *   o_t = S_t^T q_t
 *
 * per (sequence, head), with state S in R^{dk x dv} read on the key side
 * (Dual DeltaNet abstract). KDA uses a per-channel gate alpha_t in R^{dk};
 * GDN is the scalar-gate case (one alpha per token and head); Complex KDA
 * allows alpha in [-1, 1] (negative and exactly zero gates) and beta in
 * [0, 2]. The gate is applied first, then the rank-one delta term; there is
 * no query scaling and no key normalisation inside the library.
 *
 * Conventions for every entry point
 *  - All tensor pointers are DEVICE pointers (hipMalloc'd or equivalent),
 *    row-major and contiguous, aligned to their element size. The decode
 *    state S and output o, the forward's q, k, v and gate, and any
 *    workspace, must be 16-byte aligned.
 *    The caller owns every buffer.
 *  - Element type of q, k, v, gate and beta is selected by `dtype`:
 *    KDA_BF16 (bfloat16 bits) or KDA_F32. States S0, S_T, S and outputs o
 *    are always fp32, but for o (h) of kda_linattn_*, kda_swa_*, kda_glr_*
 *    and kda_paged_*, which has that type too.
 *  - `stream` is a hipStream_t (NULL = the default stream). Work is enqueued
 *    and the call returns without synchronising.
 *  - Arguments are validated before any HIP call; nothing is enqueued when
 *    validation fails. Device-side contents (cu_seqlens offsets, NaN/Inf in
 *    inputs) are not checked: NaN/Inf propagate.
 *  - Supported sizes: dk, dv in {16, 32, 64, 128}; chunk in {16, 32, 64}
 *    (kda_swa_*, kda_paged_*: d in {32, 64, 128}; kda_glr_*: any C).
 *  - The library never allocates, frees or synchronises device memory in a
 *    compute call: every call that needs scratch space takes a caller-owned
 *    workspace, and a NULL workspace (or a short one) is KDA_EINVAL.
 *  - Calls are re-entrant and keep no state between calls (the compute-unit
 *    count that picks a state walker is queried from the runtime on each
 *    call). Two calls may run concurrently on different streams if they do
 *    not share output or workspace buffers.
 */
#ifndef KDA_H_
#define KDA_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Status codes. */
#define KDA_OK 0
#define KDA_EINVAL (-1)  /* null required pointer, non-positive size, inconsistent counts, short workspace */
#define KDA_ENOTSUP (-2) /* dk, dv, chunk, dtype or gate_kind outside the supported set */
#define KDA_EALIGN (-3)  /* a pointer violates the alignment rules above */
#define KDA_EHIP (-4)    /* a HIP call failed; see kda_last_hip_error() */
#define KDA_EWAIT (-5)   /* from kda_chunk_fwd_status: a bounded wait in the state pass expired */
#define KDA_ESCRATCH (-6) /* kda_chunk_fwd_noalloc: the call needs more than KDA_NOALLOC_SCRATCH_BYTES */

/* dtype */
#define KDA_F32 0
#define KDA_BF16 1

/* gate_kind */
#define KDA_GATE_CHANNEL 0 /* gate [.., dk]: one alpha per key channel (KDA, Complex KDA) */
#define KDA_GATE_SCALAR 1  /* gate [..]: one alpha per token and head (GDN) */
#define KDA_GATE_HEAD 2    /* gate [H] fp32: one constant alpha per head (kda_linattn_* only) */

/*
 * Bytes of device workspace kda_chunk_fwd needs for these sizes (0 when the
 * arguments are invalid). For packed variable-length input pass the number
 * of sequences N and has_cu_seqlens = 1; the bound then assumes the worst
 * split of T over N sequences.
 */
size_t kda_chunk_fwd_workspace_bytes(int B, int H, int T, int dk, int dv, int chunk, int N,
                                     int has_cu_seqlens, int dtype);

/*
 * Chunkwise-parallel forward over whole sequences (the pages' chunkwise WY
 * training form of this family; Complex KDA summary, background and core
 * method; Gated DeltaNet-2 blurb). Produces exactly the token recurrence above
 * up to floating-point rounding.
 *
 * Layouts (fixed-length batch; cu_seqlens == NULL):
 *   q, k   [B, T, H, dk]      v    [B, T, H, dv]
 *   gate   [B, T, H, dk] (KDA_GATE_CHANNEL) or [B, T, H] (KDA_GATE_SCALAR)
 *   beta   [B, T, H]
 *   o      [B, T, H, dv] fp32 (output; must not alias any input)
 *   S0     [B, H, dk, dv] fp32 initial state, or NULL for zeros
 *   S_T    [B, H, dk, dv] fp32 final state, or NULL; may alias S0
 * Packed variable-length input (cu_seqlens != NULL): B must be 1; cu_seqlens
 * is a DEVICE int32 array of N+1 non-decreasing offsets with cu_seqlens[0] = 0
 * and cu_seqlens[N] = T; sequence s covers tokens [cu_seqlens[s],
 * cu_seqlens[s+1]) and starts from S0[s] (or zeros); S0 and S_T are
 * [N, H, dk, dv]. With cu_seqlens == NULL, N must equal B (or be 0).
 *
 * chunk (16, 32 or 64) sets the block size of the parallel form; results
 * agree across chunk sizes up to rounding. T need not be a multiple of it.
 *
 * workspace: device memory of at least kda_chunk_fwd_workspace_bytes(...)
 * bytes, owned by the caller and not read before it is written (required:
 * NULL or too small is KDA_EINVAL). Its first 4 bytes receive the call's
 * status word once the call's kernels have run: 0 when every bounded wait in
 * the state pass completed. The state pass's waves trade operands through LDS
 * with bounded waits that cannot expire while all waves of a workgroup run;
 * if one ever did, that wave stores neither o nor S_T and sets the status
 * word. The caller may read the word after synchronising with `stream` and
 * map it with kda_chunk_fwd_status().
 *
 * Returns KDA_OK or a negative status.
 */
int kda_chunk_fwd(const void* q, const void* k, const void* v, const void* gate, const void* beta,
                  const float* S0, float* o, float* S_T, int B, int H, int T, int dk, int dv, int chunk,
                  const int32_t* cu_seqlens, int N, int dtype, int gate_kind, void* workspace,
                  size_t workspace_bytes, void* stream);

/*
 * kda_chunk_fwd for callers that cannot allocate device memory (work recorded
 * under graph capture, allocation-free serving loops, harnesses that forbid
 * hipMalloc): the same arguments and results minus the workspace, which here
 * is a fixed device array of KDA_NOALLOC_SCRATCH_BYTES inside the library,
 * one per GPU, held until the process ends. A call whose workspace would
 * exceed it (kda_chunk_fwd_workspace_bytes(...) > KDA_NOALLOC_SCRATCH_BYTES;
 * about 1,770 (chunk, head) blocks at dk = dv = 128, chunk 64, e.g. H = 16
 * and T = 7,000) returns KDA_ESCRATCH before any HIP call. The call allocates
 * nothing; the first call with a device current looks up the array's address
 * on that device. All calls on one GPU share the array, which keeps the last
 * call's contents (its status word included): calls that overlap on one GPU
 * (concurrent streams, or host threads) race and must be ordered by the
 * caller.
 */
#define KDA_NOALLOC_SCRATCH_BYTES (128u << 20)
int kda_chunk_fwd_noalloc(const void* q, const void* k, const void* v, const void* gate, const void* beta,
                          const float* S0, float* o, float* S_T, int B, int H, int T, int dk, int dv, int chunk,
                          const int32_t* cu_seqlens, int N, int dtype, int gate_kind, void* stream);

/*
 * Maps the status word a forward left in the first 4 bytes of its workspace
 * (read by the caller after the call completed) to KDA_OK (0) or KDA_EWAIT.
 * Host-only; touches no device.
 */
int kda_chunk_fwd_status(uint32_t status_word);

/* stage for kda_chunk_fwd_stage */
#define KDA_STAGE_PREP 1  /* in-chunk work: gate products, gated Gram, UT inverse -> workspace */
#define KDA_STAGE_STATE 2 /* sequential state pass over the chunks: reads the workspace, writes o, S_T */
#define KDA_STAGE_ALL 3   /* both, in order (what kda_chunk_fwd does) */

/*
 * kda_chunk_fwd split into its two launches, for callers that schedule or
 * time them separately. Arguments as for kda_chunk_fwd. KDA_STAGE_STATE
 * consumes a workspace that a KDA_STAGE_PREP call with identical arguments
 * filled earlier on the same stream (or with ordering the caller provides).
 * KDA_STAGE_PREP writes neither o nor S_T and clears the status word;
 * KDA_STAGE_STATE only ever sets it.
 */
int kda_chunk_fwd_stage(int stage, const void* q, const void* k, const void* v, const void* gate,
                        const void* beta, const float* S0, float* o, float* S_T, int B, int H, int T, int dk,
                        int dv, int chunk, const int32_t* cu_seqlens, int N, int dtype, int gate_kind,
                        void* workspace, size_t workspace_bytes, void* stream);

/*
 * One recurrent decode step for N sequences, state updated in place (the
 * pages' recurrent inference form with constant memory per sequence; Gated
 * DeltaNet-2 blurb; Complex KDA summary, background):
 *   S' = Diag(alpha) S;  u = beta (v - S'^T k);  S <- S' + k u^T;  o = S^T q.
 *
 * Layouts: q, k [N, H, dk]; v [N, H, dv]; gate [N, H, dk] or [N, H];
 * beta [N, H]; S [N, H, dk, dv] fp32 (read and written in place);
 * o [N, H, dv] fp32 (must not alias S or the inputs).
 * The state layout equals kda_chunk_fwd's S_T, so a forward's final state
 * feeds decode directly.
 *
 * Returns KDA_OK or a negative status.
 */
int kda_decode_step(const void* q, const void* k, const void* v, const void* gate, const void* beta,
                    float* S, float* o, int N, int H, int dk, int dv, int dtype, int gate_kind,
                    void* stream);

/*
 * Decoupled erase and write gates (Gated DeltaNet-2 blurb: the delta rule's
 * memory update split into a channel-wise erase gate and a channel-wise
 * write gate; the pages name combining them with Complex KDA's gates as
 * future work, Complex KDA summary). The pages give no formula; the form
 * implemented keeps the update rank one along k and gives beta's two roles to
 * two gates:
 *   S_t = (I - k_t (e_t o k_t)^T) Diag(alpha_t) S_{t-1} + k_t (w_t o v_t)^T
 *   o_t = S_t^T q_t
 * with the erase gate e_t in R^{dk} (per key channel) and the write gate w_t
 * in R^{dv} (per value channel); e_t = w_t = beta_t (every channel) gives the
 * recurrence at the top of this header. Any alpha the forward takes is
 * allowed (channel or scalar gate, signs and zeros included).
 *
 * kda_chunk_fwd_ew: the chunkwise forward of that form. Arguments as for
 * kda_chunk_fwd, with beta replaced by
 *   erase [B, T, H, dk] and write [B, T, H, dv] in the input dtype,
 * both 16-byte aligned; the workspace is kda_chunk_fwd_workspace_bytes(...)
 * bytes (same status word). kda_decode_step_ew: one decode step of it, as
 * kda_decode_step with erase [N, H, dk] and write [N, H, dv].
 * Returns KDA_OK or a negative status.
 */
int kda_chunk_fwd_ew(const void* q, const void* k, const void* v, const void* gate, const void* erase,
                     const void* write, const float* S0, float* o, float* S_T, int B, int H, int T, int dk, int dv,
                     int chunk, const int32_t* cu_seqlens, int N, int dtype, int gate_kind, void* workspace,
                     size_t workspace_bytes, void* stream);
int kda_decode_step_ew(const void* q, const void* k, const void* v, const void* gate, const void* erase,
                       const void* write, float* S, float* o, int N, int H, int dk, int dv, int dtype, int gate_kind,
                       void* stream);

/*
 * Bytes of device workspace kda_chunk_bwd needs for these sizes (0 when the
 * arguments are invalid). Arguments as for kda_chunk_fwd_workspace_bytes.
 */
size_t kda_chunk_bwd_workspace_bytes(int B, int H, int T, int dk, int dv, int N, int has_cu_seqlens);

/*
 * Gradient of kda_chunk_fwd. The pages measure forward-plus-backward
 * training throughput of this family (Complex KDA summary, efficiency) but
 * print no backward; this is the reverse-mode derivative of the token
 * recurrence in the header comment, for the loss
 *   L = sum_t <o_t, dO_t> + sum_seq <S_T, dS_T>,
 * computed in fp32 from the same inputs (the forward states are recomputed
 * from q, k, v, gate, beta and S0; nothing from a forward call is reused).
 *
 * Inputs: q, k, v, gate, beta, S0, cu_seqlens, N, dtype and gate_kind as for
 * kda_chunk_fwd; dO [B, T, H, dv] fp32 (required when T > 0); dS_T
 * [N, H, dk, dv] fp32 or NULL (zero).
 * Outputs (fp32, written in full, must not alias inputs or each other):
 *   grad_q, grad_k [B, T, H, dk]   grad_v [B, T, H, dv]
 *   grad_gate      [B, T, H, dk] (KDA_GATE_CHANNEL) or [B, T, H] (KDA_GATE_SCALAR)
 *   grad_beta      [B, T, H]
 *   grad_S0        [N, H, dk, dv], or NULL when not wanted
 * dO, grad_v, S0, dS_T and grad_S0 must be 16-byte aligned.
 *
 * workspace: at least kda_chunk_bwd_workspace_bytes(...) bytes (state
 * checkpoints every 8 tokens, 4 * dk * dv bytes each per (sequence, head),
 * the per-token residual v - S'^T k, plus per-workgroup partial sums);
 * required (NULL is KDA_EINVAL).
 *
 * Returns KDA_OK or a negative status.
 */
int kda_chunk_bwd(const void* q, const void* k, const void* v, const void* gate, const void* beta,
                  const float* S0, const float* dO, const float* dS_T, float* grad_q, float* grad_k,
                  float* grad_v, float* grad_gate, float* grad_beta, float* grad_S0, int B, int H, int T,
                  int dk, int dv, const int32_t* cu_seqlens, int N, int dtype, int gate_kind,
                  void* workspace, size_t workspace_bytes, void* stream);

/*
 * Gradient of kda_chunk_fwd_ew (decoupled erase and write gates; Gated
 * DeltaNet-2 blurb, and the reading stated at kda_chunk_fwd_ew), by the same
 * token-recurrence method as kda_chunk_bwd: with the read key ke = e o k and
 * u = w o v - S'^T ke, the adjoint of each token reads the state with ke,
 * writes along k, and has no beta. Loss, inputs, dO, dS_T, grad_q, grad_k,
 * grad_v, grad_gate and grad_S0 as for kda_chunk_bwd (erase and write as for
 * kda_chunk_fwd_ew, same dtype as q). Outputs in place of grad_beta (fp32,
 * written in full): grad_erase [B, T, H, dk] and grad_write [B, T, H, dv]
 * (16-byte aligned). workspace: kda_chunk_bwd_ew_workspace_bytes(...) bytes
 * (as for kda_chunk_bwd, with one more partial sum per key channel instead of
 * the partial sums of dbeta); required. Every dk and dv of kda_chunk_fwd.
 * Returns KDA_OK or a negative status.
 */
size_t kda_chunk_bwd_ew_workspace_bytes(int B, int H, int T, int dk, int dv, int N, int has_cu_seqlens);
int kda_chunk_bwd_ew(const void* q, const void* k, const void* v, const void* gate, const void* erase,
                     const void* write, const float* S0, const float* dO, const float* dS_T, float* grad_q,
                     float* grad_k, float* grad_v, float* grad_gate, float* grad_erase, float* grad_write,
                     float* grad_S0, int B, int H, int T, int dk, int dv, const int32_t* cu_seqlens, int N, int dtype,
                     int gate_kind, void* workspace, size_t workspace_bytes, void* stream);

/*
 * The same gradient as kda_chunk_bwd (same arguments, outputs and layouts),
 * computed chunk by chunk (the pages' chunkwise algorithm with gate-aware
 * backpropagation for this family; Gated DeltaNet-2 blurb): per 64-token
 * chunk the gated Gram matrices, the UT inverse X = (I + Diag(beta) G)^{-1} and
 * W = X (beta o Gamma o K) in fp32; the state at every chunk start by a
 * forward walk over the chunks and the adjoint at every chunk end by a
 * reverse walk; then every chunk's gradients in parallel, all contractions on
 * fp32 MFMA. The gate gradient uses products of gates only, so exact zero and
 * negative gates have their ordinary derivatives. Supported: dk 64 or 128
 * (KDA_ENOTSUP otherwise), dv in {16, 32, 64, 128}, both dtypes and gate kinds,
 * packed sequences. dO and the workspace must be 16-byte aligned (dO rows are
 * read four values at a time); element alignment suffices for every other
 * pointer. workspace: kda_chunk_bwd_cw_workspace_bytes(...) bytes (per
 * (chunk, head) the chunk's fp32 matrices, the state and adjoint at its
 * boundaries, the chunk's U and dU, and the gradient intermediates);
 * required.
 */
size_t kda_chunk_bwd_cw_workspace_bytes(int B, int H, int T, int dk, int dv, int N, int has_cu_seqlens);
int kda_chunk_bwd_cw(const void* q, const void* k, const void* v, const void* gate, const void* beta,
                     const float* S0, const float* dO, const float* dS_T, float* grad_q, float* grad_k,
                     float* grad_v, float* grad_gate, float* grad_beta, float* grad_S0, int B, int H, int T,
                     int dk, int dv, const int32_t* cu_seqlens, int N, int dtype, int gate_kind,
                     void* workspace, size_t workspace_bytes, void* stream);

/*
 * Gauge transform of Complex KDA onto positive gates (Complex KDA summary,
 * method step 5: the cumulative gate signs are absorbed into queries and
 * keys). Per sequence, head and key channel (per sequence and head for the
 * scalar gate), with s_t = -1 where gate_t < 0 and +1 otherwise (zero and
 * -0.0 included) and c_t = s_1 ... s_t:
 *   q_out_t = c_t q_t,  k_out_t = c_t k_t,  gate_out_t = |gate_t|
 * Running the recurrence on the outputs gives the same o as on the inputs,
 * and a final state whose rows differ by c_T: S_T = Diag(c_T) S~_T.
 * Every output value is an input value with its sign changed or cleared
 * (bit-exact in both dtypes). Layouts, N, cu_seqlens, dtype and gate_kind as
 * for kda_chunk_fwd; outputs have the input layouts and dtype and must not
 * alias the inputs. q, k, their outputs and (channel gate) gate and gate_out
 * must be 16-byte aligned. sign_T: device int8 [N, H, dk] (channel gate) or [N, H]
 * (scalar gate) receiving c_T (+1 / -1), or NULL. workspace: at least
 * kda_gauge_fold_workspace_bytes(...) bytes (required).
 * Returns KDA_OK or a negative status.
 */
size_t kda_gauge_fold_workspace_bytes(int B, int H, int T, int dk, int N, int has_cu_seqlens, int gate_kind);
int kda_gauge_fold(const void* q, const void* k, const void* gate, void* q_out, void* k_out, void* gate_out,
                   int8_t* sign_T, int B, int H, int T, int dk, const int32_t* cu_seqlens, int N, int dtype,
                   int gate_kind, void* workspace, size_t workspace_bytes, void* stream);

/*
 * kda_chunk_fwd computed through the gauge transform: kda_gauge_fold into
 * the workspace, the chunkwise forward on the folded (positive-gate)
 * inputs, then S_T's rows multiplied by c_T. Same arguments, results and
 * tolerances as kda_chunk_fwd; the workspace (required) is
 * kda_chunk_fwd_gauge_workspace_bytes(...) bytes: the forward's own
 * workspace first (so its status word is again the first 4 bytes), then the
 * folded q, k and gate and the fold's scratch.
 */
size_t kda_chunk_fwd_gauge_workspace_bytes(int B, int H, int T, int dk, int dv, int chunk, int N,
                                           int has_cu_seqlens, int dtype, int gate_kind);
int kda_chunk_fwd_gauge(const void* q, const void* k, const void* v, const void* gate, const void* beta,
                        const float* S0, float* o, float* S_T, int B, int H, int T, int dk, int dv, int chunk,
                        const int32_t* cu_seqlens, int N, int dtype, int gate_kind, void* workspace,
                        size_t workspace_bytes, void* stream);

/*
 * Linear attention with a decay for each head: the recurrence without the
 * delta term,
 *   S_t = a_t S_{t-1} + k_t v_t^T,   o_t = S_t^T q_t,
 * for layers that sit beside the delta rule's in one model. Layouts of q, k,
 * v, S0, S_T, cu_seqlens and N as for kda_chunk_fwd, so states and packed
 * batches are shared. gate_kind: KDA_GATE_SCALAR (gate [B, T, H] in the input
 * dtype) or KDA_GATE_HEAD (gate [H], fp32 whatever the dtype: decays near one
 * have no bf16 neighbours). Any decay is allowed, zero and negative ones
 * included, as long as the product of the decays over every run of a sequence's
 * tokens is finite in fp32 (it is wherever they are at most one in magnitude):
 * these products are formed directly, whatever they multiply. There is no
 * query scaling.
 *
 * Unlike the delta rule's calls, o and the gradients have the input dtype
 * (bf16 halves what the call writes); states are fp32. S_T may be S0. Rows of o
 * at or behind cu_seqlens[N] are left as they are. A NaN or Inf at a token reaches every
 * later output of its sequence, and may reach earlier ones of its block of 64
 * tokens.
 *
 * q, k, v, o and the workspace must be 16-byte aligned, states to their
 * element. H <= 65535 and B * (T + 128) (packed: N * (T + 128)) < 2^31;
 * KDA_ENOTSUP otherwise. workspace: at least
 * kda_linattn_fwd_workspace_bytes(...) bytes (segment states), required; no
 * status word is kept in it. Returns KDA_OK or a negative status.
 */
size_t kda_linattn_fwd_workspace_bytes(int B, int H, int T, int dk, int dv, int N, int has_cu_seqlens, int dtype);
int kda_linattn_fwd(const void* q, const void* k, const void* v, const void* gate, const float* S0, void* o,
                    float* S_T, int B, int H, int T, int dk, int dv, const int32_t* cu_seqlens, int N, int dtype,
                    int gate_kind, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Gradient of kda_linattn_fwd for L = sum_t <o_t, dO_t> + sum_seq <S_T, dS_T>.
 * dO [B, T, H, dv] in the input dtype; dS_T [N, H, dk, dv] fp32 or NULL (zero).
 * Outputs: grad_q, grad_k, grad_v and grad_gate in the input dtype and
 * layouts, grad_S0 fp32 or NULL when not wanted. With KDA_GATE_HEAD the decay
 * is a constant: grad_gate must be NULL (a learned one goes in per token, in
 * the input dtype, and its gradient is summed; with bf16 inputs that rounds it,
 * 0.999 to 1, and with fp32 inputs it does not). grad_gate is the derivative
 * with respect to the decay itself, an ordinary one at zero and negative decays. Nothing of a forward
 * call is reused, and rows at or behind cu_seqlens[N] are left as they are. dO
 * and the gradients must be 16-byte aligned (grad_gate and
 * states: their element). workspace: kda_linattn_bwd_workspace_bytes(...)
 * bytes (segment states, and the adjoint of every block), required. At most
 * 4,000,000 sequences (KDA_ENOTSUP beyond what one launch takes).
 */
size_t kda_linattn_bwd_workspace_bytes(int B, int H, int T, int dk, int dv, int N, int has_cu_seqlens, int dtype);
int kda_linattn_bwd(const void* q, const void* k, const void* v, const void* gate, const float* S0, const void* dO,
                    const float* dS_T, void* grad_q, void* grad_k, void* grad_v, void* grad_gate, float* grad_S0,
                    int B, int H, int T, int dk, int dv, const int32_t* cu_seqlens, int N, int dtype, int gate_kind,
                    void* workspace, size_t workspace_bytes, void* stream);

/*
 * One step of the same recurrence for N sequences, S [N, H, dk, dv] fp32
 * updated in place (16-byte aligned; every other pointer to its element).
 * q, k [N, H, dk]; v, o [N, H, dv] in the input dtype; gate [N, H] in the
 * input dtype (KDA_GATE_SCALAR) or [H] fp32 (KDA_GATE_HEAD). o must not alias
 * S or the inputs. N * H * min(dk * dv / 4, 512) < 2^32 (KDA_ENOTSUP otherwise).
 */
int kda_linattn_decode_step(const void* q, const void* k, const void* v, const void* gate, float* S, void* o, int N,
                            int H, int dk, int dv, int dtype, int gate_kind, void* stream);

/*
 * Softmax attention over a sliding window with sinks, for the local layers of
 * models that mix them with the recurrences above. Row i of a sequence sees
 * the keys j <= i with i - j < window, and the first `sinks` keys (j < sinks)
 * always; window >= 1 counts the row itself, so that no row is empty. A window
 * of at least the sequence's length is causal attention.
 *   o_i = sum_j softmax_j(scale q_i . k_j) v_j,  lse_i = log sum_j exp(scale q_i . k_j)
 *
 * Layouts: q, o [B, T, Hq, d]; k, v [B, T, Hkv, d] in the input dtype, Hq a
 * multiple of Hkv (query head h reads kv head h / (Hq / Hkv)); lse [B, T, Hq]
 * fp32 or NULL; cu_seqlens and N as for kda_chunk_fwd, rows at or behind
 * cu_seqlens[N] are left as they are. d in {32, 64, 128}; scale finite. o and
 * the gradients have the input dtype. Sums and softmax statistics are fp32;
 * bf16 inputs enter the second product with probabilities rounded to bf16.
 * Sums are divided by that of the exponentials at the end: 256 times the sum
 * of |v| over the keys that a row sees has to be finite in fp32 (the step of one
 * token: the sum itself).
 *
 * A NaN or Inf in k or v of a token that a row does not see does not reach
 * that row in the forward and the decode step.
 *
 * Every pointer 16-byte aligned (lse, cu_seqlens: their element). At most
 * 65,535 sequences and heads, N * (T + 128) < 2^31, and fewer than 2^24 blocks of
 * 64 rows over all sequences and query heads (KDA_ENOTSUP otherwise).
 * Needs no workspace. Returns KDA_OK or a negative status.
 */
int kda_swa_fwd(const void* q, const void* k, const void* v, void* o, float* lse, int B, int Hq, int Hkv, int T, int d,
                int window, int sinks, float scale, const int32_t* cu_seqlens, int N, int dtype, void* stream);

/*
 * Gradient of kda_swa_fwd for L = sum <o, dO>: o and lse as the forward left
 * them (with bf16 inputs o is not read: its rounding would enter every
 * gradient), dO [B, T, Hq, d]. grad_q, grad_k, grad_v in the input dtype and
 * layouts, those of a kv head summed over its query heads; sums run in a fixed
 * order (repeated calls agree bit for bit); rows at or behind cu_seqlens[N] are
 * left as they are. workspace: kda_swa_bwd_workspace_bytes(...) bytes, required.
 * Besides kda_swa_fwd's sizes: fewer than 2^24 pairs of a kv head and a block of 64
 * keys, where each block with sinks of a sequence of more than window + 64 tokens
 * counts once more for every part that its rows are cut into, together at most 64 a
 * sequence (KDA_ENOTSUP otherwise).
 */
size_t kda_swa_bwd_workspace_bytes(int B, int Hq, int Hkv, int T, int d, int window, int sinks, int N,
                                   int has_cu_seqlens);
int kda_swa_bwd(const void* q, const void* k, const void* v, const void* o, const float* lse, const void* dO,
                void* grad_q, void* grad_k, void* grad_v, int B, int Hq, int Hkv, int T, int d, int window, int sinks,
                float scale, const int32_t* cu_seqlens, int N, int dtype, void* workspace, size_t workspace_bytes,
                void* stream);

/*
 * One token for each of N sequences over caches of constant size: K_cache,
 * V_cache [N, sinks + window, Hkv, d]. Position p of a sequence has slot p
 * (p < sinks) or sinks + (p - sinks) % window. pos [N] int32 on the device is
 * the position of the new token (the number of tokens before it); the call
 * writes k, v [N, Hkv, d] to its slot and attends q [N, Hq, d] over the slots
 * held so far, itself included. pos < 0 marks a sequence to leave out (a
 * padded batch): its cache is not touched, its o [N, Hq, d] is zero. Slots
 * that hold no token yet are never read. pos is not changed by the call.
 * workspace: kda_swa_decode_workspace_bytes(...) bytes, required; calls that
 * may overlap (two streams, two captured graphs) need one each.
 */
size_t kda_swa_decode_workspace_bytes(int N, int Hq, int Hkv, int d, int window, int sinks);
int kda_swa_decode_step(const void* q, const void* k, const void* v, void* K_cache, void* V_cache, const int32_t* pos,
                        void* o, int N, int Hq, int Hkv, int d, int window, int sinks, float scale, int dtype,
                        void* workspace, size_t workspace_bytes, void* stream);

/*
 * The caches that kda_swa_decode_step continues from after a prompt: k, v
 * [B, T, Hkv, d] (or packed, as above) to the slots of their positions, the
 * newest where several share one. Slots without a position are left as they
 * are. The next token's pos is the sequence's length.
 */
int kda_swa_cache_fill(const void* k, const void* v, void* K_cache, void* V_cache, int B, int Hkv, int T, int d,
                       int window, int sinks, const int32_t* cu_seqlens, int N, int dtype, void* stream);

/*
 * Gated linear recurrence for each channel,
 *   h_t = a_t h_{t-1} + x_t,
 * for layers whose state is a vector: the recurrence without keys and values.
 * Layouts: gate, x, h [B, T, C]; h0, h_T [N, C] fp32 (NULL: from zero; not
 * wanted); cu_seqlens and N as for kda_chunk_fwd. h has the type of x (`dtype`),
 * states are fp32. gate_dtype: KDA_F32, or KDA_BF16 with bf16 x (decays near one
 * have no bf16 neighbours, so that fp32 decays go with either). Any decay is
 * allowed, zero and negative ones included, as long as the products of the decays
 * over runs of a sequence's tokens, which are formed directly, stay within fp32: no
 * run's product may overflow, nor one that falls below fp32's smallest number be
 * brought back by decays larger than one behind it (1e-25, 1e-25, then 1e25 may pass
 * nothing on). Decays of magnitude up to one are never in question. h_T may be h0, h
 * must not alias an input. Rows of h at or behind cu_seqlens[N] are left as they are.
 * A NaN or Inf at a token reaches the later outputs of its sequence and channel, no
 * others. Tokens follow each other: of a tree of drafts (kda_paged_attn) each branch
 * is a sequence of its own here, from the state of the tokens before it.
 *
 * C <= 2^20, and N * (T + 128) < 2^31; KDA_ENOTSUP beyond, and where blocks of
 * 128 tokens (64 where C is no multiple of 8, fp32 x: of 4) and 64 channels are
 * more than one launch takes. Arrays of rows are 16-byte aligned where C is such a
 * multiple, else to their element; the workspace is 16-byte aligned, states to
 * their element. workspace: kda_glr_fwd_workspace_bytes(...) bytes, required; calls
 * that may overlap (two streams, two captured graphs) need one each. Repeated calls
 * agree bit for bit. Inside a launch blocks wait for what earlier ones leave in the
 * workspace; a wait that never ended is given up after some seconds. Where two calls
 * use a workspace at once, the results of both are undefined (they may be finite and
 * wrong); nothing outside their arrays is touched. Returns KDA_OK or a negative
 * status.
 */
size_t kda_glr_fwd_workspace_bytes(int B, int T, int C, int N, int has_cu_seqlens, int dtype);
int kda_glr_fwd(const void* gate, const void* x, const float* h0, void* h, float* h_T, int B, int T, int C,
                const int32_t* cu_seqlens, int N, int dtype, int gate_dtype, void* workspace, size_t workspace_bytes,
                void* stream);

/*
 * Gradient of kda_glr_fwd for L = sum_t <h_t, dh_t> + sum_seq <h_T, dh_T>: dh
 * [B, T, C] in the type of x, dh_T [N, C] fp32 or NULL (zero). grad_gate in the
 * type of gate, grad_x in that of x, grad_h0 [N, C] fp32 or NULL when not
 * wanted. Nothing of a forward call is reused: the states are formed again in
 * fp32. Outputs must not alias inputs; rows at or behind cu_seqlens[N] are left
 * as they are. A NaN or Inf in x reaches grad_gate of the later tokens only.
 * workspace: kda_glr_bwd_workspace_bytes(...) bytes, required, one for each of the
 * calls that may overlap.
 */
size_t kda_glr_bwd_workspace_bytes(int B, int T, int C, int N, int has_cu_seqlens, int dtype);
int kda_glr_bwd(const void* gate, const void* x, const float* h0, const void* dh, const float* dh_T, void* grad_gate,
                void* grad_x, float* grad_h0, int B, int T, int C, const int32_t* cu_seqlens, int N, int dtype,
                int gate_dtype, void* workspace, size_t workspace_bytes, void* stream);

/*
 * One step of the same recurrence for N sequences: gate, x, o [N, C], h [N, C]
 * fp32 updated in place; o is h in the type of x. Every pointer aligned to its
 * element; o must not alias h or the inputs. N * C < 2^31.
 */
int kda_glr_decode_step(const void* gate, const void* x, float* h, void* o, int N, int C, int dtype, int gate_dtype,
                        void* stream);

/*
 * A paged cache for attention over all of a sequence's tokens. K_pages, V_pages
 * [num_pages, page_size, Hkv, d]; row r of a sequence (its r-th token) lies in
 * page block_table[seq][r / page_size] at r % page_size; block_table
 * [N, table_width] int32 on the device. An entry outside [0, num_pages), and a
 * row behind the table's width, is a page that is not there: nothing is read or
 * written for it. Any page_size; num_pages * page_size < 2^31. ctx_len [N] int32
 * on the device: tokens of the sequence in the cache before the new ones; a
 * negative one leaves the sequence out (a padded batch). New token i of a
 * sequence has row ctx_len + i.
 *
 * New tokens: B sequences of T, or packed (B = 1, cu_seqlens and N as for
 * kda_chunk_fwd; any number of tokens each, none included); rows at or behind
 * cu_seqlens[N] are left as they are. d in {32, 64, 128}; Hq a multiple of Hkv,
 * at most 65,535; N * (T + 128) and (T + 128) * Hq / Hkv < 2^31 (KDA_ENOTSUP
 * beyond). Arrays of rows, pages and the workspace 16-byte aligned, the rest to
 * their element.
 *
 * kda_paged_append: k and v [B, T, Hkv, d] of the new tokens to their rows, k
 * rotated by its position on the way, and q [B, T, Hq, d] rotated to q_out (both
 * NULL: no q; Hq is then not read). The first rot_dim values of a head (a
 * multiple of 16, at most d; 0 with freqs NULL: no rotation) are rotated in
 * pairs, pair i by the angle pos * freqs[i] (freqs [rot_dim / 2] fp32 on the
 * device, radians a token; pos [B, T] int32 on the device, or NULL: the token's
 * row). pairing: KDA_PAIRS_HALVES (i and i + rot_dim / 2) or KDA_PAIRS_NEIGHBOURS
 * (2i and 2i + 1):  (x, y) -> (x cos - y sin, x sin + y cos).  Angles are
 * formed in 64 bits, the rest in fp32, rounded once. v and unrotated values are
 * copied bit for bit. q_out of a sequence that is left out is zero. Two tokens of
 * a call must not have the same row of the same page; q_out may be q.
 */
#define KDA_PAIRS_HALVES 0
#define KDA_PAIRS_NEIGHBOURS 1
int kda_paged_append(const void* q, const void* k, const void* v, const int32_t* pos, const float* freqs, void* q_out,
                     void* K_pages, void* V_pages, const int32_t* block_table, const int32_t* ctx_len, int B, int T,
                     int Hq, int Hkv, int d, int rot_dim, int pairing, int num_pages, int page_size, int table_width,
                     const int32_t* cu_seqlens, int N, int dtype, void* stream);

/*
 * Softmax attention of the new tokens over such a cache, theirs included (they
 * have been appended before): every new token sees the ctx_len rows before them,
 * and of the new ones those that tree names, or with tree NULL those up to
 * itself. tree [B, T, tree_words] int32 on the device: bit j % 32 of word j / 32
 * of a token says that it sees new token j of its sequence (itself where its own
 * bit is set); bits of tokens that the sequence does not have mean nothing, and
 * tokens behind the words are not seen. One token a sequence is decoding, a tree
 * checks drafts, tree NULL with more tokens takes a piece of a prompt.
 *   o_i = sum_j softmax_j(scale q_i . k_j) v_j,  lse_i = log sum_j exp(scale q_i . k_j)
 * q, o [B, T, Hq, d] in the input dtype, query head h reads kv head
 * h / (Hq / Hkv); lse [B, T, Hq] fp32 or NULL; scale finite. o must not alias an
 * input (several workgroups read a row of q, one writes it; o = q is KDA_EINVAL).
 * A row that sees no key has o = 0 and lse = -Inf, as every row of a sequence that
 * is left out.
 * Statistics and sums are fp32, and bf16 probabilities enter the product with v as
 * two bf16 numbers, whatever the number of rows (o is off by little more than its
 * own rounding); 256 times the sum of |v| over the keys that a row sees has to be
 * finite in fp32. A NaN or Inf in a row of the cache reaches no row of o that does
 * not see it. Repeated calls agree bit for bit. workspace:
 * kda_paged_attn_workspace_bytes(...) bytes, required; calls that may overlap
 * (two streams, two captured graphs) need one each (else the results of both are
 * undefined; nothing outside their arrays is touched). Returns KDA_OK or a negative
 * status (KDA_ENOTSUP also where the rows of all heads are more than a launch
 * takes).
 */
size_t kda_paged_attn_workspace_bytes(int B, int T, int Hq, int Hkv, int d, int N, int has_cu_seqlens);
int kda_paged_attn(const void* q, const void* K_pages, const void* V_pages, const int32_t* block_table,
                   const int32_t* ctx_len, const int32_t* tree, int tree_words, void* o, float* lse, int B, int T,
                   int Hq, int Hkv, int d, float scale, int num_pages, int page_size, int table_width,
                   const int32_t* cu_seqlens, int N, int dtype, void* workspace, size_t workspace_bytes, void* stream);

/* Static text for a status code (never NULL). */
const char* kda_strerror(int status);

/* hipError_t of the most recent KDA_EHIP on the calling thread (0 if none). */
int kda_last_hip_error(void);

/* Library version, e.g. 100 for 0.1.0. */
int kda_version(void);

#ifdef __cplusplus
}
#endif

#endif /* KDA_H_ */
