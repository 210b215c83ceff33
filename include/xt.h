/*
 * xt.h — C ABI of libxt: forward kernels and analytic backward kernels of the ops of a
 * pre-norm transformer block, for one NVIDIA GB300 (sm_103a).
 *
 * Sources (cited by page title and section):
 *   [AE] xtrain "Phase: Autograd Engine + Op Backward — Design Document": op table
 *        (forward / backward of each op), RMSNorm, RoPE, softmax and cross-entropy
 *        derivations, composed attention, tape and gradient accumulation.
 *   [BP] unhomeschool "Träna en språkmodell: Backprop i anpassad CUDA": forward pass of
 *        the GPT-style stack, forward/backward kernel pairs, saved tensors, gradient
 *        buffers with += semantics.
 *   [DO] xtrain "Phase T18: Dropout (device RNG + mask) — Design Document": counter-based
 *        RNG, per-site seeds, train/eval switch, residual-path wiring.
 *
 * Conventions shared by every entry point
 *   - Return value: XT_OK (0) or an xt_status code; xt_last_error() gives a message
 *     (thread-local, valid until the next call on the same thread).
 *   - Pointers: DEVICE pointers owned by the caller, unless a comment says "host".
 *     The library never allocates or frees memory.  Scratch space ("ws") is caller
 *     memory of at least the size the matching *_workspace_size() reports; its contents
 *     on entry do not matter, except for the matmul and block workspaces, whose first
 *     4096 bytes must be zero before their first use (every call leaves them zero).
 *   - stream: a cudaStream_t passed as void* (NULL = legacy default stream).  Every call
 *     only enqueues work on it and returns; nothing synchronises, except
 *     xt_get_device_errors().
 *   - Layout: row-major, contiguous unless a leading dimension (ld, in elements) is given.
 *     "rows, cols": x is [rows, cols].  Weights are [in, out] and a linear layer is y = x @ W.
 *   - dtype: XT_F32 or XT_BF16 storage; arithmetic is float32 (GEMMs: tf32 or bf16
 *     tensor-core products with float32 accumulation).  Saved statistics (inv_rms, mean,
 *     rstd, lse) are always float32.  Token ids and targets are int32.
 *   - accumulate flags: 0 ⇒ dst = g; 1 ⇒ dst += g ([AE] § 梯度累加: first push sets,
 *     later pushes add; [BP] § Ackumulation över mikrobatcher: backward adds into the
 *     gradient buffers).
 *   - Vector paths need 16-byte aligned pointers; misaligned pointers are still handled
 *     (a scalar path) unless a function says otherwise.  Sizes are validated on the host;
 *     invalid arguments return XT_ERR_INVALID_ARG before anything is launched.
 *   - Errors detected on the device (an id or target outside [0, V), a bounded wait that
 *     gave up) set bits in a device flag word read by xt_get_device_errors(); the offending
 *     element is skipped (its output row is written as NaN where one exists).
 */
#ifndef XT_H
#define XT_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  XT_OK = 0,
  XT_ERR_INVALID_ARG = 1,
  XT_ERR_UNSUPPORTED = 2,
  XT_ERR_ALIGNMENT = 3,
  XT_ERR_CUDA = 4,
  XT_ERR_TIMEOUT = 5
} xt_status;

typedef enum { XT_F32 = 0, XT_BF16 = 1 } xt_dtype;

/* device error flag bits */
#define XT_DEVERR_INDEX 1u   /* a token id or target outside [0, V) */
#define XT_DEVERR_TIMEOUT 2u /* a bounded mbarrier wait in a GEMM gave up */
#define XT_DEVERR_PLAN 4u    /* masked attention (or the sorted embedding gradient) was given a plan made for other sizes */

const char* xt_last_error(void);
const char* xt_version(void);

/* Synchronises `stream`, then copies the device flag word to *out (host pointer).
 * Returns XT_ERR_TIMEOUT if the timeout bit is set, XT_OK otherwise. */
int xt_get_device_errors(uint32_t* out, void* stream);
int xt_clear_device_errors(void* stream);

/* Number of CUDA kernels libxt has launched in this process (host-side counter). */
uint64_t xt_launch_count(void);

/* Limit, in nanoseconds, of the bounded waits inside the tensor-core kernels (the GEMM and the
 * fused attention) on work from their other roles: TMA copies landing, MMAs completing, an
 * accumulator being drained, a stream-K partial being published.  A wait that runs out sets
 * XT_DEVERR_TIMEOUT in the device flag; the kernel then stops issuing work, waits (with the
 * default limit) for the copies and MMAs it already issued, releases its tensor memory and
 * returns, so the context stays usable.  Process-wide; read when a launch is enqueued (a
 * captured graph keeps the value it was captured with).  ns = 0 restores the default of 2 s.
 * Limits under 1 ms poll without suspending (for tests of the give-up paths).  After a
 * give-up the outputs are undefined, and a stream-K matmul workspace may hold stale flag
 * words: zero it before its next use.  Always returns XT_OK. */
int xt_set_wait_limit_ns(uint64_t ns);
uint64_t xt_get_wait_limit_ns(void);

/* GEMM timing for measurement: with capacity > 0, the next `capacity` GEMM launches each get
 * a record tagged with its algorithmic FLOPs (2·M·N·K per batch; for the causal modes only the
 * unmasked half) and a region of a device buffer in which every CTA of the GEMM kernel (and of
 * a K split's reduce kernel) writes %globaltimer when it starts work (after its wait for the
 * preceding kernel) and when it has finished.  No event or extra node enters the stream, so the
 * launches keep their programmatic dependent-launch overlap.  The buffer (capacity × 32 KB) is
 * allocated by this call on the current device, not during the launches; capacity 0 disables
 * recording (the buffer is kept for reuse).  Launches captured into a CUDA graph keep their
 * region, so every replay rewrites it (the read returns the latest replay's timings); a graph
 * captured with profiling on should not be replayed after a later xt_profile_gemm call.
 * xt_profile_gemm_read
 * synchronises the device and copies up to max_records records into host arrays: flops,
 * milliseconds (latest end minus earliest start over the record's CTAs), and (if shapes !=
 * NULL) 8 ints per record: M, N, K, batches, tile width BN (1000 + BN for the paired-CTA
 * kernel), A MN-major, B MN-major, schedule code (causal mode, 10 × K splits, 1000 for
 * stream-K over every unit, 1000 + s for s lockstep K slices).  *n receives the number
 * recorded. */
int xt_profile_gemm(int capacity);
int xt_profile_gemm_read(double* flops, float* ms, int* shapes, int max_records, int* n);

/* ---------------------------------------------------------------------------------
 * Gradient accumulation ([AE] § 梯度累加, push_grad/accumulate): dst[i] += src[i].
 * dst and src may have different dtypes (e.g. bf16 src into an f32 dst).
 * ------------------------------------------------------------------------------- */
int xt_accumulate(void* dst, int dt_dst, const void* src, int dt_src, int64_t n, void* stream);
/* dst[i] = src[i] converted between dtypes (bf16 results round to nearest even). */
int xt_convert(void* dst, int dt_dst, const void* src, int dt_src, int64_t n, void* stream);

/* ---------------------------------------------------------------------------------
 * Elementwise ops, [AE] op table rows add / mul / scale.  n elements, one dtype.
 * Backward grads may be NULL to skip them.
 * ------------------------------------------------------------------------------- */
int xt_add_fwd(const void* a, const void* b, void* y, int64_t n, int dt, void* stream);
/* da = d, db = d (copy or accumulate) */
int xt_add_bwd(const void* d, void* da, void* db, int64_t n, int dt, int acc_a, int acc_b,
               void* stream);
int xt_mul_fwd(const void* a, const void* b, void* y, int64_t n, int dt, void* stream);
/* da = d∘b, db = d∘a.  a and b may be the same pointer (mul(x, x)). */
int xt_mul_bwd(const void* d, const void* a, const void* b, void* da, void* db, int64_t n,
               int dt, int acc_a, int acc_b, void* stream);
int xt_scale_fwd(const void* x, void* y, int64_t n, float alpha, int dt, void* stream);
/* dx = d·alpha */
int xt_scale_bwd(const void* d, void* dx, int64_t n, float alpha, int dt, int acc, void* stream);

/* Full sum to one float32 (device pointer `out`), deterministic two-stage reduction.
 * Needed by the validation loss L = Σ W∘out ([AE] § 验证方法). */
int xt_sum_workspace_size(int64_t n, size_t* bytes);
int xt_sum_fwd(const void* x, int64_t n, int dt, float* out, void* ws, void* stream);
/* dx[i] = *upstream (device float32 scalar) */
int xt_sum_bwd(const float* upstream, void* dx, int64_t n, int dt, int acc, void* stream);

/* ---------------------------------------------------------------------------------
 * add_bias ([AE] op table row add_bias): y[r,c] = x[r,c] + bias[c];
 * backward dx = d (if dx != NULL), dbias[c] = Σ_r d[r,c], summed in a fixed order
 * (per-CTA partials in ws, then one ordered pass).  bias / dbias have dtype dt_bias.
 * ------------------------------------------------------------------------------- */
int xt_colsum_workspace_size(int64_t rows, int64_t cols, size_t* bytes);
int xt_add_bias_fwd(const void* x, const void* bias, void* y, int64_t rows, int64_t cols, int dt,
                    void* stream);
int xt_add_bias_bwd(const void* d, void* dx, void* dbias, int64_t rows, int64_t cols, int dt,
                    int dt_bias, void* ws, int acc_dx, int acc_dbias, void* stream);

/* ---------------------------------------------------------------------------------
 * Activations.  silu ([AE] op table row silu): y = x·σ(x), dx = d·(σ + x·σ·(1−σ)).
 * swiglu ([AE] op table row swiglu): y = silu(g)∘u with g the gate; g and u may be
 * column blocks of one buffer (row strides ld_in), grads likewise (ld_grad).
 * gelu (exact, erf form; [BP] § kernel-pair table, k_mlp_fwd/bwd; backward reads the saved
 * pre-activation, [BP] § Sparade tensorer): y = x·Φ(x), dx = d·(Φ(x) + x·φ(x)).
 * ------------------------------------------------------------------------------- */
int xt_silu_fwd(const void* x, void* y, int64_t n, int dt, void* stream);
int xt_silu_bwd(const void* d, const void* x, void* dx, int64_t n, int dt, int acc, void* stream);
int xt_swiglu_fwd(const void* g, const void* u, int64_t ld_in, void* y, int64_t ld_out,
                  int64_t rows, int64_t cols, int dt, void* stream);
int xt_swiglu_bwd(const void* d, int64_t ld_d, const void* g, const void* u, int64_t ld_in,
                  void* dg, void* du, int64_t ld_grad, int64_t rows, int64_t cols, int dt,
                  int acc, void* stream);
int xt_gelu_fwd(const void* x, void* y, int64_t n, int dt, void* stream);
int xt_gelu_bwd(const void* d, const void* x, void* dx, int64_t n, int dt, int acc, void* stream);

/* ---------------------------------------------------------------------------------
 * RMSNorm ([AE] § RMSNorm): ir = 1/√(mean_c x² + eps), y = x·ir·γ, inv_rms[r] = ir saved.
 * Backward, g = d∘γ: dx = ir·g − x·ir³/n·Σ_c g·x; dγ[c] = Σ_r d·x·ir.
 * d, x, gamma have dtype dt; dx has dtype dt_dx (dt, or XT_F32 with bf16 inputs: a float32
 * residual-gradient buffer); dgamma has dtype dt_param.  dx or dgamma may be NULL.
 * ------------------------------------------------------------------------------- */
int xt_norm_bwd_workspace_size(int64_t rows, int64_t cols, size_t* bytes);
int xt_rms_norm_fwd(const void* x, const void* gamma, void* y, float* inv_rms, int64_t rows,
                    int64_t cols, float eps, int dt, void* stream);
int xt_rms_norm_bwd(const void* d, const void* x, const void* gamma, const float* inv_rms,
                    void* dx, void* dgamma, int64_t rows, int64_t cols, int dt, int dt_dx,
                    int dt_param, void* ws, int acc_dx, int acc_param, void* stream);

/* Allocation-free variant of xt_rms_norm_bwd (the pages have no counterpart: it exists for
 * callers, not for the method).  Some callers cannot allocate device memory where they run
 * the backward: for example a plug-in inside a host framework that owns all device memory
 * through its own pool and hands out no scratch, or a latency-critical loop in which
 * cudaMalloc (which can synchronise the device) is not allowed.  They still pass d, x, gamma,
 * inv_rms, dx and dgamma as for xt_rms_norm_bwd; the dγ partial sums go to a fixed scratch
 * array inside libxt instead of a ws buffer.  Results equal xt_rms_norm_bwd's up to the
 * summation order of dγ (at most 128 partial rows here).
 *   - Limit: cols ≤ 8192 (else XT_ERR_UNSUPPORTED); the scratch is 128 × 8192 floats (4 MiB),
 *     held by every GPU that loads libxt until the process exits.
 *   - The first call on each device looks the scratch's device address up with that device
 *     current (cudaGetSymbolAddress); make that first call before any stream capture.  The
 *     address is kept for the life of the process: after cudaDeviceReset on a device (which
 *     reloads libxt's device code there, possibly elsewhere) do not call this entry point on
 *     that device again in the same process.
 *   - At most 128 blocks walk the rows (the scratch holds one partial row per block), against
 *     up to 4 per SM for xt_rms_norm_bwd: on long inputs it is correspondingly slower.
 *   - No cudaMalloc, cudaFree or allocating library routine is called.  Nothing in the
 *     scratch needs to start at zero: each call overwrites every partial row it reads.
 *   - All calls share the one array: calls that overlap on the GPU (several streams or host
 *     threads) race on it and must be serialised by the caller. */
int xt_rms_norm_bwd_noalloc(const void* d, const void* x, const void* gamma, const float* inv_rms,
                            void* dx, void* dgamma, int64_t rows, int64_t cols, int dt, int dt_dx,
                            int dt_param, int acc_dx, int acc_param, void* stream);

/* LayerNorm (standard definition; [BP] § kernel-pair table k_layernorm_fwd/bwd and
 * § Sparade tensorer: mean and variance saved — saved here as mean and rstd):
 * μ = mean x, var = mean (x−μ)², rstd = 1/√(var+eps), x̂ = (x−μ)·rstd, y = x̂·γ + β.
 * Backward, g = d∘γ: dx = rstd·(g − mean g − x̂·mean(g∘x̂)); dγ = Σ_r d∘x̂; dβ = Σ_r d.
 * Dtypes as for xt_rms_norm_bwd. */
int xt_layernorm_fwd(const void* x, const void* gamma, const void* beta, void* y, float* mean,
                     float* rstd, int64_t rows, int64_t cols, float eps, int dt, void* stream);
int xt_layernorm_bwd(const void* d, const void* x, const void* gamma, const float* mean,
                     const float* rstd, void* dx, void* dgamma, void* dbeta, int64_t rows,
                     int64_t cols, int dt, int dt_dx, int dt_param, void* ws, int acc_dx,
                     int acc_param, void* stream);

/* ---------------------------------------------------------------------------------
 * RoPE ([AE] op table row rope and § RoPE 反向推导): for each pair (i, i+h), h = hd/2,
 * θ = s·base^(−2i/hd):  y_i = x_i cos θ − x_{i+h} sin θ;  y_{i+h} = x_{i+h} cos θ + x_i sin θ.
 * Backward is the transposed rotation: dx_i = d_i cos + d_{i+h} sin, dx_{i+h} = d_{i+h} cos − d_i sin.
 * xt_rope_table fills table[2][S][hd/2] (cos then sin, float32, angles in float64) for
 * positions pos_offset + s.  Token (b, s) head h lives at x + (b·S + s)·ld + h·hd.
 * x and y may alias (in place).  hd must be even.
 * ------------------------------------------------------------------------------- */
int xt_rope_table(float* table, int S, int hd, double base, int pos_offset, void* stream);
int xt_rope_fwd(const void* x, void* y, const float* table, int B, int S, int H, int hd,
                int64_t ld, int dt, void* stream);
int xt_rope_bwd(const void* d, void* dx, const float* table, int B, int S, int H, int hd,
                int64_t ld, int dt, int acc, void* stream);

/* RoPE over several axes: positions are given per token and per axis (time, height and width of a
 * patch; one axis: positions that restart with each document of a packed row).  pos is int32
 * [n_axes][T] (1 to 4 axes), sections a HOST array of n_axes pair counts adding up to hd/2: the
 * pairs i = 0 .. hd/2 − 1 belong to the axes in order.  θ = pos[axis(i)][t]·f_i with
 * f_i = base^(−2i/hd) (per_axis = 0), or base^(−k/sections[a]) for pair k of axis a (per_axis = 1);
 * the rotation and its backward are xt_rope_fwd's.  Angles are reduced exactly (integer arithmetic
 * modulo a turn), so any int32 position is as accurate as position 0 (base >= 1).  Token t, head h lives at
 * x + t·ld_x + h·hd (y + t·ld_y + h·hd); x and y may be one buffer with one stride (in place), except
 * with acc = 1.  hd even and at most 256 (else XT_ERR_INVALID_ARG / XT_ERR_UNSUPPORTED). */
int xt_rope_axes_fwd(const void* x, int64_t ld_x, void* y, int64_t ld_y, const int32_t* pos, int n_axes,
                     const int32_t* sections, int per_axis, double base, int64_t T, int H, int hd, int dt,
                     void* stream);
int xt_rope_axes_bwd(const void* d, int64_t ld_d, void* dx, int64_t ld_dx, const int32_t* pos, int n_axes,
                     const int32_t* sections, int per_axis, double base, int64_t T, int H, int hd, int dt, int acc,
                     void* stream);

/* ---------------------------------------------------------------------------------
 * Row-wise safe softmax ([AE] op table row softmax and § Softmax 反向推导):
 * y = exp(x − max)/Σ exp(x − max); dx = y∘(d − Σ_c d∘y).
 * causal: 0 = no mask; 1 = row r is query s = r mod q_len and columns c > s are masked
 * (y = 0 there, written); 2 = as 1, but only columns c < min(cols, 128·(⌊s/128⌋+1)) are
 * read or written (the layout the causal attention GEMMs consume; entries beyond are
 * left untouched).
 * ------------------------------------------------------------------------------- */
int xt_softmax_fwd(const void* x, void* y, int64_t rows, int64_t cols, int causal, int64_t q_len,
                   int dt, void* stream);
int xt_softmax_bwd(const void* d, const void* y, void* dx, int64_t rows, int64_t cols, int causal,
                   int64_t q_len, int dt, int acc, void* stream);

/* ---------------------------------------------------------------------------------
 * Fused attention ([AE] § Attention 用组合: per (batch, head) scores = Q Kᵀ·(1/√hd),
 * P = softmax(scores), O = P V; backward dV = Pᵀ dO, dP = dO Vᵀ, dS = softmax_bwd(dP, P),
 * dQ = dS K·(1/√hd), dK = dSᵀ Q·(1/√hd)), computed tile by tile on the tensor cores without
 * writing P: the same values as the composition up to rounding (P is rounded to bf16 before
 * it multiplies V, as in the composed bf16 path).
 *
 * Layout: token t = b·S + s is row t of each matrix; head h of q, k, v occupies columns
 * [h·hd, h·hd + hd) of its row, rows ld_qkv elements apart (q, k, v may be column blocks of
 * one [T, 3·H·hd] buffer); o and d_o likewise with ld_o; dq, dk, dv with ld_dqkv.
 * causal: 1 masks key c from query s when c > s (the masked probabilities are 0); 0 none.
 * lse (float32 [B][H][S], written by the forward, read by the backward) is the natural-log
 * normaliser log Σ_c exp(scores[s, c]) over the visible keys.
 * dq, dk, dv are overwritten.  The backward's workspace (xt_attention_bwd_workspace_size)
 * holds D = Σ_c dO∘O per (b, h, s).  o_lo (optional, may be NULL; bf16, the layout and row
 * stride of o) receives O − bf16(O) rounded to bf16, so o + o_lo holds O to ~2⁻¹⁶ relative;
 * passed to the backward it is part of the O that D is formed from, which keeps the rows of
 * dS summing to ~0 (with the bf16 O alone they carry its 2⁻⁹ rounding as a bias).
 * Supported: dt = XT_BF16, hd = 64, row strides multiples of 8 elements, all pointers
 * 16-byte aligned (else XT_ERR_UNSUPPORTED / XT_ERR_ALIGNMENT).  Device-side waits are
 * bounded; on expiry XT_DEVERR_TIMEOUT is set in the device error flag.
 * ------------------------------------------------------------------------------- */
int xt_attention_fwd(const void* q, const void* k, const void* v, int64_t ld_qkv, void* o, void* o_lo,
                     int64_t ld_o, float* lse, int B, int S, int H, int hd, int causal, int dt, void* stream);
int xt_attention_bwd_workspace_size(int B, int S, int H, size_t* bytes);
int xt_attention_bwd(const void* q, const void* k, const void* v, int64_t ld_qkv, const void* o,
                     const void* o_lo, const void* d_o, int64_t ld_o, const float* lse, void* dq, void* dk,
                     void* dv, int64_t ld_dqkv, void* ws, size_t ws_bytes, int B, int S, int H, int hd,
                     int causal, int dt, void* stream);

/* ---------------------------------------------------------------------------------
 * Masked attention over packed documents, forward and backward: for training on rows that hold several
 * texts or images.  T tokens; query head h reads key / value head h / (H / Hkv) (Hkv divides H):
 *   a_ij = scale·q_i·k_j,  c = cap·tanh(a/cap) (cap > 0; else a),  s = c − slopes[h]·|i − j| (slopes != NULL),
 *   P = softmax of s_i over the keys that i sees,  O = P V,  lse_i = log Σ exp s_ij;
 *   D_i = dO_i·O_i,  dS = P∘(dO Vᵀ − D)∘(1 − tanh²),  dQ = scale·dS K,  dK = scale·dSᵀ Q,  dV = Pᵀ dO
 *   (dK and dV are sums over the query heads that share them; slopes are constants).
 * What i sees is the plan's: keys of its own document's valid tokens, with causal = 1 only those at or
 * before i and those of the document's prefix.  A token outside every document's valid part sees nothing and
 * is not seen: O = 0, lse = −∞, gradients 0; its rows of q, k, v and d_o may hold anything.  NaN or ∞ in a
 * token reaches only the rows that see it.
 *
 * xt_attention_plan makes the plan of a batch, which every layer's forward and backward then use:
 *   doc_off  int32 [n_docs + 1], ascending token offsets; document d spans [doc_off[d], doc_off[d+1]).  NULL:
 *            n_docs spans of T / n_docs tokens (T a multiple of n_docs).
 *   doc_len  int32 [n_docs], tokens of the span that count (the rest is padding); NULL: all.
 *   prefix   int32 [n_docs], leading tokens that every token of the document sees (causal = 1; more than the
 *            document has means all); NULL: none.
 * plan: xt_attention_plan_size(T) bytes, 16-byte aligned, a function of these arrays' values when the call
 * runs.  Offsets that fall or leave [0, T], lengths outside the span and negative prefixes set
 * XT_DEVERR_INDEX; no access depends on them.  A plan made for another T sets XT_DEVERR_PLAN and the
 * attention call writes nothing.  Only T is checked: the backward must find the plan that its forward had, so a buffer is
 * not filled for the next batch (of as many tokens) before the last one's backward has been queued on the stream.
 *
 * Layout: token t of q is row t (ld_q elements apart), its head h columns [h·hd, h·hd + hd); k, v likewise
 * with Hkv heads, o, d_o and dq as q, dk and dv as k.  lse: float32 [H][T].  scale = 0 means 1/√hd.
 * Gradients are overwritten.  The backward takes the forward's o and lse; o's bf16 rounding does not reach the
 * gradients (D is formed again from P and dP in float32; xt_attention_bwd wants the residual o_lo for that).  Its
 * workspace holds D and lse by whole tiles (and partial sums where few shared key heads are split over the GPU).
 * Outputs, inputs, the plan and the workspace must not overlap (views of one buffer's columns do not).
 * Supported: dtype = XT_BF16, hd 64 or 128, row strides multiples of 8 elements, all pointers 16-byte
 * aligned, T and n_docs < 2³⁰, cap ≤ 1024 (capped scores are resolved to 1.2e-4 there) and not so small
 * that scale/cap overflows (else XT_ERR_UNSUPPORTED / XT_ERR_ALIGNMENT / XT_ERR_INVALID_ARG).  Deterministic: equal
 * calls give equal bits.  A document's last bits depend on where it lies in the row (its place among 128-token tiles)
 * and, with a cap, on the values beside it (2⁻²³ of the cap).  Device-side waits are bounded (XT_DEVERR_TIMEOUT).
 * ------------------------------------------------------------------------------- */
typedef struct xt_attention_desc {
  int64_t T;
  int32_t H, Hkv, hd, dtype;
  float scale;         /* 0: 1/sqrt(hd) */
  float cap;           /* at most 1024; 0: scores are not capped */
  const float* slopes; /* device, [H], or NULL: no distance bias */
} xt_attention_desc;

int xt_attention_plan_size(int64_t T, size_t* bytes);
int xt_attention_plan(int64_t T, int n_docs, const int32_t* doc_off, const int32_t* doc_len, const int32_t* prefix,
                      int causal, void* plan, size_t plan_bytes, void* stream);
int xt_attention_masked_fwd(const xt_attention_desc* desc, const void* plan, size_t plan_bytes, const void* q,
                            int64_t ld_q, const void* k, int64_t ld_k, const void* v, int64_t ld_v, void* o,
                            int64_t ld_o, float* lse, void* stream);
int xt_attention_masked_bwd_workspace_size(const xt_attention_desc* desc, size_t* bytes);
int xt_attention_masked_bwd(const xt_attention_desc* desc, const void* plan, size_t plan_bytes, const void* q,
                            int64_t ld_q, const void* k, int64_t ld_k, const void* v, int64_t ld_v, const void* o,
                            int64_t ld_o, const void* d_o, int64_t ld_do, const float* lse, void* dq,
                            int64_t ld_dq, void* dk, int64_t ld_dk, void* dv, int64_t ld_dv, void* ws, size_t ws_bytes,
                            void* stream);

/* ---------------------------------------------------------------------------------
 * Cross-entropy, mean over rows ([AE] op table row cross_entropy, § Cross-entropy 反向推导):
 * loss = (1/R) Σ_r (lse_r − x[r, t_r]);  dx = upstream·(softmax(x_r) − onehot(t_r))/R.
 * lse (float32 [rows]) is saved by the forward; `loss` and `upstream` are device float32
 * scalars.  dlogits may alias logits (in place) when dt_grad == dt.
 * ------------------------------------------------------------------------------- */
int xt_cross_entropy_workspace_size(int64_t rows, size_t* bytes);
/* Forward and backward in one pass over the logits (for the loss at the root of a training
 * graph): the results of xt_cross_entropy_fwd followed by xt_cross_entropy_bwd with acc = 0
 * (lse, loss, dlogits; dlogits may be logits), up to float32 summation order.  Each row is
 * held in shared memory while its lse and gradient are formed, so the logits are read from
 * HBM once.  Rows of more than 200 KB (e.g. 128256 bf16 logits) are split across a cluster of
 * 2, 4 or 8 CTAs, each holding its chunk of the row; the chunks' (max, Σ exp) pairs are
 * exchanged through distributed shared memory and merged in rank order.  Rows whose length
 * is not a multiple of 16 bytes, or buffers not 16-byte aligned, take the two-kernel path. */
int xt_cross_entropy_fwd_bwd(const void* logits, const int32_t* targets, float* lse, float* loss,
                             const float* upstream, void* dlogits, int64_t rows, int64_t V, int dt,
                             int dt_grad, void* ws, void* stream);
int xt_cross_entropy_fwd(const void* logits, const int32_t* targets, float* lse, float* loss,
                         int64_t rows, int64_t V, int dt, void* ws, void* stream);
/* The fan-out of [AE] § 梯度累加 fused: one logits tensor x [rows, V] consumed by three ops
 * whose scalar results are added, L = CE(x) + c_lin·Σx + c_sq·Σ(x∘x), forward and backward in
 * one pass over x.  The gradient is the sum of the three consumers' contributions times the
 * upstream gradient u of L (device float32 scalar; NULL means 1, the loss at the root):
 *   grad (+)= u·((softmax(x_r) − onehot(t_r))/rows + c_lin + 2·c_sq·x)   (float32, [rows, V]),
 * written once (acc = 1 adds it to grad's contents: later pushes add).  Outputs (device
 * float32): loss = CE mean, sums[0] = Σx, sums[1] = Σx², sums[2] = L; lse [rows].  Rows are
 * split across a cluster of CTAs as in xt_cross_entropy_fwd_bwd; V·element size must be a
 * multiple of 16 bytes and logits / grad 16-byte aligned (XT_ERR_ALIGNMENT).  ws:
 * xt_cross_entropy_fanout_workspace_size bytes.  A target outside [0, V) sets XT_DEVERR_INDEX
 * and makes that row's loss term and gradient NaN. */
int xt_cross_entropy_fanout_workspace_size(int64_t rows, size_t* bytes);
/* Process-wide override of how the one-pass cross-entropy splits wide rows: clusters of cl ∈
 * {1, 2, 4, 8} CTAs with nb ∈ {1, 2} chunk buffers each (where the chunks fit), or (0, 0) for
 * the automatic choice (default).  For measurement and tests; XT_ERR_INVALID_ARG otherwise. */
int xt_ce_set_split(int cl, int nb);
int xt_cross_entropy_fanout_fwd_bwd(const void* logits, const int32_t* targets, float c_lin, float c_sq,
                                    const float* upstream, float* lse, float* loss, float* sums, void* grad,
                                    int acc, int64_t rows, int64_t V, int dt, void* ws, size_t ws_bytes,
                                    void* stream);
int xt_cross_entropy_bwd(const void* logits, const int32_t* targets, const float* lse,
                         const float* upstream, void* dlogits, int64_t rows, int64_t V, int dt,
                         int dt_grad, int acc, void* stream);

/* ---------------------------------------------------------------------------------
 * Log probabilities of given tokens, with each row's entropy and its most probable tokens: what a loss on the
 * tokens' own probabilities (a policy gradient, a distillation, scoring) needs where the mean cross-entropy does
 * not do.  Per row r, z = scale·x[r] (scale: 1 / temperature), p = softmax(z):
 *   logp[r] = log p[tokens[r]],   entropy[r] = −Σ_v p_v log p_v,
 *   top_logp[r][0..top), top_ids[r][0..top): the largest logits in falling order, equal ones by rising id, and
 *   their log p (top ≤ 32 and ≤ V; 0: none, pointers ignored);
 *   stats[r] = {max x, ln Σ exp(z − scale·max x)}, for the backward.
 * Backward, from d_logp and d_entropy (float32 [rows]; either may be NULL: nought):
 *   dx_v (+)= scale·(d_logp·([v = token] − p_v) − d_entropy·p_v·(log p_v + entropy)).
 * A row whose d_logp and d_entropy are both 0 gets zeros whatever it holds (padding).
 * entropy and stats may be NULL in the forward; the backward needs stats, and entropy where d_entropy is given.
 * Logits of −∞ (banned tokens) have p = 0 and gradient 0, but scale·d_logp where the row's token is one; a row that
 * holds a NaN or +∞, or nothing but −∞, has no distribution: NaN in all its values, −1 as its ids.  Any finite logits
 * are allowed, those of the type's lowest value among them.  A token outside [0, V) sets XT_DEVERR_INDEX and makes logp and the gradient of its row NaN.
 * Layout: row r of logits at logits + r·ld (ld ≥ V), dlogits likewise with ld_d; dlogits may be logits (one dtype
 * and stride, acc = 0).  Any alignment of the element type; rows of aligned 16 bytes need no more than that.
 * scale in [1e-6, 1e6].  No log probability is above 0.  Entropies are accurate to about 1e-6 absolute.  Deterministic.
 * ------------------------------------------------------------------------------- */
int xt_token_logprobs_fwd(const void* logits, int64_t ld, const int32_t* tokens, float scale, int top, float* logp,
                          float* entropy, float* stats, float* top_logp, int32_t* top_ids, int64_t rows, int64_t V,
                          int dt, void* stream);
int xt_token_logprobs_bwd(const void* logits, int64_t ld, const int32_t* tokens, const float* stats,
                          const float* entropy, const float* d_logp, const float* d_entropy, float scale,
                          void* dlogits, int64_t ld_d, int64_t rows, int64_t V, int dt, int dt_grad, int acc,
                          void* stream);

/* ---------------------------------------------------------------------------------
 * Inverted dropout with a counter-based mask ([DO] § RNG：counter-based, § dropout 节点的
 * backward): for flat element index i (uint64),
 *   key = seed ⊕ (i·0x9E3779B97F4A7C15), h = splitmix64(key), u = (h>>40)·2⁻²⁴ (float32),
 *   keep = u ≥ p, y = keep ? x·scale : 0 with scale = float32(1/(1−p)).
 * The backward regenerates the same mask from (seed, i).  p == 0 or training == 0 is an
 * exact copy.  p must be in [0, 1).  xt_dropout_mask writes the keep mask (1/0 bytes).
 * xt_dropout_add_fwd fuses the residual: out = h + dropout(a) (out may alias h).
 * ------------------------------------------------------------------------------- */
int xt_dropout_fwd(const void* x, void* y, int64_t n, float p, uint64_t seed, int training,
                   int dt, void* stream);
int xt_dropout_bwd(const void* d, void* dx, int64_t n, float p, uint64_t seed, int training,
                   int dt, int acc, void* stream);
/* Same, with d of dtype dt_d (e.g. a float32 residual gradient) and dx of dtype dt_dx. */
int xt_dropout_bwd_ex(const void* d, int dt_d, void* dx, int dt_dx, int64_t n, float p,
                      uint64_t seed, int training, int acc, void* stream);
int xt_dropout_mask(uint8_t* mask, int64_t n, float p, uint64_t seed, void* stream);
int xt_dropout_add_fwd(const void* h, const void* a, void* out, int64_t n, float p,
                       uint64_t seed, int training, int dt, void* stream);

enum { XT_NORM_RMS = 0, XT_NORM_LN = 1 };  /* norm kinds (also the block stack's norm field) */

/* ---------------------------------------------------------------------------------
 * The residual path's dropout fused with its neighbouring pre-norm ([DO] § dropout 接在哪
 * (wiring): every residual add of the block is followed by the next sub-block's norm, and
 * every norm backward by the preceding site's dropout backward).  Same masks, same
 * arithmetic, same results as the separate calls, one pass over the rows:
 *   xt_dropout_add_norm_fwd: sum = h + dropout(a) over [rows, cols] (flat index i = r·cols + c,
 *     as xt_dropout_add_fwd), then y = norm(sum as stored) with its statistics:
 *     norm = XT_NORM_RMS: stat0 = inv_rms (xt_rms_norm_fwd; beta, stat1 unused);
 *     norm = XT_NORM_LN:  stat0 = mean, stat1 = rstd (xt_layernorm_fwd).
 *   xt_norm_bwd_dropout: the norm backward (xt_rms_norm_bwd with stat0 = inv_rms, or
 *     xt_layernorm_bwd with stat0 = mean, stat1 = rstd; dx required) that also writes
 *     g = dropout_bwd(dx as stored) (xt_dropout_bwd_ex from dx to g), g of dtype dt.
 * ------------------------------------------------------------------------------- */
int xt_dropout_add_norm_fwd(const void* h, const void* a, void* sum, const void* gamma,
                            const void* beta, void* y, float* stat0, float* stat1, int64_t rows,
                            int64_t cols, float p, uint64_t seed, int training, int norm, float eps,
                            int dt, void* stream);
int xt_norm_bwd_dropout(int norm, const void* d, const void* x, const void* gamma, const float* stat0,
                        const float* stat1, void* dx, void* dgamma, void* dbeta, void* g, int64_t rows,
                        int64_t cols, int dt, int dt_dx, int dt_param, void* ws, int acc_dx,
                        int acc_param, float p, uint64_t seed, int training, void* stream);

/* ---------------------------------------------------------------------------------
 * Embedding ([BP] § kernel-pair table k_embed_fwd/bwd; § Var gradienter lever i minnet):
 * h[t] = E[ids[t]] (+ P[t mod S] when P != NULL).  Backward: dE[v] = Σ_{t: ids[t]=v} dh[t]
 * summed in ascending t (deterministic), dP[s] = Σ_b dh[b·S+s].  With acc == 0 the rows
 * of dE that no token touches are zeroed.  T ≤ 16384.  The workspace (kept for the
 * interface) may be NULL.
 * ------------------------------------------------------------------------------- */
int xt_embedding_workspace_size(int64_t T, size_t* bytes);
int xt_embedding_fwd(const int32_t* ids, const void* E, const void* P, void* h, int64_t T, int S,
                     int64_t d, int64_t V, int dt, void* stream);
int xt_embedding_bwd(const int32_t* ids, const void* dh, void* dE, void* dP, int64_t T, int S,
                     int64_t d, int64_t V, int dt_dh, int dt_grad, void* ws, int acc,
                     void* stream);

/* Embedding lookup with a scale and its gradient by sorted tokens, for any number of tokens T < 2³⁰:
 *   h[t] = scale·E[ids[t]],   dE[v] (+)= scale·Σ_{t: ids[t]=v} dh[t]   (float32 sums, a fixed order: deterministic).
 * xt_embedding_plan sorts a batch's ids once into plan (xt_embedding_plan_size bytes, 16-byte aligned): every table
 * that the batch looks up, and every backward of it, can use that plan.  With acc = 0 rows of dE that no token touches
 * are zeroed.  An id outside [0, V) sets XT_DEVERR_INDEX, its row of h is NaN and its row of dh is left out.  A plan
 * made for another T or V sets XT_DEVERR_PLAN and the backward writes nothing.  The workspace
 * (xt_embedding_sorted_bwd_workspace_size, 16-byte aligned) holds the shares of ids whose tokens are summed in several
 * pieces; its contents on entry do not matter, and one made for a larger T serves any smaller one.  dh, dE, the plan and
 * the workspace must not overlap.  E and h, and dh and dE, may have different dtypes; rows are contiguous, any d
 * (multiples of 8 in 16-byte aligned buffers run on 16-byte accesses). */
int xt_embedding_lookup_fwd(const int32_t* ids, const void* E, void* h, int64_t T, int64_t d, int64_t V, float scale,
                            int dt_e, int dt_h, void* stream);
int xt_embedding_plan_size(int64_t T, size_t* bytes);
int xt_embedding_plan(const int32_t* ids, int64_t T, int64_t V, void* plan, size_t plan_bytes, void* stream);
int xt_embedding_sorted_bwd_workspace_size(int64_t T, int64_t d, size_t* bytes);
int xt_embedding_sorted_bwd(const void* plan, size_t plan_bytes, const void* dh, void* dE, int64_t T, int64_t d,
                            int64_t V, float scale, int dt_dh, int dt_grad, int acc, void* ws, size_t ws_bytes,
                            void* stream);

/* ---------------------------------------------------------------------------------
 * Matmul on the tensor cores ([AE] op table row matmul: C = A@B; dA = d@Bᵀ, dB = Aᵀ@d).
 *   op(A) is M×K: trans_a = 0 ⇒ A stored [M, K] (ld lda); 1 ⇒ A stored [K, M].
 *   op(B) is K×N: trans_b = 0 ⇒ B stored [K, N] (ld ldb); 1 ⇒ B stored [N, K].
 *   C [M, N] (ld ldc) = alpha·op(A)@op(B)  (+ C when accumulate).
 * Two batch levels (outer × inner) with element strides, e.g. (batch, head) for attention.
 * dtype_ab: XT_BF16 (bf16 products) or XT_F32 (tf32 products); dtype_c: XT_F32 or XT_BF16.
 * Requirements (else XT_ERR_ALIGNMENT): A, B 16-byte aligned; lda, ldb and the A/B batch
 * strides are multiples of 16 bytes; C 16-byte aligned and ldc a multiple of 16 bytes.
 * causal (square attention blocks, 128-row granularity): 0 none; 1 skip output tiles
 * entirely above the diagonal block (n0 ≥ m0+128); 2 stop the K loop at m0+128 (A is a
 * causal probability block); 3 start the K loop at m0 (A is a transposed causal block).
 * ------------------------------------------------------------------------------- */
typedef struct xt_matmul_desc {
  int32_t M, N, K;
  int32_t trans_a, trans_b;
  int32_t batch_outer, batch_inner;
  int32_t dtype_ab, dtype_c;
  int32_t accumulate;
  int32_t causal;
  float alpha;
  int64_t lda, ldb, ldc;
  int64_t stride_a_outer, stride_a_inner;
  int64_t stride_b_outer, stride_b_inner;
  int64_t stride_c_outer, stride_c_inner;
} xt_matmul_desc;

/* Scratch bytes the call needs, laid out as
 *   [4096 bytes of stream-K flag words][tf32 staging][partial tiles]:
 *   - flag words: zero before the workspace's first use (e.g. cudaMemset once when it is
 *     allocated); each call leaves them zero.  A stream-K launch's CTAs signal through them
 *     that a partial tile is ready, so two matmul calls must not share a workspace while
 *     both can run (on two streams);
 *   - staging: XT_F32 operands read MN-major (trans_a = 1 or trans_b = 0) are first copied,
 *     transposed, into K-major scratch because the tf32 MMA is fed K-major operands only;
 *   - partial tiles: fp32 partial accumulators of a K split or of the stream-K schedule.
 * The schedule is chosen per problem from a per-tile time model: whole output tiles over
 * persistent CTAs, or (with a workspace, non-causal) a K split reduced in a fixed order by a
 * second kernel, or stream-K: every SM's CTA an equal share of the tiles' k-block
 * iterations, or tiles × s CTAs each computing one K slice of one tile; a tile shared by
 * several CTAs is summed, in CTA order, by the CTA holding its first k-blocks.  All are
 * deterministic.  ws = NULL (or fewer bytes than reported) restricts the choice
 * to whole tiles, and is an error for the tf32 staging case. */
int xt_matmul_workspace_size(const xt_matmul_desc* desc, size_t* bytes);
/* Schedule override for every later matmul call of the process (tests, tuning): 0 the
 * time model's choice (default), 1 whole tiles only, 2 a K split wherever one is allowed,
 * 3 stream-K over every SM wherever allowed, 4 stream-K in lockstep K slices (tiles × s
 * CTAs, each one K slice of one tile) wherever allowed.  XT_ERR_INVALID_ARG otherwise. */
int xt_gemm_set_schedule(int mode);
/* Process-wide override of the paired-CTA GEMM (bf16 operands, no causal mode, no GELU
 * epilogue): two CTAs of a cluster compute one 256-row tile with the paired tensor-core MMA,
 * each staging its own 128 rows of A and half of B's rows.  Its multicast form runs clusters
 * of two such pairs on vertically adjacent 256 × 256 tiles (whole tiles, an even number of
 * 256-row tiles), each CTA loading half of its B rows for both pairs.  0 = the time model's
 * choice (default; never the multicast form, which measured slower than the plain pairs on
 * the 12-layer stack's shapes), 1 = never, 2 = the plain pairs wherever allowed, 3 = the
 * multicast form wherever allowed (else as 2; XT_ERR_UNSUPPORTED where the process sees several GPUs or
 * is one of several ranks, WORLD_SIZE > 1).  The gated block's own products and Muon's choose pairs by their sizes
 * unless the mode is 1.  Every kernel accumulates in fp32 over the same K order; the
 * choice is deterministic for a given shape.  XT_ERR_INVALID_ARG otherwise. */
int xt_gemm_set_pairing(int mode);
/* Process-wide override of the GEMM tile width: 0 = the time model's choice (default), else
 * BN ∈ {64, 128, 192, 256} wherever it is a candidate for the problem (the model's choice
 * otherwise).  For measurement and tests.  XT_ERR_INVALID_ARG for other values. */
int xt_gemm_set_tile(int bn);
int xt_matmul_fwd(const xt_matmul_desc* desc, const void* A, const void* B, void* C, void* ws,
                  size_t ws_bytes, void* stream);
/* Backward of C = alpha·op(A)@op(B) given dC (layout of C, dtype dtype_ab):
 * dA = alpha·dC@op(B)ᵀ into A's layout, dB = alpha·op(A)ᵀ@dC into B's layout; dA/dB have
 * dtype dt_grad_a / dt_grad_b; either may be NULL.  causal must be 0. */
/* The GELU of the MLP ([BP] § Framåtgåendet: the up projection followed by exact GELU) fused
 * into the GEMM epilogue, gelu(a) = a·Φ(a):
 *   xt_matmul_gelu_fwd: C = alpha·op(A)@op(B) (the pre-activation, rounded to bf16) and
 *                       Y = gelu(C) evaluated on that rounded value;
 *   xt_matmul_gelu_bwd: C = (alpha·op(A)@op(B)) ∘ gelu'(X) with gelu'(a) = Φ(a) + a·φ(a),
 *                       X the saved pre-activation (the GELU backward applied to the product).
 * Y and X are bf16 with C's layout (ldc).  Restrictions (else XT_ERR_UNSUPPORTED /
 * XT_ERR_INVALID_ARG): dtype_ab = dtype_c = XT_BF16, one batch, accumulate = 0, causal = 0,
 * N a multiple of 64; Y / X 16-byte aligned.  Workspace as xt_matmul_workspace_size. */
int xt_matmul_gelu_fwd(const xt_matmul_desc* desc, const void* A, const void* B, void* C, void* Y,
                       void* ws, size_t ws_bytes, void* stream);
int xt_matmul_gelu_bwd(const xt_matmul_desc* desc, const void* A, const void* B, const void* X, void* C,
                       void* ws, size_t ws_bytes, void* stream);

int xt_matmul_bwd_workspace_size(const xt_matmul_desc* desc, size_t* bytes);
int xt_matmul_bwd(const xt_matmul_desc* desc, const void* A, const void* B, const void* dC,
                  void* dA, void* dB, int dt_grad_a, int dt_grad_b, int acc_a, int acc_b,
                  void* ws, size_t ws_bytes, void* stream);

/* ---------------------------------------------------------------------------------
 * Gated feed-forward block, bf16, x [T, d], W_up = [Wg | Wu] [d, 2F], W_down [F, d] (the block stack's layout):
 *   g = x Wg,  u = x Wu,  h = act(g)∘u,  y = h W_down        (act: silu, or the exact gelu)
 *   dh = dy W_downᵀ,  dg = dh∘u∘act'(g),  du = dh∘act(g),  dx = dg Wgᵀ + du Wuᵀ,
 *   dW_up = xᵀ [dg | du],  dW_down = hᵀ dy.
 * Both projections, the activation and the product are one kernel; the backward forms dg and du in the epilogue of dh,
 * which is never written.  Forward: gu ([T, 2F]: g and u rounded to bf16, what the backward reads) may be NULL, and y
 * (then w_down too) where only h is wanted.  act is evaluated on the float32 g; h is rounded to bf16 once.
 * Backward: dgu [T, 2F] bf16 is scratch that receives [dg | du]; dx (bf16), dw_up and dw_down (dt_grad) may be NULL.
 * acc_dx, acc_dw: add to what is there.  T = 0: the weights' gradients are 0 (acc_dw = 0).
 * d and F multiples of 8, all pointers 16-byte aligned (else XT_ERR_ALIGNMENT); dt = XT_BF16 (else
 * XT_ERR_UNSUPPORTED).  ws: xt_gated_mlp_workspace_size bytes of matmul workspace (its first 4096 bytes zero before
 * the first use; not shared by calls that can run at once), or NULL as for xt_matmul_fwd.  Outputs must not overlap
 * inputs.  Deterministic; device-side waits are bounded (XT_DEVERR_TIMEOUT).
 * ------------------------------------------------------------------------------- */
enum { XT_GATE_SILU = 0, XT_GATE_GELU = 1 };
int xt_gated_mlp_workspace_size(int64_t T, int64_t d, int64_t F, size_t* bytes);
int xt_gated_mlp_fwd(const void* x, const void* w_up, const void* w_down, void* gu, void* h, void* y, int64_t T,
                     int64_t d, int64_t F, int act, int dt, void* ws, size_t ws_bytes, void* stream);
int xt_gated_mlp_bwd(const void* x, const void* w_up, const void* w_down, const void* gu, const void* h, const void* dy,
                     void* dgu, void* dx, void* dw_up, void* dw_down, int64_t T, int64_t d, int64_t F, int act, int dt,
                     int dt_grad, int acc_dx, int acc_dw, void* ws, size_t ws_bytes, void* stream);

/* ---------------------------------------------------------------------------------
 * FP8 E4M3 ([BP] § Vad generiska ramverk kostar, item 4: an FP8 E4M3 tensor-core path in the
 * mixed-precision pipeline; the pages give no format details, so the OCP E4M3 format is used:
 * bias 7, 3 mantissa bits, subnormals m·2⁻⁹, largest finite 448, no infinities).
 *   xt_quantize_fp8: per-tensor quantization of n elements of x (XT_F32 / XT_BF16):
 *     scale = 448 / max|x| (one float32 division; 1 when all are 0), out[i] = e4m3(x[i]·scale)
 *     rounded to nearest even and saturated to ±448; *dequant (device float) = max|x| / 448
 *     (1 when all are 0), the factor a code is multiplied by to stand for x.  The workspace
 *     (xt_quantize_fp8_workspace_size) holds per-block maxima.  Deterministic.
 *   xt_matmul_fp8_fwd: C [M, N] (+)= alpha · (*scale_a) · (*scale_b) · A Bᵀ on the tensor cores
 *     (tcgen05 kind::f8f6f4, float32 accumulation): A [M, K] and B [N, K] e4m3 codes with K
 *     contiguous (rows lda / ldb bytes apart, multiples of 16), C float32 or bf16 (ldc
 *     elements); scale_a / scale_b are device floats (may be NULL: 1), e.g. the dequant factors
 *     of xt_quantize_fp8.  A, B, C 16-byte aligned (else XT_ERR_ALIGNMENT).
 * ------------------------------------------------------------------------------- */
int xt_quantize_fp8_workspace_size(int64_t n, size_t* bytes);
int xt_quantize_fp8(const void* x, int64_t n, int dt, uint8_t* out, float* dequant, void* ws, size_t ws_bytes,
                    void* stream);
int xt_matmul_fp8_fwd(int64_t M, int64_t N, int64_t K, const uint8_t* A, int64_t lda, const uint8_t* B, int64_t ldb,
                      void* C, int64_t ldc, int dt_c, float alpha, const float* scale_a, const float* scale_b,
                      int accumulate, void* stream);

/* ---------------------------------------------------------------------------------
 * Optimizer step after the backward ([BP] § Ackumulation över mikrobatcher: gradients of
 * every microbatch are summed into the buffers, then scaled by 1/n_microbatches before one
 * optimizer step; [BP] § Parningsdisciplinen: gradient clipping as a partial and a final
 * gradient-norm reduction and a gradient scale; [BP] § Optimiser-tillståndet: AdamW with a
 * first moment m and a second moment v per weight).  Over n tensors i, all float32:
 *   s    = grad_scale (e.g. 1 / n_microbatches),  norm = ‖s·g‖₂ over every element of every
 *          tensor,  c = min(1, max_grad_norm / (norm + 1e-6))  (c = 1 when max_grad_norm ≤ 0),
 *   g'   = s·c·g,   m ← β₁ m + (1−β₁) g',   v ← β₂ v + (1−β₂) g'²,
 *   θ    ← θ (1 − lr·λ) − lr · (m / (1−β₁ᵗ)) / (√(v / (1−β₂ᵗ)) + ε)   (t = step ≥ 1).
 * param, m, v are updated in place; grad is read only.  shadow (NULL, or per tensor NULL or
 * a device pointer) receives the updated θ converted to shadow_dtype (XT_BF16 / XT_F32): the
 * working copy a bf16 model computes with while param holds the float32 master weights.
 * param, grad, m, v, shadow and numel are HOST arrays of n entries (device pointers, sizes).
 * norm_out (device float, may be NULL) receives norm.  The workspace
 * (xt_adamw_workspace_size) holds one partial sum per 4096-element tile and is needed when
 * clipping or norm_out is requested.  Deterministic: fixed-order sums, no atomics.
 * ------------------------------------------------------------------------------- */
typedef struct xt_adamw_config {
  float lr, beta1, beta2, eps, weight_decay;
  float max_grad_norm; /* ≤ 0: no clipping */
  float grad_scale;    /* applied to every gradient before the norm (1 / n_microbatches) */
  int32_t step;        /* t ≥ 1, for the bias corrections */
} xt_adamw_config;

int xt_adamw_workspace_size(int n, const int64_t* numel, size_t* bytes);
int xt_adamw_step(const xt_adamw_config* cfg, int n, float* const* param, const float* const* grad, float* const* m,
                  float* const* v, void* const* shadow, int shadow_dtype, const int64_t* numel, float* norm_out,
                  void* ws, size_t ws_bytes, void* stream);

/* The same step with both moments held in 8 bits (2 bytes and 2/64 of state per weight instead of 8).
 * 256 consecutive elements of a tensor share one float32 scale for each moment (xt_adamw8_scales(numel)
 * = ceil(numel / 256) of them per tensor): m = m_scale·c·|c| with c the int8 code, √v = r_scale·c² with c
 * the uint8 code.  A step decodes m and v, forms
 *   g' = f·g,  m' = β₁ m + (1−β₁) g',  v' = β₂ v + ((1−β₂) g')·g',
 * each operation rounded to float32 by itself (f: grad_scale·c of xt_adamw_step, c from the norm taken in
 * 64-bit accuracy), updates θ from m' and v' as xt_adamw_step does, and codes them again:
 *   m_scale = max|m'|/127², c = sign(m')·rint(√(|m'|/m_scale)), r_scale = √(max v')/255²,
 *   c = rint(√(√v'/r_scale)), but at least 1 where v' > 0,
 * so the codes are defined to the last bit.  State of zeros (codes and scales) is the state before the first
 * step.  A gradient that is not finite, or whose square is not (|g'| above 1.8e19/√(1−β₂)), leaves its block of 256 with
 * scales that decode to NaN (θ of the element is NaN at once, of the block by the next step).
 * Arguments as for xt_adamw_step, with m_code, r_code, m_scale and r_scale HOST arrays of device pointers.
 * The workspace (xt_adamw8_workspace_size, 8-byte aligned) is needed when clipping or norm_out is
 * requested; its contents on entry do not matter.  Deterministic.
 * xt_adamw8_decode writes the float32 moments that the codes stand for (m, v: HOST arrays whose entries,
 * or which themselves, may be NULL). */
int xt_adamw8_scales(int64_t numel, int64_t* count);
int xt_adamw8_workspace_size(int n, const int64_t* numel, size_t* bytes);
int xt_adamw8_step(const xt_adamw_config* cfg, int n, float* const* param, const float* const* grad,
                   int8_t* const* m_code, uint8_t* const* r_code, float* const* m_scale, float* const* r_scale,
                   void* const* shadow, int shadow_dtype, const int64_t* numel, float* norm_out, void* ws,
                   size_t ws_bytes, void* stream);
int xt_adamw8_decode(int n, const int8_t* const* m_code, const uint8_t* const* r_code, const float* const* m_scale,
                     const float* const* r_scale, float* const* m, float* const* v, const int64_t* numel,
                     void* stream);

/* The Muon step over n matrices W [rows[i], cols[i]] (float32 master weights), in place of AdamW for a model's hidden
 * matrices; two-dimensional parameters such as embeddings, and vectors, stay with xt_adamw_step:
 *   M ← μ M + s·G,   U = s·G + μ M (nesterov = 1; else U = M),   X = U / (‖U‖_F + ε),
 *   steps times  X ← a X + (b A + c A²) X with A = X Xᵀ (Xᵀ X from the right where rows > cols),
 *     a, b, c = 3.4445, −4.7750, 2.0315 (singular values go to about 1: 0.68 .. 1.21),
 *   W ← W (1 − lr·λ) − lr·rms·√max(rows, cols)·X      (rms: the update's root mean square is about rms·lr).
 * s = grad_scale, μ = momentum, λ = weight_decay.  momentum buffers M (float32) start at 0 and are updated in place with
 * W; grad is read only; shadow as for xt_adamw_step.  Products are taken on f16 tensor cores from operands in two terms
 * (22 bits) with float32 sums that they cut off instead of rounding: X is good to a few 1e-6 in norm, two to five times
 * the error of float32 products, growing with the sides.  A matrix is orthogonalised as it is given: projections that are
 * stored side by side in one ([Wq | Wk | Wv]) are taken as one matrix, in the polynomial and in √max(rows, cols).
 * Gradients may be of any finite size (as long as M and U are finite too).  A gradient of 0 with a momentum of 0 leaves
 * X = 0; one that is not finite makes its own matrix NaN.  param, grad, momentum, shadow, rows and cols are HOST arrays;
 * buffers are contiguous, of any alignment of float32 (multiples of 8 columns in 16-byte aligned buffers run on 16-byte
 * accesses), and must not overlap.  At most 64 different shapes; matrices of one shape run as a batch.  Workspace: xt_muon_workspace_size
 * bytes, 16-byte aligned, contents on entry do not matter; about 8 bytes per weight and 8·min(rows, cols)² per matrix.
 * Deterministic.  Device-side waits are bounded (XT_DEVERR_TIMEOUT). */
typedef struct xt_muon_config {
  float lr, momentum, weight_decay;
  float rms;        /* e.g. 0.2 */
  float eps;        /* e.g. 1e-7 */
  float grad_scale; /* applied to every gradient (1 / n_microbatches) */
  int32_t nesterov; /* 0 or 1 */
  int32_t steps;    /* 1 .. 20; usually 5 */
} xt_muon_config;

int xt_muon_workspace_size(int n, const int64_t* rows, const int64_t* cols, size_t* bytes);
int xt_muon_step(const xt_muon_config* cfg, int n, float* const* param, const float* const* grad, float* const* momentum,
                 void* const* shadow, int shadow_dtype, const int64_t* rows, const int64_t* cols, void* ws,
                 size_t ws_bytes, void* stream);

/* ---------------------------------------------------------------------------------
 * Native block stack ([BP] § Framåtgåendet; [DO] § dropout 接在哪（wiring）):
 *   h = E[ids] (+ P);  per layer l:  h += dropout(attn(norm1 h), seed ⊕ l ⊕ 0xA77),
 *                                    h += dropout(mlp(norm2 h),  seed ⊕ l ⊕ 0xF70);
 *   logits = norm_f(h) @ Eᵀ;  loss = cross_entropy(logits, targets).
 * attn: q,k,v = x@W_qkv (W_qkv = [W_Q | W_K | W_V], [d, 3d]); optional RoPE on q, k;
 * per (b, head) P = softmax_causal(q kᵀ/√hd), o = P v; attn = o @ W_O.
 * mlp: SWIGLU: (silu(x@W_g) ∘ x@W_u) @ W_d with W_gu = [W_g | W_u] ([d, 2F]);
 *      GELU:   gelu(x@W_1) @ W_2.
 * xt_block_fwd runs the forward and keeps the saved tensors in ws; xt_block_bwd then adds
 * every parameter gradient into the grad buffers (+=, [BP] § Ackumulation över mikrobatcher);
 * call xt_block_zero_grads first for a fresh step.  No host synchronisation; the pair can
 * be captured in a CUDA graph.  xt_block_bwd runs the weight-gradient GEMMs on a second
 * stream of the device (created by the first xt_block_workspace_size call, never destroyed),
 * forked from and joined back into `stream` with events, so the work it enqueues is complete
 * when `stream` reaches its end; calls on one device must not be issued concurrently from
 * several host threads (they share that stream's events).  With recompute = 1 everything
 * stays on `stream`.
 * ------------------------------------------------------------------------------- */
enum { XT_MLP_SWIGLU = 0, XT_MLP_GELU = 1 };
/* Attention path: AUTO runs the fused kernels (xt_attention_*) when dtype is XT_BF16, hd is
 * 64 and d is a multiple of 8, else the composition of causal-tile GEMMs around the row
 * softmax (which also saves P [B, H, S, S]); COMPOSED forces the latter; FUSED requires the
 * former (XT_ERR_UNSUPPORTED otherwise). */
enum { XT_ATTN_AUTO = 0, XT_ATTN_COMPOSED = 1, XT_ATTN_FUSED = 2 };

typedef struct xt_block_config {
  int32_t B, S, d, H, hd, F, V, n_layers;
  int32_t norm;       /* XT_NORM_RMS or XT_NORM_LN */
  int32_t mlp;        /* XT_MLP_SWIGLU or XT_MLP_GELU */
  int32_t rope;       /* 1: rotate q and k */
  int32_t learned_pos;/* 1: P [S, d] added to the embedding */
  int32_t causal;     /* must be 1 */
  int32_t training;   /* 0: dropout is the identity */
  int32_t dtype;      /* activation and weight storage: XT_F32 or XT_BF16 */
  int32_t grad_dtype; /* parameter-gradient storage: XT_F32 or XT_BF16 */
  float eps;
  float p;            /* residual dropout probability */
  double rope_base;
  uint64_t base_seed;
  int32_t attention;  /* XT_ATTN_AUTO, XT_ATTN_COMPOSED or XT_ATTN_FUSED */
  int32_t recompute;  /* 1: activation recompute — the workspace keeps each layer's input only
                         and the backward recomputes the layer's forward (norm, projections,
                         attention, activation) from it before its backward; the recomputed
                         values are the forward's bit for bit (same kernels, same inputs,
                         counter-based dropout), so are the gradients; 0: keep everything */
} xt_block_config;

/* Per-layer parameter (and gradient) pointers; arrays of n_layers device pointers,
 * held in HOST memory.  Fields unused by the configuration may be NULL. */
typedef struct xt_block_params {
  const void* E;      /* [V, d] */
  const void* P;      /* [S, d] or NULL */
  const void* const* g1; const void* const* b1;
  const void* const* Wqkv; const void* const* Wo;
  const void* const* g2; const void* const* b2;
  const void* const* W_up;   /* [d, 2F] (SWIGLU) or [d, F] (GELU) */
  const void* const* W_down; /* [F, d] */
  const void* gf; const void* bf;
  void* dE; void* dP;
  void* const* dg1; void* const* db1;
  void* const* dWqkv; void* const* dWo;
  void* const* dg2; void* const* db2;
  void* const* dW_up; void* const* dW_down;
  void* dgf; void* dbf;
} xt_block_params;

/* The workspace holds the saved activations and every scratch buffer of the step; its first
 * 4096 bytes (the matmul scratch's stream-K flag words) must be zero before its first use. */
int xt_block_workspace_size(const xt_block_config* cfg, size_t* bytes);
int xt_block_fwd(const xt_block_config* cfg, const xt_block_params* prm, const int32_t* ids,
                 const int32_t* targets, float* loss, void* ws, void* stream);
int xt_block_bwd(const xt_block_config* cfg, const xt_block_params* prm, const int32_t* ids,
                 const int32_t* targets, void* ws, void* stream);
int xt_block_zero_grads(const xt_block_config* cfg, const xt_block_params* prm, void* stream);
/* Process-wide: 1 (default) the backward's weight-gradient GEMMs run on the second stream; 0 all
 * on `stream` (for measurement: a GEMM launch timed beside other kernels includes the time it
 * waits for SMs they hold).  Applies to backward calls enqueued afterwards; XT_ERR_INVALID_ARG
 * for other values. */
int xt_block_set_overlap(int on);

#ifdef __cplusplus
}
#endif
#endif /* XT_H */
