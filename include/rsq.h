/*
 * rsq.h - C ABI of the fused low-bit recurrent-state decode step (gfx950).
 *
 * One decode step of a linear-attention / state-space recurrence whose
 * per-head state S (d_k x d_v) is stored as group-wise low-bit codes:
 *
 *   S_t = A_t S_{t-1} + B_t                       (Table 1 of "Preserving
 *                                                  Updates in Low-Bit Recurrent
 *                                                  State Quantization")
 *     RetNet  A = gamma I            B = k v^T
 *     Mamba2  A = alpha_t I          B = k v^T
 *     GLA     A = Diag(alpha_t)      B = k v^T
 *     GDN     A = alpha_t I          B = beta_t k (v - (A S_{t-1})^T k)^T
 *   o_t = S_t^T q_t    (read before requantization)
 *
 * after which the state is requantized (the abstract of the same page: a
 * recurrent state is requantized after every update) with dynamic,
 * persistent or reference-yoked step sizes (abstract of "When Dynamic
 * Scaling Fails: A Scale-State Feedback Governs Recurrent-State Quantization
 * in Linear-Attention and SSM LLMs"), optional Bounded Directional Rounding
 * and an optional Low-Rank Bypass merged every m steps ("Preserving Updates
 * ...", abstract, Fig. 3, Fig. 4, Table 6).
 *
 * Conventions for every call
 *  - Plain C, no exceptions cross the ABI. Every call returns rsq_status
 *    (RSQ_OK = 0, errors < 0) except rsq_last_error / rsq_abi_version.
 *  - "device" pointers are HIP device memory of the current device; "host"
 *    pointers are ordinary host memory. The caller owns all memory; the
 *    library allocates only the small host handle rsq_state.
 *  - `stream` is a hipStream_t (NULL = the default stream). Every call is
 *    stream-ordered and asynchronous except rsq_get_status and
 *    rsq_state_alloc(RSQ_ATTACH), which synchronize the stream.
 *  - Argument errors are detected on the host before anything is launched;
 *    the call then returns RSQ_E_* and rsq_last_error() describes it.
 *  - Calls on one state must not overlap in time on different streams.
 */
#ifndef RSQ_H
#define RSQ_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define RSQ_ABI_VERSION 3

typedef int32_t rsq_status;
enum {
  RSQ_OK = 0,
  RSQ_E_INVALID = -1,      /* bad argument or configuration */
  RSQ_E_UNSUPPORTED = -2,  /* valid, but a shape/feature this build does not run */
  RSQ_E_BUFFER = -3,       /* device buffer too small */
  RSQ_E_BYPASS_FULL = -4,  /* decode step with k+m bypass columns in use: merge first */
  RSQ_E_NO_BYPASS = -5,    /* merge on a state without a bypass */
  RSQ_E_HIP = -6,          /* a HIP runtime call failed */
  RSQ_E_ATTACH = -7        /* RSQ_ATTACH found a header that does not match the config */
};

/* Table 1 rows. */
enum { RSQ_RETNET = 0, RSQ_MAMBA2 = 1, RSQ_GLA = 2, RSQ_GDN = 3 };
/* Scale policies (abstract of "When Dynamic Scaling Fails ..."). */
enum { RSQ_SCALE_DYNAMIC = 0, RSQ_SCALE_PERSISTENT = 1, RSQ_SCALE_YOKED = 2 };
/* Element types. INT8 and E4M3 (OCP, saturating) are 8-bit codes with scales. */
enum { RSQ_F32 = 0, RSQ_F16 = 1, RSQ_BF16 = 2, RSQ_INT8 = 3, RSQ_E4M3 = 4 };
/* Activations: of rsq_causal_conv the first two, of rsq_block_norm's gate any. */
enum { RSQ_ACT_NONE = 0, RSQ_ACT_SILU = 1, RSQ_ACT_SIGMOID = 2 };
/* rsq_state_alloc modes. */
enum { RSQ_INIT_ZERO = 0, RSQ_ATTACH = 1 };
/* Device status bits (rsq_get_status). */
enum {
  RSQ_F_NONFINITE = 1,       /* a non-finite value reached the state or the output */
  RSQ_F_SCALE_OVERFLOW = 2,  /* a step size overflowed binary16 */
  RSQ_F_CLIPPED = 4          /* a code was clamped to the code range */
};

/*
 * Configuration. All fields are read at rsq_state_alloc and copied.
 *
 *  abi_version     must be RSQ_ABI_VERSION
 *  model           RSQ_RETNET | RSQ_MAMBA2 | RSQ_GLA | RSQ_GDN
 *  batch, heads    tiles are (b, h) pairs, b-major; inputs are [batch][heads][.]
 *  d_k, d_v        per-head state is d_k x d_v (rows = key channels)
 *  group           scale group size along d_v: 8, 16, 32, 64 or 128, dividing d_v
 *  bits            4, 6, 8, or 32 (32 = unquantized fp32 state, the comparator
 *                  of "FP32 states"); ignored when head_bits != NULL
 *  head_bits       NULL, or host array [heads] of per-head widths in {4, 6, 8}
 *  scale_mode      RSQ_SCALE_DYNAMIC | RSQ_SCALE_PERSISTENT | RSQ_SCALE_YOKED
 *  scale_dtype     RSQ_F32 | RSQ_F16 (storage of the per-group step size)
 *  persist_trigger persistent step grows when absmax > trigger * qmax * s (> 0)
 *  bdr, bdr_eps    Bounded Directional Rounding on/off; a reversed element moves
 *                  one code toward its update when the new error stays within
 *                  (0.5 + bdr_eps) * s (bdr_eps >= 0.5 corrects every reversal
 *                  whose corrected code is inside the code range)
 *  lrb_k, lrb_m    Low-Rank Bypass: k residual columns kept by a merge, a merge
 *                  every m steps (capacity k + m fp16 column pairs); m = 0 = off.
 *                  Every update goes into the bypass as one column pair
 *                  (fp16(k), fp16(w)) and the codes only decay between merges.
 *                  With GDN the delta rule reads the stored state plus the
 *                  bypass: u = s_hat^T k + W (U^T k) ("Preserving Updates ...",
 *                  Table 6 GDN row, Tables 7 and 8)
 *  lrb_eps         merge threshold eps_L: |L_ij| > eps_L * s moves into the state
 *  gamma           RetNet only: host array [heads] of decays; NULL otherwise
 *  in_dtype        RSQ_F32 | RSQ_BF16: element type of q, k, v
 *  hadamard        0, or 1 for the INT4+Had baseline of "Preserving Updates",
 *                  Table 2: codes and steps describe each scale group of a
 *                  row rotated by the g x g Sylvester-Hadamard matrix H
 *                  (entries +-1): y = x H is what is quantized, and the state
 *                  reads back as (c s) H / g. Quantized widths with dynamic or
 *                  persistent scales only: no BDR, bypass or yoked scales
 *  pw_window       0, or W in [1, 16]: Gated DeltaNet pure-write window
 *                  ("Low-Bit GDN Recurrent-State Quantization: Global
 *                  Gradient-aware Allocation and Pure-Write Sliding Windows",
 *                  abstract). The state is the low-bit history H plus the last
 *                  W writes as FP8 (OCP E4M3, saturating) pairs (u, w) =
 *                  (k_t, beta_t v_t), slot (t - 1) mod W. Each step the pairs
 *                  that stay take the transition u <- alpha (u - beta k (k^T u)).
 *                  H takes it alone (the delta-rule step with v = 0); the pair
 *                  written W steps earlier takes it too, unrounded, and joins
 *                  H after it, x = H' + u' w^T, before requantization. Then
 *                  o_t = x^T q + sum_c w_c (u_c^T q). Quantized widths with
 *                  dynamic or persistent scales only
 *
 * Supported shapes (others return RSQ_E_UNSUPPORTED): d_v a multiple of
 * 8 * max(4, group / 8); d_k a multiple of 512 / max(4, group / 8) rows per
 * wavefront (128 for group <= 32, 64 for group 64, 32 for group 128) with
 * d_k * d_v <= 32768; GDN needs d_k to be a power of two; yoked scales run
 * without a bypass.
 */
typedef struct rsq_config {
  uint32_t abi_version;
  int32_t model, batch, heads, d_k, d_v;
  int32_t group;
  int32_t bits;
  const int32_t* head_bits;
  int32_t scale_mode, scale_dtype;
  float persist_trigger;
  int32_t bdr;
  float bdr_eps;
  int32_t lrb_k, lrb_m;
  float lrb_eps;
  const float* gamma;
  int32_t in_dtype;
  int32_t hadamard;
  int32_t pw_window;
} rsq_config;

typedef struct rsq_state rsq_state;  /* opaque host handle */

/*
 * Byte layout of a state buffer (all offsets from the buffer start; the
 * buffer must be 256-byte aligned).
 *
 *   [0, 256)            header: u32 magic 'RSQ1', u32 abi version, u64 config
 *                       hash, i64 step count t, i32 bypass fill n; the u32
 *                       device status word sits at byte 128
 *   head_table          heads x 32 bytes {i32 bits, f32 gamma, u64 tile offset
 *                       inside a batch row, u32 scales, bypass_u, bypass_w and
 *                       ref section offsets inside the tile (codes at 0)}
 *   tile (b, h)         at tiles + b * batch_stride + head_offset[h]; inside a
 *                       tile, sections at the offsets below (each 256-aligned):
 *     codes   d_k*d_v*bits/8 bytes in 8x8 chunks. Chunk (rb, cb) (row block
 *             rb = i/8, column block cb = j/8) starts at
 *             (cb * d_k/8 + rb) * 8 * bits bytes. Inside a chunk, row r:
 *               bits 4: u32 word r; byte c (c < 4) holds column c in bits 0-3
 *                       and column c+4 in bits 4-7
 *               bits 8: bytes 8r .. 8r+7 hold columns 0..7
 *               bits 6: code = 4*hi + lo, hi a signed nibble stored like
 *                       bits 4 in the first 32 bytes, lo in [0,3] in the last
 *                       16 bytes: u32 word p holds rows 2p and 2p+1, byte c
 *                       = lo(2p,c) | lo(2p,c+4)<<2 | lo(2p+1,c)<<4 | lo(2p+1,c+4)<<6
 *               bits 32: floats 8r .. 8r+7 hold columns 0..7
 *             4/6/8-bit codes are two's complement, in [-2^(b-1), 2^(b-1)-1].
 *     scales  [d_v/group][d_k] step sizes (scale_dtype); value = code * step
 *     bypass_u [k+m][d_k] fp16 (column c contiguous), bypass_w [k+m][d_v] fp16;
 *             with a pure-write window the same sections hold u [W][d_k] and
 *             w [W][d_v] as E4M3 bytes
 *     ref     yoked reference state, fp32, chunk layout as bits 32
 */
typedef struct rsq_layout {
  size_t header;        /* 0 */
  size_t status;        /* byte offset of the u32 status word */
  size_t head_table;
  size_t tiles;         /* start of tile (0, 0) */
  size_t batch_stride;  /* bytes between tiles (b, h) and (b+1, h) */
  size_t tile_codes;    /* section offsets inside a tile of head h are given by */
  size_t tile_scales;   /*   rsq_tile_sections(); these fields hold head 0's */
  size_t tile_bypass_u;
  size_t tile_bypass_w;
  size_t tile_ref;
  size_t total;         /* == rsq_state_bytes */
} rsq_layout;

/* Bytes the caller must allocate for cfg. */
rsq_status rsq_state_bytes(const rsq_config* cfg, size_t* bytes);

/*
 * Bind a caller-owned device buffer (>= rsq_state_bytes, 256-byte aligned) to
 * a new handle. RSQ_INIT_ZERO clears the buffer (codes 0, steps 0, empty
 * bypass, zero reference: the initial state) and writes the header, stream-
 * ordered. RSQ_ATTACH keeps the contents (a saved state) after checking the
 * header's magic, version and config hash, and restores t and n from it; it
 * synchronizes `stream`. The buffer must stay alive until rsq_state_free.
 */
rsq_status rsq_state_alloc(const rsq_config* cfg, void* dev_buf, size_t buf_bytes,
                           int32_t init, void* stream, rsq_state** out);

/* Free the host handle (not the device buffer). NULL is accepted. */
rsq_status rsq_state_free(rsq_state* st);

/* Layout of the bound buffer (host struct, filled by the call). */
rsq_status rsq_state_layout(const rsq_state* st, rsq_layout* out);

/* Section offsets of a tile of head h, relative to the tile start, and the
 * tile's offset inside a batch row. Any pointer may be NULL. */
rsq_status rsq_tile_sections(const rsq_state* st, int32_t head, size_t* head_offset,
                             size_t* codes, size_t* scales, size_t* bypass_u,
                             size_t* bypass_w, size_t* ref, int32_t* bits);

/* Host-side step count t and bypass fill n of the handle. */
rsq_status rsq_state_counters(const rsq_state* st, int64_t* t, int32_t* n);

/*
 * One decode step of every tile, in place.
 *   q, k  device [batch][heads][d_k] of in_dtype;  v device [batch][heads][d_v]
 *   alpha device fp32: NULL for RetNet; [batch][heads] for Mamba2 and GDN;
 *         [batch][heads][d_k] for GLA (per key channel)
 *   beta  device fp32 [batch][heads], GDN only (NULL otherwise)
 *   o     device fp32 [batch][heads][d_v], written: o_t = S_t^T q_t from the
 *         updated state before requantization (plus W (U^T q) with a bypass)
 * Inputs must be contiguous and 16-byte aligned. With a bypass, returns
 * RSQ_E_BYPASS_FULL once k+m columns are in use (call rsq_merge_bypass).
 * Steps of states without a bypass or window can be captured in a HIP graph
 * and replayed; with a bypass or a pure-write window the step's column or
 * slot comes from the host handle, so such a step (and rsq_merge_bypass)
 * returns RSQ_E_UNSUPPORTED while `stream` is capturing.
 */
rsq_status rsq_decode_step(rsq_state* st, const void* q, const void* k, const void* v,
                           const float* alpha, const float* beta, float* o, void* stream);

/*
 * rsq_decode_step for profiling: the step's decode kernel records
 * start_event (a hipEvent_t, may be NULL) when it begins and stop_event when
 * it ends. The timestamps come from the kernel's own dispatch, so no extra
 * command enters the stream and back-to-back steps stay back to back. The
 * events belong to the caller and must exist on the stream's device.
 */
rsq_status rsq_decode_step_timed(rsq_state* st, const void* q, const void* k, const void* v,
                                 const float* alpha, const float* beta, float* o, void* stream,
                                 void* start_event, void* stop_event);

/*
 * rsq_decode_step with error accounting ("Preserving Updates ...", Fig. 1:
 * per-step rounding errors R and their decayed sum E_T; Fig. 2: the coherent
 * gain g_T and its parts on lost and moved updates; Fig. 4: lost, moved and
 * reversed updates; Table 5: |b| / step and the lost fraction). The state
 * advances exactly as rsq_decode_step would (same codes, steps and o). Per
 * element of each tile, with b = fl(k_i w_j) the element's update B_t,
 * s' the step after the scale rule, x the value before rounding, r the
 * no-update value fl(c fl(a s)) and c the stored code:
 *   R = fl(c s' - x); lost: b != 0 and c equals the code r rounds to on the
 *   same grid; moved: b != 0 and not lost; reversed: b != 0 and c s' lies
 *   strictly on the other side of r from b.
 *   acc    device fp32 [tiles][6][d_k*d_v], each plane in the bits-32 chunk
 *          layout of the codes (tiles b-major): E, D, E_lost, D_lost, E_moved,
 *          D_moved, updated in place with a = the row decay of Table 1:
 *          E <- fl(fl(a E) + R_m), D <- fl(fl(fl(a a) D) + fl(R_m R_m)),
 *          R_m = R on the plane's mask (all, lost, moved), 0 elsewhere.
 *          Zero it to start a window; g_T = sum E^2 / sum D.
 *   ratio  device fp32 [tiles][d_k*d_v] (chunk layout) or NULL: this step's
 *          fl(|b| RN(1/s')) for updated elements with a finite s' > 0, else -1
 *   counts device u32 [tiles][4]: updated, lost, moved, reversed, added to
 * Buffers are 16-byte aligned and owned by the caller. Returns
 * RSQ_E_UNSUPPORTED for fp32 states, a bypass or yoked scales.
 */
rsq_status rsq_decode_step_diag(rsq_state* st, const void* q, const void* k, const void* v,
                                const float* alpha, const float* beta, float* o, float* acc,
                                float* ratio, uint32_t* counts, void* stream);

/*
 * Low-Rank Bypass merge: L = U W^T; elements with |L_ij| > eps_L * s move
 * into the quantized state, which is requantized (with BDR when enabled,
 * toward sign(L_ij)); the rest is replaced by a rank-k approximation kept as
 * k fp16 column pairs. Sets n = k. RSQ_E_NO_BYPASS without a bypass.
 */
rsq_status rsq_merge_bypass(rsq_state* st, void* stream);

/* rsq_merge_bypass for profiling: the merge kernel's dispatch records
 * start_event / stop_event (hipEvent_t, either may be NULL), as in
 * rsq_decode_step_timed. */
rsq_status rsq_merge_bypass_timed(rsq_state* st, void* stream, void* start_event, void* stop_event);

/* o = deq(S)^T q (+ W (U^T q)); reads the state only. q as in decode_step. */
rsq_status rsq_readout(const rsq_state* st, const void* q, float* o, void* stream);

/* Synchronize `stream`, then return and clear the device status bits. */
rsq_status rsq_get_status(rsq_state* st, uint32_t* flags, void* stream);

/*
 * Decay-aware per-head widths (host only; "Low-Bit Recurrent States in Hybrid
 * Language Models", abstract: Gramian distortion weights and normalised state
 * ranges). Head h at width b costs w_h / (2^(b-1) - 1)^2 with
 * w_h = range[h]^2 / (1 - decay_sq[h]): 1 / (1 - E[a^2]) is how much of an
 * injected error a state decaying by a_t keeps over the future steps. The
 * widths {4, 6, 8} written to bits_out (host array [heads]) minimise the total
 * cost with sum(bits) <= floor(mean_bits * heads); ties go to the lower head
 * index, and a head gains width only where that lowers the cost.
 *   decay_sq  host [heads]: E[a_t^2] of the head's decay, in [0, 1)
 *             (GLA: the mean over key channels of E[a_t,i^2])
 *   range     host [heads]: the head's typical group absmax (>= 0, finite)
 *   mean_bits in [4, 8]
 * Returns RSQ_E_INVALID on a bad argument (bits_out is then unspecified).
 * The result can be passed as rsq_config.head_bits.
 */
rsq_status rsq_allocate_head_bits(const float* decay_sq, const float* range, int32_t heads,
                                  float mean_bits, int32_t* bits_out);

/* ------------------------------------------------------------------------
 * Operators of the layer around the decode step. Activations are fp32 or bf16
 * (`dtype`), parameters fp32; rows are `*_stride` elements apart, with their
 * elements contiguous. Sums, norms and states are fp32. An output that overlaps
 * another argument's memory is refused. Every call can be captured in a graph
 * and replayed.
 *
 * Sequences of a prompt batch are packed: `tokens` rows in all, sequence s at
 * rows offsets[s] .. offsets[s + 1] - 1 (device int32 [seqs + 1]), none longer
 * than max_len. offsets NULL: every sequence has max_len rows, tokens = seqs *
 * max_len. Empty sequences are allowed. Offsets live on the device, so they are
 * not checked on the host: the kernels clamp them into [0, tokens], and of a
 * sequence longer than max_len only its first max_len rows are taken. Rows of y
 * that belong to no sequence are left as they were; what a row of two sequences
 * gets is one of their two results.
 * ------------------------------------------------------------------------ */

/*
 * Short causal convolution of each channel (before a selective scan):
 *   y[t, c] = act(bias[c] + sum_{j < width} weight[c, j] x[t - width + 1 + j, c])
 *   dtype      RSQ_F32 | RSQ_BF16: x, y, state
 *   width      2..4 (others RSQ_E_UNSUPPORTED)
 *   weight     device fp32 [channels][width], the last tap on the current token
 *   bias       device fp32 [channels], or NULL
 *   state      device [seqs][channels][width - 1] of dtype, oldest input first:
 *              the inputs before each sequence, replaced by its last width - 1
 *              inputs (an empty sequence keeps its own); NULL: zeros, none kept
 * One token of every sequence (offsets NULL, max_len 1) is the decode form.
 */
typedef struct rsq_conv {
  int32_t dtype, seqs, channels, width, activation;
  int64_t tokens, max_len;
  const int32_t* offsets;
  const void* x;
  int64_t x_stride;
  const float* weight;
  const float* bias;
  void* state;
  void* y;
  int64_t y_stride;
} rsq_conv;
rsq_status rsq_causal_conv(const rsq_conv* conv, void* stream);

/*
 * Selective state-space recurrence (the Mamba2 row of Table 1 with its gates):
 *   delta = softplus(dt + dt_bias), or dt + dt_bias when softplus is 0
 *   S     = exp(delta A[h]) S + delta B x^T          (S: d_k x d_v, fp32)
 *   y     = S^T C + D[h] x
 * for every head h; heads are split evenly over `groups`, and the heads of a
 * group share B and C.
 *   dtype      RSQ_F32 | RSQ_BF16: x, B, C, dt, y
 *   x, y       device [tokens][heads][d_v];  B, C device [tokens][groups][d_k]
 *   dt         device [tokens][heads]
 *   A          device fp32 [heads] (negative for a decay)
 *   D, dt_bias device fp32 [heads], or NULL
 *   state      device fp32 [seqs][heads][d_k][d_v], replaced by the state after
 *              each sequence. state_in 0: start from zero, the contents are not
 *              read; 1: start from the contents (an empty sequence keeps them)
 *   workspace  rsq_ssm_scan_workspace bytes, 16-byte aligned (scan only; it may
 *              be NULL when that is 0). Its contents need not be kept.
 * x, B, C, y and state are 16-byte aligned, the strides of x, B, C and y
 * multiples of 16 bytes; d_k and d_v are multiples of 8.
 * rsq_ssm_scan takes d_k <= 256 (bf16) or 128 (fp32), d_v <= 4096, max_len
 * below 2^31 - 4096, rows at most 2^24 bytes apart and fewer than 2^24 workgroups
 * (heads * ceil(d_v / 64) for each sequence, and for each segment of long ones;
 * RSQ_E_UNSUPPORTED beyond). bf16: S and the token weights enter y as two bf16
 * pieces each (2^-16 of its terms, before y is rounded to bf16); the state itself
 * is exact to fp32. An infinite or NaN x makes its column NaN from its token on;
 * earlier tokens are not touched.
 * rsq_ssm_step takes one row of every sequence: offsets NULL, max_len 1; d_v <=
 * 1024, d_k <= 4096; seqs * heads below 2^24 (RSQ_E_UNSUPPORTED beyond).
 */
typedef struct rsq_ssm {
  int32_t dtype, seqs, heads, groups, d_k, d_v;
  int32_t softplus, state_in;
  int64_t tokens, max_len;
  const int32_t* offsets;
  const void* x;
  int64_t x_stride;
  const void* B;
  int64_t b_stride;
  const void* C;
  int64_t c_stride;
  const void* dt;
  int64_t dt_stride;
  const float* A;
  const float* D;
  const float* dt_bias;
  float* state;
  void* y;
  int64_t y_stride;
  void* workspace;
  size_t workspace_bytes;
} rsq_ssm;
rsq_status rsq_ssm_scan_workspace(const rsq_ssm* ssm, size_t* bytes);
rsq_status rsq_ssm_scan(const rsq_ssm* ssm, void* stream);
rsq_status rsq_ssm_step(const rsq_ssm* ssm, void* stream);

/*
 * The same single-token step on a quantized state (model RSQ_MAMBA2; dtype,
 * seqs, heads, d_k and d_v as configured; ssm->state NULL): the gates, then
 * rsq_decode_step with q = C, k = B, v = delta x (rounded to dtype) and alpha =
 * exp(delta A), then y = o + D x. The workspace is 256-byte aligned. Capture
 * and a full bypass as in rsq_decode_step.
 */
rsq_status rsq_decode_ssm_workspace(const rsq_state* st, size_t* bytes);
rsq_status rsq_decode_ssm_step(rsq_state* st, const rsq_ssm* ssm, void* stream);

/*
 * Put a dense fp32 state (device [batch][heads][d_k][d_v], 16-byte aligned,
 * such as a scan's) into a state of any model, as its first one: every group's
 * step is absmax / qmax, the codes are rounded to nearest-even, a yoked
 * reference takes the dense values, the bypass or the window is empty and the
 * step count 0. RSQ_E_UNSUPPORTED while `stream` is capturing.
 */
rsq_status rsq_state_load(rsq_state* st, const float* dense, void* stream);

/*
 * Attention with a decay for each head over prompts (RetNet, Mamba2 and, with beta,
 * Gated DeltaNet rows of Table 1), on a dense fp32 state that rsq_state_load takes:
 *   u_t = v_t, or with beta the delta rule u_t = beta_t (v_t - alpha_t S_{t-1}^T k_t)
 *   S_t = alpha_t S_{t-1} + k_t u_t^T          (S: d_k x d_v)
 *   o_t = S_t^T q_t
 * for every head h; heads are split evenly over key_heads, and those of one share
 * its q and k.
 *   dtype      RSQ_F32 | RSQ_BF16: q, k, v, o
 *   q, k       device [tokens][key_heads][d_k];  v, o device [tokens][heads][d_v]
 *   alpha      device fp32 [tokens][heads], not negative; alpha_stride 0: [heads], the
 *              same for all tokens; NULL: 1. An alpha of 0 clears a finite state; a
 *              column that is not finite stays so (0 times an infinity is a NaN): to
 *              drop a state whatever it holds, start from zero with state_in 0
 *   beta       device fp32 [tokens][heads]; NULL: no delta rule
 *   state      device fp32 [seqs][heads][d_k][d_v], replaced by the state after
 *              each sequence. state_in 0: start from zero, the contents are not
 *              read; 1: start from the contents (an empty sequence keeps them)
 *   workspace  rsq_linear_attention_workspace bytes, 16-byte aligned (prompts only;
 *              NULL where that is 0). With beta 400 bytes a token and head, of fp32
 *              inputs 496 and 1536 a token and key head, with tokens counted in
 *              chunks of 64 (none with max_len up to 8). Its contents need not be kept.
 * q, k, v, o and state are 16-byte aligned, the strides of q, k, v and o multiples
 * of 16 bytes; d_k and d_v are multiples of 8, d_v <= 4096.
 * rsq_linear_attention takes d_k <= 256 (bf16) or 128 (fp32), max_len below 2^31 -
 * 4096, rows at most 2^24 bytes apart and fewer than 2^24 workgroups (with beta 2^23;
 * RSQ_E_UNSUPPORTED beyond). With beta, sequences must not share rows: where offsets fall, results are
 * unspecified. bf16: S, u and the token weights enter o as two bf16 pieces each (2^-16
 * of its terms, before o is rounded to bf16); the state itself is exact to fp32. A v
 * that is not finite makes its column NaN from its token on, a k, alpha or beta (with
 * beta given) the whole head; earlier tokens are not touched.
 * A call gives the same bits every time. The last bits of a sequence's o and state may
 * differ with the number of heads and with what else is in the batch, which decide how
 * the work is cut up, and so the order of sums.
 * rsq_linear_attention_step takes one row of every sequence: offsets NULL, max_len
 * 1; d_k <= 256; alpha and beta [seqs][heads].
 */
typedef struct rsq_linear_attn {
  int32_t dtype, seqs, heads, key_heads, d_k, d_v;
  int32_t state_in;
  int64_t tokens, max_len;
  const int32_t* offsets;
  const void* q;
  int64_t q_stride;
  const void* k;
  int64_t k_stride;
  const void* v;
  int64_t v_stride;
  const float* alpha;
  int64_t alpha_stride;
  const float* beta;
  int64_t beta_stride;
  float* state;
  void* o;
  int64_t o_stride;
  void* workspace;
  size_t workspace_bytes;
} rsq_linear_attn;
rsq_status rsq_linear_attention_workspace(const rsq_linear_attn* attn, size_t* bytes);
rsq_status rsq_linear_attention(const rsq_linear_attn* attn, void* stream);
rsq_status rsq_linear_attention_step(const rsq_linear_attn* attn, void* stream);

/*
 * Root-mean-square norm of rows:
 *   h = x + residual (stored back to residual, rounded to dtype; residual NULL: h = x)
 *   y = h / sqrt(mean(h^2) + eps) * weight, of the fp32 h
 *   dtype      RSQ_F32 | RSQ_BF16: x, residual
 *   out_dtype  RSQ_F32 | RSQ_BF16, or RSQ_INT8 | RSQ_E4M3: codes round(y / scale),
 *              nearest-even, with scale = absmax(y) / qmax (127 or 448); a zero
 *              scale stores code 0
 *   group      0: a scale per row; 32, 64 or 128 dividing cols: one per group
 *   scales     device fp32 [rows][cols / group] (group 0: [rows]); NULL without codes
 *   cols       at most 32768
 * The sum of the squares is fp32: a row of magnitudes above 2^63 / sqrt(cols), whose
 * squares overflow, gives zeros.
 */
typedef struct rsq_norm {
  int32_t dtype, out_dtype, cols, group;
  float eps;
  int64_t rows;
  const void* x;
  int64_t x_stride;
  void* residual;
  int64_t residual_stride;
  const float* weight;
  void* y;
  int64_t y_stride;
  float* scales;
} rsq_norm;
rsq_status rsq_rms_norm(const rsq_norm* norm, void* stream);

/*
 * Norms before and after a block, with its gate and residual; of each row
 *   u = x                       (gate_first: x * act(gate))
 *   u = u / sqrt(mean(u^2) + eps) * weight          (weight NULL: u as it is)
 *   u = u * act(gate)           (unless it came first; gate NULL: u as it is)
 *   h = residual + residual_scale * u (stored back to residual, rounded to dtype; NULL: h = u)
 *   y = h / sqrt(mean(h^2) + eps) * next_weight, of the fp32 h (next_weight NULL: y = h)
 *   dtype        RSQ_F32 | RSQ_BF16: x, gate, residual
 *   out_dtype, scale_group, scales  of y, as out_dtype, group and scales of rsq_rms_norm
 *   group        the first mean's columns: 0 (the row), or a multiple of 8 that
 *                divides cols (heads normed one by one)
 *   weight       device fp32 [weight_cols]: cols of them, or one group's for all
 *   activation   RSQ_ACT_NONE | RSQ_ACT_SILU | RSQ_ACT_SIGMOID
 *   residual_scale  finite; 1 without a residual
 *   y            may be NULL where the residual is the result: with a residual,
 *                without next_weight and codes (out_dtype is then not looked at
 *                beyond being a type)
 *   cols         at most 32768
 * The sums of squares are fp32, as in rsq_rms_norm. With a residual and next_weight
 * alone it is rsq_rms_norm's operation; of its own are the first norm, groups, gate and
 * residual_scale. Of 8193 to 16384 columns the last bits may differ with the rows.
 */
typedef struct rsq_block {
  int32_t dtype, out_dtype, cols, group, weight_cols, scale_group, activation, gate_first;
  float eps, residual_scale;
  int64_t rows;
  const void* x;
  int64_t x_stride;
  const void* gate;
  int64_t gate_stride;
  void* residual;
  int64_t residual_stride;
  const float* weight;
  const float* next_weight;
  void* y;
  int64_t y_stride;
  float* scales;
} rsq_block;
rsq_status rsq_block_norm(const rsq_block* block, void* stream);

/*
 * Products with 4-bit weights: y[m, n] = sum_j x[m, j] codes[n, j] scales[n, j / group].
 *   group        32, 64 or 128, dividing k
 *   codes        device int8 [n][k], values -8..7 (their low four bits are taken)
 *   scales       device [n][k / group] of scale_dtype (RSQ_F32 | RSQ_F16)
 * rsq_w4_pack lays both out once into `packed` (rsq_w4_bytes bytes, 16-byte
 * aligned): 16 rows x 128 columns in 1 KB, rows and columns padded with zeros,
 * then the scales [k / group][n].
 *   x_dtype      RSQ_F32 | RSQ_BF16, or RSQ_INT8 | RSQ_E4M3 with x_scale
 *   x_scale      device fp32 [m] (x_group 0) or [m][k / group] (x_group = group);
 *                NULL without 8-bit x
 *   out_dtype    RSQ_F32 | RSQ_BF16
 * Sums are fp32 (int8: int32 inside a group). Meant for few rows: every 16 or 32
 * rows of x read the weights once. fp32 and bf16 x may reach 2^100 (beyond, the
 * offset that codes carry inside may overflow). n up to 2^26, k to 2^22, below
 * 2^34 weights (with the padding), rows of x at most 2^24 bytes apart
 * (RSQ_E_UNSUPPORTED beyond).
 */
rsq_status rsq_w4_bytes(int32_t n, int32_t k, int32_t group, int32_t scale_dtype, size_t* bytes);
rsq_status rsq_w4_pack(const int8_t* codes, const void* scales, int32_t n, int32_t k, int32_t group,
                       int32_t scale_dtype, void* packed, size_t packed_bytes, void* stream);
typedef struct rsq_w4 {
  int32_t x_dtype, out_dtype, m, n, k, group, scale_dtype, x_group;
  const void* x;
  int64_t x_stride;
  const float* x_scale;
  const void* packed;
  size_t packed_bytes;
  void* y;
  int64_t y_stride;
} rsq_w4;
rsq_status rsq_w4_linear(const rsq_w4* w4, void* stream);

/*
 * Products of 8-bit integers with a scale for each token and each channel, for the
 * projections of prompts:
 *   y[m, n] = x_scale[m] scales[n] sum_j x[m, j] codes[n, j] (+ bias[n])
 *   codes        device int8 [n][k], scales device fp32 [n]
 * rsq_w8_pack lays both out once into `packed` (rsq_w8_bytes bytes, 16-byte
 * aligned): 16 rows x 64 columns in 1 KB, rows and columns padded with zeros, then
 * the scales.
 *   x            device int8 [m][k], rows x_stride bytes apart
 *   x_scale      device fp32 [m], as rsq_rms_norm and rsq_block_norm give them
 *   bias         device fp32 [n], or NULL
 *   out_dtype    RSQ_F32 | RSQ_BF16
 *   workspace    rsq_w8_workspace bytes, 16-byte aligned (rows of x that do not begin
 *                at multiples of 16 bytes are laid out again where there are many of
 *                them; NULL where that is 0). Its contents need not be kept.
 * Sums are exact (int32: k below 2^17), then rounded to fp32 before the scales. n up
 * to 2^26 (RSQ_E_UNSUPPORTED beyond).
 */
rsq_status rsq_w8_bytes(int32_t n, int32_t k, size_t* bytes);
rsq_status rsq_w8_pack(const int8_t* codes, const float* scales, int32_t n, int32_t k, void* packed,
                       size_t packed_bytes, void* stream);
typedef struct rsq_w8 {
  int32_t out_dtype, m, n, k;
  const int8_t* x;
  int64_t x_stride;
  const float* x_scale;
  const float* bias;
  const void* packed;
  size_t packed_bytes;
  void* y;
  int64_t y_stride;
  void* workspace;
  size_t workspace_bytes;
} rsq_w8;
rsq_status rsq_w8_workspace(const rsq_w8* w8, size_t* bytes);
rsq_status rsq_w8_linear(const rsq_w8* w8, void* stream);

/* Thread-local description of the last error (never NULL). */
const char* rsq_last_error(void);

int32_t rsq_abi_version(void);

#ifdef __cplusplus
}
#endif
#endif /* RSQ_H */
