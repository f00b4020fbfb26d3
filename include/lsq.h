/*
 * lsq — decode step of a linear recurrence whose matrix state is stored at low
 * bit-width, for AMD Instinct MI355X (gfx950).  C ABI.
 *
 * The operation (one decode step, for every batch*head independently):
 *
 *   S_t = S_{t-1} Lambda_t (I - delta beta_t k_t k_t^T) + beta_t v_t k_t^T
 *
 * is Eq. (1) of "LinQuant: Functional Invariances for Low-Precision Linear
 * Recurrences" (summary page, Theoretical Foundation), with scalar decay
 * Lambda_t = alpha_t I or diagonal decay diag(alpha_t), write gate beta_t > 0
 * and delta in {0,1} (Key structural choices).  S_t is Dv x Dk.  The step
 * emits o_t = S_t q_t, then requantises the state, as "When Dynamic Scaling
 * Fails" (abstract) describes: the state is rewritten and requantised at every
 * decode step with uniform group-wise INT4/INT8, the group scale being
 *   DYNAMIC    read from the new state itself (per-token absmax; project page,
 *              mechanism paragraph),
 *   PERSISTENT frozen once by calibration (the abstract's persistent arm),
 *   YOKED      read from an fp32 reference state advanced alongside (the
 *              project page's control arm: the same quantiser, with the scale
 *              no longer fed back from the quantised state),
 * and rounded either to nearest-even or by Bounded Directional Rounding
 * ("Preserving Updates in Low-Bit Recurrent State Quantization", abstract): an
 * element whose rounded value moved opposite to its update is rounded one
 * grid step toward the update, or with a deterministic golden-ratio Weyl
 * dither ("Low-Discrepancy Dither for Quantized Recurrent State Caches",
 * listing entry; the sequence below is this library's reading of it).
 *
 * Arithmetic contract (every step below is what the kernels compute):
 *   m_c   = fl(s_group(c) * alpha_c)            alpha_c = alpha for scalar decay
 *   S'_c  = fl(C_c * m_c)                       dequantise with the decay folded in
 *   u     = dot(S', k)                          only when delta = 1, else 0
 *   w     = fl(beta * fl(v_r - u))
 *   S_c   = fma(w, k_c, S'_c)
 *   o_r   = dot(S, q)                           read before requantisation
 *   s_new = DYNAMIC: fl(max|S_c| / qmax) per group; PERSISTENT: s;
 *           YOKED: fl(max|R_c| / qmax) with R advanced by the same update in fp32
 *   inv   = s_new == 0 ? 0 : fl(1 / s_new)
 *   c1    = clamp(round-half-even(S_c * inv exactly), -qmax, qmax)
 *   BDR:    sigma_c = sign(w) sign(k_c); if (c1 - S'_c * inv) * sigma_c < 0
 *           (exact), then c = clamp(c1 + sigma_c), else c = c1
 *   DITHER: c = clamp(floor(S_c * inv + u_i) exactly, -qmax, qmax) in place of
 *           c1, u_i = ((i * 0x9E3779B9) mod 2^32 >> 9) * 2^-23 (the Weyl
 *           sequence frac(i (sqrt(5)-1)/2) in fixed point, 23 bits), i =
 *           (t Dv Dk + r Dk + c) mod 2^32 with t the handle's step index
 *   BDR_A, BDR_B (sensitivity flags; frozen scale s, stored code C_old): the
 *           readings of "update" and "move" not taken by BDR.  A: sigma_c =
 *           sign(S_c - C_old s) (exact); B': sigma_c = sign(w) sign(k_c).  If
 *           (c1 - C_old) * sigma_c < 0 and s > 0 then c = c1 + sigma_c, else c1.
 *           On a frozen grid A never fires (it equals RNE).
 * with qmax = 2^(bits-1) - 1 (7 for INT4, 127 for INT8).  dot(a, b) is an
 * fp32 sum in one fixed order (the pages leave the order open; fixing it makes
 * every code, scale and output reproducible bit for bit): the columns are
 * taken in consecutive blocks of 32, inside a block the products accumulate by
 * a chain of fused multiply-adds from zero in column order, and the block sums
 * are added in adjacent pairs, level by level ((b0 + b1) + (b2 + b3) at Dk =
 * 128).  The unquantised mode (bits 32) keeps the same formulas with its own
 * summation order.
 *
 * Memory: every pointer below is a DEVICE pointer (row-major, 16-byte
 * aligned) unless stated.  The library never allocates device memory: the
 * caller allocates the state buffers (lsq_state_sizes gives their sizes) and
 * the inputs/outputs, and binds them to a handle.  The handle itself is a
 * small host object.
 *
 * Packed state layout (per handle, heads = batch*heads):
 *   codes  [heads][Dv][Dk*bits/8] bytes.  INT8: one two's-complement byte per
 *          element.  INT4: element c of a row in byte c/2, low nibble for even
 *          c, two's-complement nibble.  Codes lie in [-qmax, qmax]; the
 *          most negative code (-8, -128) is never produced and is not a
 *          valid input.
 *   scales [heads][Dv][Dk/group], one per contiguous group along Dk: fp32,
 *          or (scale_fmt) IEEE binary16 or bfloat16 bit patterns, 2 bytes;
 *          group = 0: [heads] fp32, one per head.
 *   ref    [heads][Dv][Dk] fp32, the yoked policy's reference state.
 *   f32    [heads][Dv][Dk] fp32, the state of the unquantised mode (bits 32).
 *   lrb    Low-Rank Bypass buffer (lrb_rank = r > 0), fp32: a [heads][r][Dv]
 *          followed by b [heads][2][r][Dk] (copy 1 used by diagonal decay).
 *
 * Low-Rank Bypass ("Preserving Updates in Low-Bit Recurrent State
 * Quantization", abstract: small updates collect in a low-rank buffer, and
 * the parts of it that have grown large enough enter the state from time to
 * time; rank, period and threshold are not given there).  This
 * library's reading: slot j holds a_j [Dv], b_j [Dk], B = sum_j a_j b_j^T;
 * at step t, n = t mod r slots are filled (the handle's step index t).  The
 * buffer decays with the state (scalar decay: a_j = fl(alpha a_j); diagonal:
 * b_j = fl(b_j alpha)); u and o are taken from S' + B (o also includes the
 * new write); the write fills slot n (a_n = w, b_n = k) instead of entering
 * the quantised state, which is requantised from S' alone; when n = r-1 the
 * step merges instead: X = S' then X = fma(a_j, b_j, X) for j = 0..n in slot
 * order, the scale policy and rounding applied to X (BDR's update sign is the
 * sign of U built the same way from 0), and the buffer empties.  b is read from
 * copy t mod 2 and written to copy (t+1) mod 2 under diagonal decay (copy 0
 * only under scalar decay).  Supported: bits 4/8, DYNAMIC or PERSISTENT,
 * groups of 32 or more, r <= 8; the buffer starts as lsq_state_zero leaves it.
 * Inputs per step: q, k [heads][Dk]; v [heads][Dv]; alpha [heads] (scalar
 * decay) or [heads][Dk] (diagonal); beta [heads].  Output o [heads][Dv];
 * o_ref [heads][Dv] (yoked only, nullable).
 *
 * Errors and streams: calls are asynchronous on the given HIP stream (a
 * hipStream_t passed as void*, NULL for the default stream).  Argument checks
 * happen on the host before any launch and return a status without touching
 * the device.  Launch failures return LSQ_ERR_HIP.  No C++ exception crosses
 * the ABI.  A handle must not be used on two streams at once.  Inputs must be
 * finite and the state far from overflow (scales and |S| below 2^100); a
 * nonzero scale must be a normal float (>= 2^-126), since fl(1/s) overflows
 * below 2^-128 and 0 * inf has no code; the data is not scanned.  With batch*heads == 0 every call is a no-op and its
 * data pointers may be NULL.
 */
#ifndef LSQ_H
#define LSQ_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  LSQ_OK = 0,
  LSQ_ERR_INVALID_ARG = 1,     /* null pointer, bad value, misaligned buffer */
  LSQ_ERR_UNSUPPORTED = 2,     /* a valid configuration this library has no kernel for */
  LSQ_ERR_BUFFER_TOO_SMALL = 3,
  LSQ_ERR_NOT_CALIBRATED = 4,  /* persistent policy stepped before its scales were frozen */
  LSQ_ERR_HIP = 5              /* a HIP runtime call or kernel launch failed */
} lsq_status;

typedef enum {
  LSQ_POLICY_NONE = 0,        /* bits == 32: unquantised fp32 state */
  LSQ_POLICY_DYNAMIC = 1,
  LSQ_POLICY_PERSISTENT = 2,
  LSQ_POLICY_YOKED = 3
} lsq_policy;

/* BDR_A and BDR_B are the two readings of directional rounding this library
 * does not take, for sensitivity runs (persistent scale only, groups of 32 or
 * more, fp32 scales, no bypass; see the rounding contract above). */
typedef enum {
  LSQ_ROUND_RNE = 0,
  LSQ_ROUND_BDR = 1,
  LSQ_ROUND_DITHER = 2,
  LSQ_ROUND_BDR_A = 3,
  LSQ_ROUND_BDR_B = 4
} lsq_rounding;
typedef enum { LSQ_DECAY_SCALAR = 0, LSQ_DECAY_DIAG = 1 } lsq_decay;
typedef enum { LSQ_SCALE_F32 = 0, LSQ_SCALE_F16 = 1, LSQ_SCALE_BF16 = 2 } lsq_scale_format;

/* Shape, format and method flags of one handle.
 *   bits   4, 8 (quantised) or 32 (fp32 state, policy NONE)
 *   group  group size along Dk; must divide dk.  This library supports
 *          power-of-two groups of 16 to Dk elements (one lane owns 32
 *          consecutive elements of a row: one group, part of one, or two
 *          16-element groups) and Dk in {64, 128}.  group = Dk is one scale
 *          per row.  group = 0 is one scale per head for the whole Dv x Dk
 *          state (scales [heads] fp32): DYNAMIC (the absmax over every
 *          element after the step's update, so all rows are updated before
 *          any is requantised) or PERSISTENT (calibrated over the head), RNE
 *          or BDR, fp32 scale, no bypass, Dv <= 1024.  INT4 with 16-element
 *          groups and fp32 scales stores 6 bits per element, 5.33x less
 *          than an fp32 state.
 *   delta  0: linear write, 1: delta-rule correction
 *   scale_fmt  stored format of the group scales (the pages fix none; 16-bit
 *          scales are the scale-format variant of "Preserving Updates in
 *          Low-Bit Recurrent State Quantization", whose memory saving of at
 *          most 5.3x leaves the format open).  A computed scale (dynamic, yoked,
 *          calibration) is rounded to the format, to nearest with ties to
 *          even (binary16 with subnormals, overflow to infinity; bfloat16 on
 *          the upper half of the fp32 pattern), and the codes are formed with
 *          that stored value: inv = fl(1/s_stored); elements beyond qmax
 *          steps of a scale that rounded down clamp.  Quantised states only;
 *          not with the bypass.  INT4 g32 with bfloat16
 *          scales stores 4.5 bits per element (7.1x less than fp32), INT4
 *          g16 5 bits (6.4x).
 */
typedef struct {
  int32_t batch, heads, dk, dv;
  int32_t bits, group, policy, rounding, delta, decay;
  int32_t lrb_rank;   /* Low-Rank Bypass slots r, 0 (off) to 8; see below */
  int32_t scale_fmt;  /* lsq_scale_format (LSQ_SCALE_F32 = 0) */
} lsq_config;

/* Caller-owned device buffers and their capacities in bytes.  Buffers the
 * configuration does not use may be NULL with capacity 0. */
typedef struct {
  void* codes;   size_t codes_bytes;
  float* scales; size_t scales_bytes;
  float* ref;    size_t ref_bytes;
  float* f32;    size_t f32_bytes;
  float* lrb;    size_t lrb_bytes;    /* Low-Rank Bypass buffer (lrb_rank > 0) */
} lsq_buffers;

typedef struct lsq_state lsq_state;

/* Byte sizes of the state buffers a configuration needs (0 when unused).
 * Host only.  Any output pointer may be NULL. */
lsq_status lsq_state_sizes(const lsq_config* cfg, size_t* codes_bytes, size_t* scales_bytes,
                           size_t* ref_bytes, size_t* f32_bytes, size_t* lrb_bytes);

/* Create a handle that binds the caller's buffers.  Allocates only the host
 * handle.  Checks: valid config, non-null and 16-byte aligned buffers for
 * what the config uses, capacities >= lsq_state_sizes.  The buffer contents
 * are not read.  A persistent-policy handle starts uncalibrated. */
lsq_status lsq_state_alloc(const lsq_config* cfg, const lsq_buffers* bufs, lsq_state** out);

/* Destroy a handle (the device buffers stay the caller's).  NULL is a no-op. */
void lsq_state_free(lsq_state* st);

/* Copy of the handle's configuration (host). */
lsq_status lsq_state_config(const lsq_state* st, lsq_config* out);

/* S_0 = 0: zero codes, scales, ref and f32 with a fill kernel (capturable in
 * a HIP graph).  A persistent-policy handle becomes uncalibrated. */
lsq_status lsq_state_zero(lsq_state* st, void* stream);

/* Load an fp32 state S [heads][Dv][Dk] (device) into the handle: one scale per
 * group s = fl(absmax/qmax), codes clamp(RNE(S * fl(1/s))); the yoked policy
 * also copies S into ref; bits 32 copies S into f32.  Freezes the scales of a
 * persistent-policy handle (marks it calibrated).  This is the calibration of
 * the persistent-scale arm of "When Dynamic Scaling Fails" (abstract). */
lsq_status lsq_state_calibrate(lsq_state* st, const float* S, void* stream);

/* The dequantised state: S [heads][Dv][Dk] fp32 (device, caller-owned, 16-byte
 * aligned) receives fl(C s) for every element, C the stored code and s its
 * group's scale in the stored format (or the head's scale for group 0), the
 * value a step starts from before its decay ("Preserving Updates in Low-Bit
 * Recurrent State Quantization", abstract: the low-bit state stands for the
 * full-precision one; its norm against an fp32 reference is the quantity of
 * "When Dynamic Scaling Fails", norm-inflation figure).  bits 32 copies the
 * fp32 state.  Asynchronous on stream; the handle is not changed.
 * INVALID_ARG for a null or misaligned S. */
lsq_status lsq_state_dequantize(const lsq_state* st, float* S, void* stream);

/* Declare that the bound scale buffer already holds frozen scales (resuming a
 * persistent-policy state from a copy of its buffers). */
lsq_status lsq_state_set_calibrated(lsq_state* st, int32_t calibrated);

/* The handle's step index t: the sequence position the next step uses for
 * dithered rounding.  It starts at 0 (lsq_state_alloc, lsq_state_zero) and
 * advances by one per step (lsq_decode_run: by H), whatever the rounding.
 * A checkpoint restores it with lsq_state_set_step_index (t >= 0, else
 * INVALID_ARG).  Host-only calls, no device work. */
lsq_status lsq_state_step_index(const lsq_state* st, int64_t* t);
lsq_status lsq_state_set_step_index(lsq_state* st, int64_t t);

/* One decode step for all heads (shapes above): Eq. (1) of "LinQuant:
 * Functional Invariances for Low-Precision Linear Recurrences" (Theoretical
 * Foundation) applied to the dequantised state, the output read from the
 * updated fp32 state, and the state requantised under the handle's scale
 * policy and rounding, as "When Dynamic Scaling Fails" (abstract) describes
 * the per-token requantisation of the decode step; the arithmetic contract at
 * the top of this file states every operation.  alpha has [heads] or
 * [heads][Dk] entries by the decay flag.  o_ref may be NULL; it is written
 * only by the yoked policy.  The state is updated in place and the handle's
 * step index advances by one.
 *
 * Ownership and errors: every pointer is a device pointer the caller owns;
 * nothing is retained after the call returns (the launch is asynchronous on
 * stream).  INVALID_ARG for a null handle or data pointer, or one that is not
 * 16-byte aligned (q, k, a diagonal alpha) or 4-byte aligned (v, a scalar
 * alpha, beta, o); NOT_CALIBRATED for a persistent-policy handle that was never
 * calibrated; HIP for a launch failure.
 *
 * HIP graphs: the launch allocates nothing and records no memset, so it can be
 * captured.  The step index, and with it the dither's sequence positions, the
 * bypass slot that is filled and which of the two b copies is read, is taken
 * from the handle on the host when the launch is issued: a captured launch
 * keeps the values of the step it was captured at.  Replaying a captured
 * sequence therefore redoes those same steps (same positions, same slots); to
 * advance a decode with a graph, capture as many steps as one replay should
 * take and, for the bypass, a whole number of merge periods starting at a
 * period boundary, and set the handle's step index (lsq_state_set_step_index)
 * to what the replays have reached before issuing further uncaptured steps. */
lsq_status lsq_decode_step(lsq_state* st, const float* q, const float* k, const float* v,
                           const float* alpha, const float* beta, float* o, float* o_ref,
                           void* stream);

/* H sequential decode steps over a decode horizon H: the state is rewritten
 * and requantised at every step of the horizon ("When Dynamic Scaling Fails",
 * abstract: the requantisation happens per token, and its effect is measured
 * against the horizon H), each step exactly lsq_decode_step.  Every input
 * carries a leading [H] axis (contiguous, step-major), o (and o_ref) receive
 * [H][heads][Dv].  The state round-trips through device memory every step; H
 * kernel launches are issued on stream; the step index advances by H.  H = 0
 * or no heads: nothing is launched.  Errors as lsq_decode_step (a negative H
 * is INVALID_ARG); a launch failure part-way returns HIP with the earlier
 * steps issued. */
lsq_status lsq_decode_run(lsq_state* st, int32_t H, const float* q, const float* k,
                          const float* v, const float* alpha, const float* beta, float* o,
                          float* o_ref, void* stream);

/* Chunkwise prefill of T tokens (linear write, no readout), after the
 * low-precision chunkwise realisation in the Methodology of "LinQuant:
 * Functional Invariances for Low-Precision Linear Recurrences".  Tokens are
 * taken in chunks of 64 (the last one may be shorter).  Per chunk and head:
 *   Gamma->_t  product of the decays of the chunk's later tokens (fp32, from
 *              the chunk's end; the diagonal decay per column),
 *   gamma^C    the product over the whole chunk,
 *   H          = Q(beta v)^T Q(Gamma-> (.) k): each operand block ([tokens x
 *              Dv] and [tokens x Dk]) is quantised to INT8 with one absmax
 *              scale s = max|x| / 127 and round-half-even codes; the integer
 *              product is exact and H = fl(h * fl(s_V * s_K)),
 *   X          = fma(gamma^C, S, H), requantised in the state's own group
 *              format and policy with round-half-even (a dynamic scale
 *              rounded to the stored scale format first, as in the decode
 *              step); the dequantised state fl(code * s) is carried to the
 *              next chunk.
 * Inputs carry a leading [T] axis (contiguous, token-major): k [T][heads][Dk],
 * v [T][heads][Dv], alpha [T][heads] (or [T][heads][Dk] for a diagonal
 * decay), beta [T][heads]; device pointers, 4-byte aligned, read-only.
 * Supported: bits 4 and 8; policy DYNAMIC or PERSISTENT (calibrated first);
 * delta 0 (the delta-rule write is sequential per token: use
 * lsq_decode_run); no bypass (lrb_rank 0); group scales along Dk (group >=
 * Dk / 8) in any stored format, or one scale per head (group 0: a dynamic
 * head scale is taken over all of the head's X at every chunk); Dk and Dv in
 * {64, 128}; otherwise UNSUPPORTED.  The state pass rounds half to even whatever the
 * handle's rounding field says.  T = 0 or no heads: nothing to do.  The step
 * index advances by T.  One workgroup per head walks the chunks in order. */
lsq_status lsq_prefill(lsq_state* st, int32_t T, const float* k, const float* v,
                       const float* alpha, const float* beta, void* stream);

/* ---- Slots: a serving program's states, addressed by sequence ----
 *
 * A handle's batch axis is a pool of sequences: slot b is heads [b*heads,
 * (b+1)*heads) of the state buffers.  The four calls below work on chosen
 * slots: a packed batch of prompts (lsq_attend), one token each
 * (lsq_step_slots), and copies between an fp32 handle and a quantised one
 * (lsq_state_store_slots, lsq_state_load_slots: a state cache).  Slot numbers
 * and sequence offsets are device data, so a captured launch may be replayed
 * with other slots; the host does not see them and the kernels check them:
 *   - a negative slot marks a padded entry: nothing of it is read or written
 *     (its output rows stay as they were);
 *   - a slot >= batch, or one that an earlier entry of the same call already
 *     takes, is refused on the device: no state is touched and the entry's
 *     output rows are filled with NaN (a copy of slots leaves the destination
 *     as it was).  The first entry that has something to do with a slot takes
 *     it: an empty sequence takes none, nor does a copy whose source is padded
 *     or beyond its handle.
 * Token inputs use LSQ_IO_* types for q, k, v and o; alpha and beta are fp32.
 */
typedef enum { LSQ_IO_F32 = 0, LSQ_IO_F16 = 1, LSQ_IO_BF16 = 2 } lsq_io_type;

/* A packed batch of tokens.  Token t of q and k holds qk_heads vectors of dk
 * elements, of v and o heads vectors of dv elements, contiguous within the
 * token; consecutive tokens are q_stride, ... elements apart (a slice of a
 * wider projection, or 0 for an input that all tokens share).  Value head h
 * reads q and k of head h / (heads / qk_heads).  alpha is [tokens][heads], or
 * [tokens][heads][dk] under a diagonal decay, and beta [tokens][heads], both
 * contiguous.  Sequence i owns tokens [cu_seqlens[i], cu_seqlens[i+1]) and
 * slot slots[i]; tokens outside every sequence are neither read nor written.
 * Offsets must not decrease and lie in [0, tokens]; others are clamped, so
 * that nothing outside the batch is touched, and their sequences' values are
 * unspecified.  fresh[i] != 0 starts sequence i from S = 0 instead of its slot's
 * state (whose old contents, even NaN, do not matter).  An empty sequence
 * leaves its slot as it was. */
typedef struct {
  int32_t io;                 /* lsq_io_type of q, k, v and o */
  int32_t qk_heads;           /* heads of q and k; divides the handle's heads */
  int32_t seqs;               /* sequences (entries) */
  int64_t tokens;             /* rows of q, k, v, alpha, beta and o */
  int64_t q_stride, k_stride, v_stride, o_stride;   /* elements from one token to the next */
  const void* q;
  const void* k;
  const void* v;
  const float* alpha;
  const float* beta;
  void* o;
  const int32_t* cu_seqlens;  /* [seqs + 1]; not read by lsq_step_slots */
  const int32_t* slots;       /* [seqs], or NULL: entry i is slot i */
  const uint8_t* fresh;       /* [seqs], or NULL: none is fresh */
} lsq_token_batch;

/* Bytes of workspace lsq_attend needs for this batch (0 when it needs none, as
 * every batch of up to 1024 tokens).
 * Host only; depends on the handle's configuration, io, qk_heads, seqs and
 * tokens alone. */
lsq_status lsq_attend_workspace(const lsq_state* st, const lsq_token_batch* batch, size_t* bytes);

/* Linear attention over a packed batch of prompts, with outputs: for every
 * sequence the recurrence of Eq. (1) of "LinQuant: Functional Invariances for
 * Low-Precision Linear Recurrences" (Theoretical Foundation) from its slot's
 * state (or 0), o_t = S_t q_t for every token, and the final state back to
 * the slot.  The handle is an fp32 one (bits 32).  With a scalar decay and
 * the linear write (delta 0) the tokens are taken in chunks on the matrix
 * cores, as in that page's chunkwise realisation (Methodology) without its
 * INT8 operands: states and sums are fp32, operands are split so that the
 * state and fp32 outputs keep fp32 accuracy (magnitudes from 2^-100 to 2^127;
 * smaller ones lose their last bits, larger ones may count as infinite).  The
 * operands of a 16-bit output are held to 16 bits: before its one rounding it
 * is off by at most 2^-16 (bf16) or 3 2^-16 (binary16) of the sum of its terms'
 * magnitudes, beside fp32's own rounding.  A diagonal decay or the delta rule
 * walks the tokens one by one with the state in registers, all in fp32.
 * alpha lies in [0, 1].  The chunk form works with its logarithm: an alpha
 * below 2^-126 counts as 0 and forgets what was before (a product of several
 * alphas below it may too); a negative one gives NaN from its token on.  The walk,
 * like lsq_step_slots, multiplies the state by alpha as it stands, also by one
 * that is negative or subnormal.  A NaN alpha gives NaN from its token on.  A v
 * that is not finite makes its value column so from its token on (NaN in the
 * chunk form), a q its own output; nothing reaches an earlier token, another
 * column or, of alpha and beta, another head.
 * A long sequence is taken in segments whose states pass through the
 * workspace; the same batch gives the same bits on every call.
 *
 * q, k (and a diagonal alpha): 16-byte aligned, their token strides a
 * multiple of 16 bytes; v, o, alpha and beta element-aligned (wide accesses
 * are used where their addresses allow).  o must not overlap an input.  The
 * workspace is device memory, 16-byte aligned, used by this call alone until
 * the stream has passed it (two captured graphs that may run at once need two).
 * The step index does not move.  INVALID_ARG: null or misaligned pointers,
 * seqs < 0, tokens < 0, qk_heads not dividing heads, an o_stride below
 * heads * dv or a negative stride, a workspace of NULL where one is needed;
 * BUFFER_TOO_SMALL: a smaller workspace; UNSUPPORTED: a quantised handle, a
 * token stride of 32 MiB or more (chunk form), or a launch of 2^32 threads or
 * more. */
lsq_status lsq_attend(lsq_state* st, const lsq_token_batch* batch, void* workspace,
                      size_t workspace_bytes, void* stream);

/* The recurrent form: one token for every entry (tokens == seqs, token i is
 * entry i's; cu_seqlens is not read).  fp32 handle, either decay, either
 * delta.  The arithmetic is the fp32 step's: S' = fl(alpha_c S), w = fl(beta
 * fl(v - delta S'.k)), S = fma(w, k_c, S'), o = S.q rounded once to the io
 * type.  The step index does not move.  Errors as lsq_attend. */
lsq_status lsq_step_slots(lsq_state* st, const lsq_token_batch* batch, void* stream);

/* Quantise slots of an fp32 handle into slots of a quantised one: entry i
 * takes slot src_slots[i] of src to slot dst_slots[i] of dst (either array
 * NULL: entry i is slot i), with the scales and codes of
 * lsq_state_calibrate, in dst's group format (the yoked reference is copied
 * too).  Only dst's slots are checked for repetition: one state may go to
 * many pages.  dst's calibrated flag does not move: a persistent handle whose
 * slots are all filled this way is declared with lsq_state_set_calibrated.
 * INVALID_ARG: null handles, a negative count, handles of different heads,
 * dk or dv; UNSUPPORTED: src not fp32, dst not quantised or with a bypass
 * (its buffer belongs to one step index for all slots). */
lsq_status lsq_state_store_slots(lsq_state* dst, const lsq_state* src, int32_t count,
                                 const int32_t* dst_slots, const int32_t* src_slots,
                                 void* stream);

/* The reverse: slots of a quantised handle read back into slots of an fp32
 * one, S = fl(C s) as lsq_state_dequantize gives it.  Checks and errors as
 * lsq_state_store_slots with the handles' roles exchanged. */
lsq_status lsq_state_load_slots(lsq_state* dst, const lsq_state* src, int32_t count,
                                const int32_t* dst_slots, const int32_t* src_slots,
                                void* stream);

/* ---- Drafted tokens over the slots of an fp32 handle ----
 *
 * A program that drafts tokens holds, for each sequence, a tree of nodes: node j
 * continues node parents[j] < j, or the slot's own state where parents[j] is
 * -1 (node 0 is usually the last token of the sequence, which the slot does
 * not hold yet).  lsq_step_tree gives the output of every node, lsq_verify_tree
 * tests the drafted nodes against the target model's probabilities, and
 * lsq_accept_path writes the nodes of the accepted path into the slot.  Trees
 * have up to 64 nodes.  Node numbers count within their tree; node j of entry i
 * is row cu[i] + j of the packed arrays.  As in the calls above, slots,
 * offsets, parents and paths are device data, checked by the kernels, and the
 * calls may be captured and replayed with other values in them.
 */

/* The recurrence along every path of the trees: for node j with parent p,
 *   S_j = alpha_j S_p + beta_j (v_j - delta alpha_j S_p k_j) k_j^T,   o_j = S_j q_j,
 * where S_-1 is the slot's state (0 for a fresh entry).  The batch is
 * lsq_attend's, cu_seqlens [seqs + 1] being the nodes' offsets (clamped as there);
 * max_nodes bounds the nodes of a tree.  The slots are read only, so several
 * entries may name one slot.  Output rows outside every tree, and those of
 * negative slots, are not written.  A slot >= batch, a tree of more than
 * max_nodes nodes and one with a parent outside [-1, j) are refused on the
 * device: their output rows are filled with NaN.  The step index does not
 * move.  max_nodes also chooses the kernel's size (16, 32 or 64 nodes): a bound
 * above what the trees need costs time (256 trees of 8 nodes: 109 us for 16, 121
 * for 32, 127 for 64).
 *
 * The nodes are worked together on the matrix cores, the state read once.
 * Operands and sums keep fp32 accuracy for every io type (magnitudes from 2^-100
 * to 2^127, as lsq_attend's fp32 outputs), and an output is rounded once.
 * |alpha| is at most 1; a
 * negative one is taken as it stands; under a scalar decay one below 2^-126 in
 * magnitude counts as 0.  An input that is not finite makes outputs NaN or
 * infinite on its node and the nodes behind it, v its own value column alone,
 * q its own node alone; nothing reaches a node off its paths or another head.
 *
 * Alignment and errors as lsq_attend (no workspace); INVALID_ARG also:
 * max_nodes < 1, null or misaligned parents; UNSUPPORTED: a quantised handle,
 * max_nodes > 64, a token stride of 2^31 elements or more, or a launch of 2^32
 * threads or more. */
lsq_status lsq_step_tree(const lsq_state* st, const lsq_token_batch* batch, const int32_t* parents,
                         int32_t max_nodes, void* stream);

/* Accepted paths into the state: entry i advances its slot (or 0 where fresh) by
 * nodes path[i][0 .. lengths[i]), in this order, each as one token of the
 * recurrence; path is [seqs][depth].  The batch is lsq_step_tree's; its q and o
 * are not used and may be NULL.  An entry with a length of 0 or less does
 * nothing, like one with a negative slot, and takes no slot.  A slot >= batch or
 * taken by an earlier entry, a length above depth, and a node outside the
 * entry's tree are refused on the device: the state stays as it was (a refused
 * entry with a length above 0 takes its slot all the same).  The
 * arithmetic is lsq_step_slots', token by token in fp32, whatever the io type.
 * depth = 0 does nothing.  Errors as lsq_step_slots; INVALID_ARG also: null or
 * misaligned path or lengths, depth < 0; UNSUPPORTED also: depth > 64. */
lsq_status lsq_accept_path(lsq_state* st, const lsq_token_batch* batch, const int32_t* path,
                           const int32_t* lengths, int32_t depth, void* stream);

/* Trees of drafted tokens and the probabilities they are tested against.  Row j
 * of target (and draft) is the target (draft) model's distribution behind node
 * j, that of its children; consecutive rows are target_stride (draft_stride)
 * elements apart.  ids[j] is node j's token (node 0's is not used), uniform[j]
 * the number in [0, 1) that decides on node j, uniform_next[i] the one that
 * draws entry i's next token.  draft NULL: the drafts have no probabilities
 * (each is certain to its model: a one-hot row).  replacement: siblings were
 * drawn independently of each other (1), or without replacement (0; not used
 * where draft is NULL). */
typedef struct {
  int32_t seqs, vocab;
  int32_t depth;               /* most nodes of a path, columns of path */
  int32_t replacement;
  int64_t nodes;               /* rows */
  int64_t target_stride, draft_stride;
  const float* target;
  const float* draft;          /* or NULL */
  const int32_t* ids;          /* [nodes] */
  const int32_t* parents;      /* [nodes] */
  const int32_t* cu_nodes;     /* [seqs + 1] */
  const float* uniform;        /* [nodes] */
  const float* uniform_next;   /* [seqs] */
  int32_t* path;               /* [seqs][depth], out */
  int32_t* lengths;            /* [seqs], out */
  int32_t* next;               /* [seqs], out */
} lsq_draft_batch;

/* Bytes of workspace lsq_verify_tree needs for this batch (0 for vocabularies of
 * up to 65536 tokens).  Host only; depends on seqs, nodes, vocab and whether draft
 * is NULL alone. */
lsq_status lsq_verify_workspace(const lsq_draft_batch* batch, size_t* bytes);

/* Verification: entry i's walk starts at node 0, which is accepted as it
 * stands, and tests the children x_1, x_2, ... of the node it is at, in order (a
 * second node with parent -1 is nobody's child), with p and q the node's target
 * and draft row.  P_1 = p, T_1 = Q_1 = 1, c_1 = 0:
 *   x_i is accepted if uniform T_i q(x_i) < P_i(x_i) Q_i, and the walk goes on
 *   there; otherwise c_i+1 = c_i + T_i / Q_i, P_i+1 = max(p - c_i+1 q, 0), T_i+1 is
 *   its sum, and Q_i+1 is 1, or without replacement 1 - q(x_1) - ... - q(x_i) and,
 *   where that is below 1/16, the sum of q over the tokens not tried (in a small
 *   difference a row's own rounding would count).
 * (P / T is what the residual rule of rejection sampling leaves for the next
 * sibling, so that every accepted or drawn token has the target's distribution.)
 * Without draft probabilities x_i is accepted if uniform T_i < P_i(x_i), else P_i+1
 * is P_i without x_i and T_i+1 = T_i - P_i(x_i).  Where no child is accepted,
 * or the path has depth nodes, the next token is the first y whose cumulative
 * sum of P (of p where the path is full) exceeds uniform_next times its sum;
 * where P is empty, of p; -1 where that is empty too.  All of it is fp64.  Of a
 * node's draft row only its children's tokens count where no child is rejected:
 * the rows of nodes without children may hold anything.
 * A NaN or a negative number counts as 0 in either row, and a node whose token
 * lies outside [0, vocab) is passed over.  Out: path, node 0 first, -1 behind its end; its
 * length; next.  An empty tree, one of more than 64 nodes, and one with a
 * parent outside [-1, j) get the length 0, next -1 and a path of -1; offsets
 * are clamped to [0, nodes].  The workspace is device memory, 16-byte aligned,
 * used by this call alone until the stream has passed it.  INVALID_ARG: null
 * arrays, arrays not 4-byte aligned, seqs < 0, nodes < 0, vocab < 1, depth < 1,
 * a negative stride, replacement not 0 or 1, a workspace of NULL where one is
 * needed; BUFFER_TOO_SMALL: a smaller workspace; UNSUPPORTED: vocab > 2^22, or
 * a launch of 2^32 threads or more. */
lsq_status lsq_verify_tree(const lsq_draft_batch* batch, void* workspace, size_t workspace_bytes,
                           void* stream);

/* Static description of a status code. */
const char* lsq_status_string(lsq_status s);

/* Detail of the last failing call on the calling thread ("" if none). */
const char* lsq_last_error(void);

/* Library version, major*10000 + minor*100 + patch. */
int32_t lsq_version(void);

#ifdef __cplusplus
}
#endif
#endif /* LSQ_H */
