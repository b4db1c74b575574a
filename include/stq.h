/*
 * stq.h — C ABI of the low-bit recurrent-state decode-step library (gfx950).
 *
 * The library keeps a pool of per-request recurrent states of gated
 * Delta-rule linear attention in packed 4/6/8-bit codes (plus FP16 "pivot"
 * units) with one 16-bit scale per key row and one per value column, and
 * advances them one decode token at a time:
 *
 *   unpack + dequantize -> gate -> delta update -> readout o = S^T q
 *   -> refit row/column scales -> requantize + repack.
 *
 * Sources (the method this implements is described, not specified, by these
 * pages; every choice they leave open is fixed below and marked READING):
 *  [P1] "直播预告！聊聊线性注意力的低比特量化方法：STEPQuant" (qingkeai.online),
 *       sections "高并发场景下的显存困境…" (per-token requantization of an
 *       approximate state), "STEPQuant 核心设计…" (dual-axis key-row fitting,
 *       lifetime-aware bits), "从状态压缩到高效服务…" (packed-state kernels).
 *  [P3] "线性注意力每生成一个token都要搬状态,LeapQuant…" (wink.run), techniques
 *       one, two and three: per-window quantization, compensator tokens
 *       (outliers kept at high precision), residual row smoothing.
 *  [P4] "STEPQuant: estados recurrentes a «6 bit»…" (gpt-diffusion.com),
 *       "Las dos ideas" (bit units: head for GDN, key row for KDA; FP16
 *       pivots) and "Qué dice realmente el «6-bit»" (6 + 16/128 + 16/128 bits
 *       per value: one 16-bit scale per row and per column).
 *  [P5] e-cogni.com.br STEPQuant analysis, "Contexto" (GDN scalar gate, KDA
 *       per-channel gate), "O que os autores propõem" and "Como funciona"
 *       (row scale from current row magnitude and row-impact score, column
 *       scale weighted toward high-impact rows, square-root smoothing,
 *       geometric-mean normalisation of the row factors).
 *
 * ------------------------------------------------------------------------
 * OWNERSHIP AND ERRORS
 *  - The caller owns all device memory (the pool buffer, every input and
 *    output) and every stream.  The library never allocates device memory,
 *    never synchronises, and keeps no global state; a stq_pool is a small
 *    host-side handle (host memory, owned by the library until
 *    stq_pool_destroy).
 *  - Arguments are validated synchronously on the host; a bad argument
 *    returns a negative status and enqueues nothing.  A failed launch
 *    returns STQ_ERR_HIP.  Device-side faults surface at the caller's next
 *    synchronisation of the stream.
 *  - Undefined (not checked on the device): duplicate slots within one call,
 *    non-finite inputs, |k| far from 1, b outside [0,1], concurrent calls on
 *    one pool from different streams, slot indices outside [0, n_slots).
 *    (Slot indices are range-checked on the device: out-of-range entries
 *    are skipped and their outputs left untouched.)
 *  - All pointers named *_dev are device pointers, all others host.
 *
 * ------------------------------------------------------------------------
 * STATE TILE (one per (slot, head)): S is d_k x d_v, row i = key channel,
 * column j = value channel (READING: the update is written for this
 * orientation; the page formula that names S k is the same map for S^T).
 * Supported d_k, d_v in {64, 128}.
 *
 * Widths n in {4, 6, 8, 16}; qmax(n) = 2^(n-1) - 1 in {7, 31, 127}.
 * n = 16 marks a PIVOT unit stored as IEEE binary16 without scales.
 * GDN pools (unit_kind HEAD): one width per head.  A pivot head is a whole
 * fp16 tile.
 *
 * Code field encoding (READING: the pages fix only the widths): a code Q in
 * [-qmax, qmax] is stored as the unsigned field Q + 2^(n-1) (offset binary;
 * the all-zero field is never produced).
 *
 * LANE LAYOUT.  Let NRC = d_k/32 (32-row chunks), NCC = 8/NRC (16-column
 * chunks per wave), CPW = 16*NCC (columns per 64-lane wave), NW = d_v/CPW.
 * Wave w in [0,NW), lane l in [0,64): G = l / 16, n = l % 16.  The lane
 * owns the 64 elements e = 8b + t (b = cc*NRC + rc in [0,8), t in [0,8)):
 *     row i = 32*rc + 16*(t/4) + 4*G + t%4,   col j = w*CPW + 16*cc + n.
 * Its LANE STREAM is the 16 GROUPS q = e/4 = 0..15 in order; group q holds
 * the codes of elements 4q..4q+3 (four consecutive rows of one column,
 * f0 = the lowest row) packed in n/2 bytes:
 *     n=4 : 2 bytes, byte0 = f0 | f1<<4, byte1 = f2 | f3<<4
 *     n=6 : 3 bytes, little-endian 24-bit word f0 | f1<<6 | f2<<12 | f3<<18
 *     n=8 : 4 bytes f0, f1, f2, f3
 *     n=16: 8 bytes, four binary16 values, little-endian
 * (f = stored field).  The lane stream has K = n/2 chunks of 16 bytes; chunk
 * k of lane l of wave w sits at code-region offset 16*((w*K + k)*64 + l), so
 * that one 16-byte load per lane reads 1 KiB contiguous per wave.  (The two
 * groups of chunk b are the lane's operand of a 32 x 16 block in the gfx950
 * 16x16x32 fp16 matrix instruction: G picks 8 of the 32 rows, n the column.)
 *
 * PER-ROW WIDTHS (unit_kind ROW, the KDA allocation unit = key row, [P4]
 * "Las dos ideas"): a tile is a list of ROW RECORDS, one per key row, each
 * the row's d_v codes in column order as 4-code groups of the encoding
 * above (d_v*n/8 bytes; a binary16 pivot row is d_v binary16 values),
 * records sorted by width (4, 6, 8, then 16; original order kept within a
 * width), then sigma[d_k] in original row order and c[d_v].  Pivot rows are
 * excluded from both scale fits (R2, R5).  Window mode is per-head only.
 *
 * TILE BYTES: codes (d_k*d_v*n/8 bytes), then for n != 16 the row scales
 * sigma[d_k] and column scales c[d_v] as bf16 little-endian.  Tile stride =
 * tile bytes rounded up to a multiple of 256.  (6-bit, 128x128: 12288 + 512
 * = 12800 bytes = 6.25 bits/value, i.e. 6 + 16/128 + 16/128 as in [P4].)
 *
 * ------------------------------------------------------------------------
 * REFIT R (requantize an fp32 tile S; [P1] core design, [P5] Como funciona).
 * fl() = binary32 round-to-nearest-even, bf16_rne/bf16_ru = round the value
 * to bfloat16 to nearest-even / toward +inf.  w_i = row-impact weight.
 *  R1  m_i = max_j |S_ij|.
 *  R2  non-pivot rows with p_i = fl(m_i*w_i) > 0: rho_i = fl(sqrt(p_i)),
 *      s_i = bf16_rne(rho_i), e_i = floor(log2 s_i); the set of such rows is
 *      A.  Every other row: s_i = 1.                       (square-root smoothing)
 *  R3  E = floor((2*sum_{i in A} e_i + |A|) / (2|A|)), E = 0 if A is empty
 *      (rounded mean exponent; READING of "geometric mean of the row
 *      factors is one": normalise by a power of two so codes never depend
 *      on it).
 *  R4  X_ij = fl(S_ij * fl(1/s_i)).
 *  R5  M_j = max over non-pivot rows of fl(|X_ij| * fl(1/qmax(n_i)));
 *      t_j = 1 if M_j == 0 (or no non-pivot row), else
 *      t_j = max(bf16_ru(M_j), 2^-126).
 *      (Rounding toward +inf guarantees |Q| <= qmax without clipping.)
 *  R6  Q_ij = round-half-even(X_ij * fl(1/t_j)) of the exact product.
 *  R7  pivot rows: H_ij = binary16 round-half-even of S_ij clamped to
 *      [-65504, 65504].
 *  R8  stored sigma_i = s_i * 2^-E and c_j = t_j * 2^E, as exponent-field
 *      arithmetic on the bf16 values with the biased exponent clamped to
 *      [1, 254].
 * DEQUANTIZE D: S^_ij = fl(fl(sigma_i*c_j)*Q_ij) (exact for non-extreme
 * scales: 8 x 8 x 7 significant bits), pivot: binary16 -> binary32.
 *
 * DECODE STEP (per (request, head) tile; [P5] Contexto, [P1] memory dilemma):
 *   GDN: A = a*S^, a scalar per (request, head).   KDA: A = Diag(a) S^.
 *   u = A^T k, delta = b*(v - u), S' = A + k delta^T  (= a(I - b k k^T)S^ +
 *   b k v^T for GDN), o = S'^T q read from the fp32 S' before requantizing,
 *   then the tile becomes R(S').  IDENTITY RULE (READING): when the update
 *   is exactly the identity (a == 1 for every gate of the tile and b == 0),
 *   S' = S^ is already represented exactly and the tile bytes are left
 *   unchanged instead of being refitted.  The fused kernel computes S' in binary32;
 *   its codes agree with R applied to the exactly rounded S' except for rare
 *   one-step rounding flips.  Gates lie in [0, 1]; a gate of 0 (or below the
 *   binary32 normal range) forgets the unit's old state: S'_i = k_i delta.
 *
 * WINDOW MODE (window = W > 0, GDN gate; [P3] per-window quantization and
 * residual smoothing): the quantized base S0 is frozen inside a window.  Per
 * token t the cache appends (k_t, u_t, G_t) in binary32 where G_t is the
 * product of the gates since the window opened (G_t = fl(G_{t-1} * a_t)),
 *   u_t = b_t (v_t - G_t S0^T k_t - sum_{s<t} (G_t/G_s)(k_s.k_t) u_s),
 *   o_t = G_t S0^T q_t + sum_{s<=t} (G_t/G_s)(k_s.q_t) u_s,
 * which is exactly the per-token recurrence started from S0.  After token
 * W's readout (or on stq_window_flush) the window is folded:
 *   S_W = G_W S0 + sum_s (G_W/G_s) k_s u_s^T  ->  R  -> new base, cache cleared.
 * (Use row_weight = 1 for the pages' plain per-row smoothing.)  The ratios
 * G_t/G_s need every G of a window to be a normal binary32 number: gates in
 * (0, 1] whose product over W tokens stays >= 2^-126.  Smaller products are
 * outside the contract of window mode (the per-token mode accepts any gate).
 *
 * COMPENSATOR TOKENS (n_comp = C > 0, window mode; [P3] technique two, the
 * largest outliers kept at high precision as rank-one terms on the window's
 * update path).  READING: whenever a quantized tile's base is written (ingest,
 * fold, flush), the C key rows of largest absolute value of the binary32
 * state being written (row absmax; ties to the lower row; all-zero rows never)
 * are kept exactly, in binary32, as rank-one terms e_i u^T (u = that row), and
 * R quantizes the residual, those rows set to zero.  The represented base is
 * then S0 = D(tile) + sum_c e_{i_c} u_c^T; inside a window the compensators are
 * gated with it and read out as cached tokens with k = e_{i_c} and G = 1:
 *   u_t, o_t as above with S0 including them; the fold materialises S_W from
 *   that S0 and takes its compensators anew.  A binary16 pivot head takes
 *   none (its slots hold row -1 and zeros).  A fresh pool holds row 0 with
 *   zero values in every slot, which adds nothing.
 *
 * ------------------------------------------------------------------------
 * POOL BUFFER (one caller-owned device buffer of stq_pool_bytes() bytes):
 *  header (HDR bytes):
 *    [0,4) magic 0x31515453 ('STQ1')  [4,8) n_slots  [8,12) n_heads
 *    [12,16) d_k  [16,20) d_v  [20,24) gate_kind  [24,28) unit_kind
 *    [28,32) window | n_comp << 16  [32,40) slot_bytes  [40,48) slots_off  [48,56) cache_off
 *    [56,64) cache_stride   (integers little-endian, u64 for the last four)
 *    [64, 64+4H)    int32 width of head h (0 for per-row units)
 *    [64+4H, 64+8H) uint32 byte offset of head h's tile inside a slot
 *    [WOFF, WOFF+4*H*d_k) fp32 row weights [H][d_k], WOFF = roundup(64+8H,256)
 *    ROFF = roundup(WOFF + 4*H*d_k, 256); per-row units only:
 *    [ROFF, +H*d_k) uint8 width of row i of head h (original order),
 *    [+H*d_k, +2H*d_k) uint8 original row of record p, then int32 [H][4]
 *    counts of rows of width 4, 6, 8, 16;
 *    HDR = ROFF (per-head units) or roundup(ROFF + 2*H*d_k + 16*H, 256)
 *  slots: slots_off = HDR, slot s at slots_off + s*slot_bytes; head h's tile
 *    at + head_off[h]; head_off = running sum of tile strides.
 *  window caches (window > 0): cache_off = slots_off + n_slots*slot_bytes,
 *    tile (s,h) at cache_off + (s*H + h)*cache_stride, cache_stride =
 *    256 + 4*W*(d_k + d_v) + 4*C*d_v:  [0,4) int32 t = tokens in the open
 *    window, [4+4m) fp32 G of token m+1 (m < W), [192 + 4c) int32 row of
 *    compensator c, [256 + 4*d_k*m) fp32 k of token m+1,
 *    [256 + 4*W*d_k + 4*d_v*m) fp32 u of token m+1,
 *    [256 + 4*W*(d_k + d_v) + 4*d_v*c) fp32 values of compensator c.
 * Inputs of a call with n requests: q, k, v fp32 [n][H][d] (d = d_k for q, k,
 * d_v for v), a fp32 [n][H] (GDN) or [n][H][d_k] (KDA), b fp32 [n][H],
 * o fp32 [n][H][d_v]; request c of the call uses slot slots_dev[c].
 */
#ifndef STQ_H
#define STQ_H

#include <stddef.h>
#include <stdint.h>
#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef int32_t stq_status;
#define STQ_OK               0
#define STQ_ERR_ARG         -1  /* bad pointer, size, count or descriptor field */
#define STQ_ERR_LAYOUT      -2  /* buffer too small / misaligned, header mismatch */
#define STQ_ERR_HIP         -3  /* a HIP runtime call or launch failed */
#define STQ_ERR_STATE       -4  /* call not valid for this pool (e.g. flush without window) */
#define STQ_ERR_UNSUPPORTED -5  /* valid request outside what the library implements */

#define STQ_GATE_HEAD     0  /* GDN: scalar gate per (request, head) */
#define STQ_GATE_CHANNEL  1  /* KDA: gate per (request, head, key channel) */
#define STQ_UNIT_HEAD     0  /* one bit width per head */
#define STQ_UNIT_ROW      1  /* one bit width per key row */

typedef struct stq_pool stq_pool;

/* Static pool description (the offline "plan": bit map and row impacts are
 * calibrated once and frozen across requests, [P4] "Las dos ideas", [P5]
 * Limitações).  All arrays are host memory, read during the call only. */
typedef struct stq_pool_desc {
  int32_t n_slots;      /* persistent request states in the pool (>= 1)      */
  int32_t n_heads;      /* H >= 1                                           */
  int32_t d_k, d_v;     /* each 64 or 128                                   */
  int32_t gate_kind;    /* STQ_GATE_HEAD or STQ_GATE_CHANNEL                */
  int32_t unit_kind;    /* STQ_UNIT_HEAD or STQ_UNIT_ROW                    */
  int32_t window;       /* 0 = requantize every token; W in [1,32] = window */
  int32_t n_comp;       /* window mode: compensator rows per tile, 0..8,     */
                        /* window + n_comp <= 32; 0 without a window         */
  const int32_t* unit_bits;  /* [H] (HEAD) or [H][d_k] (ROW): 4, 6, 8 or 16   */
  const float* row_weight;   /* [H][d_k] row-impact weights, finite and > 0   */
} stq_pool_desc;

/* Human-readable name of a status code (static string, never NULL). */
const char* stq_status_str(stq_status s);

/* Bytes of the single device buffer a pool with this description needs
 * (header + slots + window caches).  Returns 0 for an invalid description. */
size_t stq_pool_bytes(const stq_pool_desc* desc);

/* Validates desc, checks dev_buf (256-byte aligned, >= stq_pool_bytes) and
 * enqueues on `stream` the header upload and the zeroing of all slots and
 * caches (an all-zero state: codes 0, scales 1, empty windows).  *out
 * receives a host handle.  The header's host staging copy lives in the
 * handle, so the upload may still be in flight when this returns; the
 * handle records an event after it (stq_pool_destroy waits for that event).
 * STQ_ERR_HIP if the event, the upload or the zeroing launch fails. */
stq_status stq_pool_create(const stq_pool_desc* desc, void* dev_buf, size_t bytes,
                           hipStream_t stream, stq_pool** out);

/* Frees the host handle only (the device buffer stays the caller's).  It
 * first waits for the header upload that stq_pool_create enqueued (the
 * upload reads the handle's staging copy); no other work is waited for:
 * steps, stores and fetches enqueued through the handle may still be
 * running, they do not read the handle.  STQ_ERR_HIP if that wait fails
 * (the handle is freed all the same). */
stq_status stq_pool_destroy(stq_pool* pool);

/* Ingest: for each c < n, tile (slots_dev[c], h) := R(S_dev[c][h]) for every
 * head (S_dev fp32 [n][H][d_k][d_v], row-major), and the slot's windows are
 * emptied.  Bit-exact with the definition of R above. */
stq_status stq_pool_store(stq_pool* pool, const int32_t* slots_dev, int32_t n,
                          const float* S_dev, hipStream_t stream);

/* Inspect: S_dev[c][h] := D(tile (slots_dev[c], h)) (in window mode the
 * frozen base only, without the open window's updates; with compensator
 * tokens the base includes them: D(tile) + sum_c e_{i_c} u_c^T). */
stq_status stq_pool_fetch(const stq_pool* pool, const int32_t* slots_dev, int32_t n,
                          float* S_dev, hipStream_t stream);

/* One decode token for n requests and all heads (see DECODE STEP / WINDOW
 * MODE above): reads q, k, v, a, b, writes o and advances the states.
 * Range: every entry of q and k must have magnitude below 2 (queries and keys
 * of the gated delta rule are L2-normalised, so |entry| <= 1).  The step
 * feeds the matrix cores the products gate * row scale * (q or k) as binary16
 * pairs scaled so that the largest gate * row scale of the tile (per-key-row
 * units: of the 32 key rows a wave holds) sits in [2^14, 2^15); larger entries
 * overflow binary16 and the results of that tile are undefined.  Not checked
 * (the vectors live on the device). */
stq_status stq_decode_step(stq_pool* pool, const int32_t* slots_dev, int32_t n,
                           const float* q_dev, const float* k_dev, const float* v_dev,
                           const float* a_dev, const float* b_dev, float* o_dev,
                           hipStream_t stream);

/* Prefill ingest ([P3] section on decode cost and state memory under prefix
 * caching: a request's state is produced once from its prompt and then held
 * in the pool).  For request c < n and every head h, runs the gated delta
 * rule over the request's tokens seq_start_dev[c] .. seq_start_dev[c+1]-1,
 * starting from D(tile (slots_dev[c], h)) (the all-zero state of a fresh
 * slot), and
 *   - writes the readout o_t = S_t^T q_t of every token, S_t the binary32
 *     state after token t (no requantization between tokens), and
 *   - writes the final state into the tile through R once.
 * A request with no tokens, or whose tokens are all the identity (a = 1 and
 * b = 0), leaves its tiles as they are (the decode step's identity rule; in
 * a window pool, as they are after the fold below).
 * Layouts, token-major as a packed batch of prompts: q_dev, k_dev fp32
 * [tok][H][d_k]; v_dev [tok][H][d_v]; a_dev [tok][H] (per-channel gate:
 * [tok][H][d_k]); b_dev [tok][H]; o_dev [tok][H][d_v]; seq_start_dev int32
 * [n+1], non-decreasing (a decreasing pair is an empty request).  All device
 * pointers, owned by the caller.
 * The state runs in binary32 (its products on the matrix cores in binary32;
 * the chunks' gate products formed in binary64 and rounded once):
 * S_T and o differ from the exact recurrence by binary32 rounding only, so
 * a final code can differ from R of the exact state where that state sits
 * within rounding of a code boundary.  Requests must name distinct slots.
 * Window pools: every listed slot's open window is folded first (as
 * stq_window_flush does); the prompt then runs from the base plus its
 * compensator rows, and the final state is written as stq_pool_store writes
 * one (compensator rows taken again, window empty).
 * Every pool kind, by the chunkwise form on the matrix cores (chunks of 32
 * tokens; with per-channel gates the chunk's gate products Gamma_t, per key
 * channel, scale the keys and queries, K.Gamma, Q.Gamma and K/Gamma, and from
 * a chunk whose smallest Gamma falls below 2^-60, a zero gate included, the
 * request's remaining tokens run token by token); per-key-row units run
 * the state in record-row order (rows sorted by width, k, q and gates read
 * through the head's record -> row permutation) and write the final state
 * through R for per-key-row widths, packed into the row records on chip. */
stq_status stq_prefill(stq_pool* pool, const int32_t* slots_dev, int32_t n,
                       const int32_t* seq_start_dev, const float* q_dev, const float* k_dev,
                       const float* v_dev, const float* a_dev, const float* b_dev, float* o_dev,
                       hipStream_t stream);

/* Prefill on plain binary32 states, no pool: S_dev [n][n_heads][d_k][d_v]
 * (row-major tiles, the layout of stq_pool_fetch) is advanced in place over
 * each request's tokens exactly as stq_prefill advances a tile's state
 * (same paths, same layouts of seq_start, q, k, v, a, b, o; gate_kind
 * STQ_GATE_HEAD or STQ_GATE_CHANNEL), and every token's readout is written.
 * It is also a direct check of the evaluation: the state after the prompt,
 * before any requantization.  A request with no tokens leaves its state as
 * it is.  STQ_ERR_ARG on bad sizes or null pointers. */
stq_status stq_prefill_states(int32_t n, int32_t n_heads, int32_t d_k, int32_t d_v, int32_t gate_kind,
                              float* S_dev, const int32_t* seq_start_dev, const float* q_dev,
                              const float* k_dev, const float* v_dev, const float* a_dev,
                              const float* b_dev, float* o_dev, hipStream_t stream);

/* The decode step split in two, for overlapped writeback ([P4] "Las dos
 * ideas": the pages' serving system writes back on a separate stream so that
 * the state updates overlap the model's other work).  stq_decode_readout
 * writes o exactly as stq_decode_step would and leaves the pool untouched;
 * stq_decode_commit then advances the states exactly as stq_decode_step
 * would (same bytes), writing no o.  Same inputs, same layouts and range
 * contract as stq_decode_step.  The commit rewrites the tiles the readout
 * reads: it must be ordered after the readout of the same slots (same
 * stream, or an event), and the next readout of those slots after the
 * commit.  The pair reads each tile twice (one read more than the fused
 * step): it can make o available before the writeback where the memory is
 * otherwise idle between layers; it adds bytes, never removes them.
 * Per-head units without a window only; otherwise STQ_ERR_UNSUPPORTED. */
stq_status stq_decode_readout(stq_pool* pool, const int32_t* slots_dev, int32_t n,
                              const float* q_dev, const float* k_dev, const float* v_dev,
                              const float* a_dev, const float* b_dev, float* o_dev,
                              hipStream_t stream);
stq_status stq_decode_commit(stq_pool* pool, const int32_t* slots_dev, int32_t n,
                             const float* q_dev, const float* k_dev, const float* v_dev,
                             const float* a_dev, const float* b_dev, hipStream_t stream);

/* Window mode only: fold the open window of each listed slot into its base
 * now (S = G_t S0 + sum_s (G_t/G_s) k_s u_s^T -> R), e.g. when a request ends
 * or before a snapshot.  A slot with an empty window is left unchanged.
 * Returns STQ_ERR_STATE on a pool without a window. */
stq_status stq_window_flush(stq_pool* pool, const int32_t* slots_dev, int32_t n,
                            hipStream_t stream);

/* Lifetime-aware bit allocation (host only; the offline step that produces a
 * pool's unit_bits).  [P1] "STEPQuant 核心设计…" (time axis: widths from each
 * unit's error per width and its lifetime, under a fixed budget); [P5] "O que
 * os autores propõem" (lifetime-weighted distortion minimised under a fixed
 * bit budget, riskiest units kept in binary16 as pivots) and "Como funciona"
 * (the lifetime weight decays about exponentially); [P4] "Qué dice realmente
 * el «6-bit»" (pivots counted apart from the nominal budget).  READING:
 *   w_u = sum_{t>=0} 2^(-t/h_u) = 1/(1 - 2^(-1/h_u)), h_u = half_life[u] > 0;
 *   the n_pivots units of largest w_u err[u][2] (ties to the lower index)
 *   become binary16 pivots (bits 16, no distortion);
 *   the other m units take b_u in {4, 6, 8} minimising
 *   sum_u w_u err[u][(b_u - 4)/2] subject to sum_u (b_u - 4)/2 <=
 *   floor((budget_bits - 4) m / 2) (binary64), i.e. mean width <= budget_bits.
 * err: host [n][3] distortion per step at 4, 6, 8 bits (finite, >= 0);
 * bits_out: host [n]; objective_out (may be NULL): the minimised sum.  Exact
 * (dynamic programming) while m * (budget steps + 1) <= 2^26; larger inputs
 * take greedy upgrades along each unit's lower convex hull (within one
 * unit's gain of the optimum).  STQ_ERR_ARG on n < 1, n_pivots outside
 * [0, n], budget_bits < 4, a non-positive half-life or a negative error. */
stq_status stq_allocate_bits(int32_t n, const double* err, const double* half_life, int32_t n_pivots,
                             double budget_bits, int32_t* bits_out, double* objective_out);

/* Test export (exact invariant "fixed-scale round trip"): requantize each
 * listed tile's own decoded state against its STORED scales,
 *   Q'_ij = round-half-even(fl(S^_ij * fl(1/sigma_i)) * fl(1/c_j)),
 * S^ = D(tile), sigma and c kept.  For every tile (whatever produced it)
 * this rewrites identical bytes: |Q| <= 127 keeps the two binary32
 * roundings far below half a code step.  Pivot units are rewritten as
 * binary16 of their own binary32 value, also unchanged. */
stq_status stq_requant_fixed_scales(stq_pool* pool, const int32_t* slots_dev, int32_t n,
                                    hipStream_t stream);

/* Diagnostic: out_dev[b] (fp32 [65536]) := the kernels' correctly rounded
 * reciprocal of the bf16 value with bit pattern b (meaningful for positive
 * normal values whose reciprocal is normal).  Used by the tests to check the
 * device reciprocal exhaustively against IEEE division. */
stq_status stq_debug_rcp_bf16(float* out_dev, hipStream_t stream);

/* ------------------------------------------------------------------------
 * THE SOFTMAX LAYERS OF A HYBRID MODEL.  The models whose recurrent states
 * this pool holds mix those layers with softmax attention ([P5] Contexto;
 * [P1] introduction).  The calls below serve the latter, in the pool's
 * manner: the caller owns every device buffer and stream, nothing is
 * allocated, nothing synchronises, arguments are checked on the host.  They
 * take no handle: a descriptor is read during the call only.
 *
 * KEY/VALUE CACHE: n_blocks blocks of block_tokens token slots each; token
 * slot s is slot s % block_tokens of block s / block_tokens.  A token's keys
 * and values hold, per key/value head, d channels in 4 bits: E2M1 codes
 * (magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6 for the low three bits, bit 3 the
 * sign) with one power-of-two scale 2^e per 32 channels, stored as the byte
 * e + 127.  Value = code * 2^e.  Of a block of 32 channels with largest
 * magnitude m, e is the least integer with m <= 6 * 2^e, held in [-23, 13]
 * (every cached value is then exact in binary16; magnitudes beyond 6 * 2^13
 * saturate), e = 0 for m = 0; codes round to the nearest level, ties to the
 * even code, and carry their element's sign, a zero's too.  A token and head whose key or value has an infinity or a NaN
 * is stored with NaN scales (byte 255) on the key and zeros as the value: a
 * query that sees it gets NaN, every other query is unaffected.
 * Bytes of block b, head h at (b * n_kv_heads + h) * block_tokens * d*17/16:
 *   key codes   [block_tokens][d/2]   byte i: channel 2i low, 2i+1 high nibble
 *   value codes [block_tokens][d/2]
 *   key scales  [d/32][block_tokens], value scales [d/32][block_tokens]
 */
typedef struct stq_kv_desc {
  int32_t n_blocks;      /* >= 1                                             */
  int32_t block_tokens;  /* 32, 64, 128 or 256                               */
  int32_t n_kv_heads;    /* >= 1                                             */
  int32_t d;             /* 64 or 128 channels of a head                     */
} stq_kv_desc;

#define STQ_BF16 0  /* element types of the calls below */
#define STQ_FP16 1
#define STQ_FP32 2

/* Bytes of the cache's device buffer; 0 for an invalid description.  The
 * buffer must be 16-byte aligned; its contents need no initialisation. */
size_t stq_kv_bytes(const stq_kv_desc* desc);

/* Block tables and slot maps from request lengths, in one launch.  Request
 * i < n has cached_dev[i] tokens in the cache and brings new_dev[i] more
 * (negative counts are taken as 0); row i of table_dev [n][table_cols] holds
 * its blocks, the first blocks(cached) entries on entry.  Writes
 *   tok_start_dev [n+1]  exclusive prefix sums of the new counts, and their sum;
 *   len_dev [n]          cached + new;
 *   table_dev            entries blocks(cached) .. blocks(cached+new)-1 of each
 *                        row, taken from free_dev in request order (-1 once
 *                        its n_free entries are used up); columns from
 *                        table_cols on are neither taken nor written, every
 *                        other entry is left as it was;
 *   pos_dev [n_tok]      position of new token t in its request;
 *   slot_dev [n_tok]     its token slot; -1 where its table entry is outside
 *                        [0, n_blocks) or past table_cols;
 *   used_dev [1]         blocks wanted; above n_free, the free list was short.
 * blocks(c) = ceil(c / block_tokens).  Entries of pos and slot from
 * tok_start[n] on (a padded batch) become -1; new tokens past n_tok get no
 * entry.  n in [1, 4096]; token and block sums must stay below 2^31.  No
 * output may overlap the counts or the free list (STQ_ERR_ARG). */
stq_status stq_kv_plan(int32_t n, const int32_t* cached_dev, const int32_t* new_dev, const int32_t* free_dev,
                       int32_t n_free, int32_t n_blocks, int32_t block_tokens, int32_t* table_dev,
                       int32_t table_cols, int32_t n_tok, int32_t* tok_start_dev, int32_t* len_dev,
                       int32_t* pos_dev, int64_t* slot_dev, int32_t* used_dev, hipStream_t stream);

#define STQ_NORM_NONE 0
#define STQ_NORM_RMS  1  /* y = x / sqrt(mean(x^2) + eps) * weight */
#define STQ_NORM_L2   2  /* y = x / sqrt(sum(x^2) + eps) * weight  */
#define STQ_ROT_HALVES   0  /* channel pairs (i, i + n_rot/2) */
#define STQ_ROT_ADJACENT 1  /* channel pairs (2i, 2i + 1)     */

/* Norm of queries and keys per head, with the position rotation of the first
 * n_rot channels in the same pass (binary32 inside, one rounding at the end).
 * The L2 form with binary32 output is the q and k of stq_decode_step and
 * stq_prefill.  Heads of one token are contiguous ([n_heads][d]); tokens are
 * *_stride elements apart. */
typedef struct stq_norm_desc {
  int32_t n_tok;            /* 0 .. 2^28                                      */
  int32_t n_q_heads;        /* >= 1                                           */
  int32_t n_k_heads;        /* >= 0 (0: no keys, k pointers unused)           */
  int32_t d;                /* 64, 128 or 256                                 */
  int32_t in_type;          /* STQ_BF16, STQ_FP16 or STQ_FP32                 */
  int32_t out_type;         /* in_type or STQ_FP32                            */
  int32_t norm;             /* STQ_NORM_*                                     */
  float eps;                /* > 0 with a norm                                */
  int32_t n_rot;            /* channels rotated: 0 or a multiple of 16, <= d  */
  int32_t rot_pairs;        /* STQ_ROT_*                                      */
  int32_t n_pos;            /* rows of the cosine and sine table              */
  int64_t q_stride, k_stride, q_out_stride, k_out_stride;
} stq_norm_desc;

/* q_weight_dev, k_weight_dev: fp32 [d] or NULL (ones).  With n_rot > 0,
 * pos_dev int32 [n_tok] and cos_sin_dev fp32 [n_pos][n_rot], a row the n_rot/2
 * cosines, then the n_rot/2 sines; pair (x, y) becomes (x cos - y sin,
 * y cos + x sin).  Rows of a token whose position lies outside [0, n_pos)
 * (a padded batch) are left as they were.  Outputs may be the inputs
 * themselves (same pointer, type and stride), else they must not overlap them
 * or each other (STQ_ERR_ARG; rows side by side in one buffer do not).
 * Pointers 16-byte aligned, strides a multiple of 16 bytes, else
 * STQ_ERR_LAYOUT. */
stq_status stq_qk_norm_rope(const stq_norm_desc* desc, const void* q_dev, const void* k_dev,
                            const float* q_weight_dev, const float* k_weight_dev, const int32_t* pos_dev,
                            const float* cos_sin_dev, void* q_out_dev, void* k_out_dev, hipStream_t stream);

/* Cache write: token t < n_tok of k_dev, v_dev ([n_kv_heads][d] contiguous,
 * tokens k_stride, v_stride elements apart, element type `type`) goes to token
 * slot slot_dev[t] in the format above.  Slots outside the cache (-1 of a
 * padded batch) are skipped; a slot must not be named twice in one call. */
stq_status stq_kv_store(const stq_kv_desc* desc, void* cache_dev, size_t bytes, const int64_t* slot_dev,
                        int32_t n_tok, const void* k_dev, const void* v_dev, int64_t k_stride, int64_t v_stride,
                        int32_t type, hipStream_t stream);

/* Read-back: the values the cache holds at the listed slots, exact in every
 * element type; k_out_dev, v_out_dev [n_tok][n_kv_heads][d] contiguous.
 * Rows of slots outside the cache are left as they were. */
stq_status stq_kv_fetch(const stq_kv_desc* desc, const void* cache_dev, size_t bytes, const int64_t* slot_dev,
                        int32_t n_tok, void* k_out_dev, void* v_out_dev, int32_t type, hipStream_t stream);

/* Attention over the cache.  Request i < n_req owns query tokens
 * tok_start[i] .. tok_start[i+1]-1; its cache (through its table row) holds
 * len[i] tokens, the last of which are its query tokens' own, so query j sits
 * at position p = len[i] - (tok_start[i+1] - tok_start[i]) + j.  It sees cached
 * position s when s <= p and (window == 0, or s > p - window, or s < n_sink).
 *   o = sum_s softmax_s(scale * q . k_s) v_s, query head h reading key/value
 *   head h / (n_heads / n_kv_heads); a query that sees nothing gets 0.
 *
 * One kernel and one split of the work serve a whole call, by max_new and
 * max_len.  Requests of one or a few new tokens therefore belong in a call of
 * their own, apart from prompts: with requests a .. b-1 side by side, the call
 * takes table + a * table_cols, tok_start + a, len + a, n_req = b - a and the
 * same q, o and n_tok.  (32 heads over 8, d = 128, a prompt of 2,048 tokens with
 * 63 requests of 2,048 to 8,191: 136 us in two calls, 270 in one; with 8 of
 * 32,768 to 131,072: 212 us, 2,690 in one.) */
typedef struct stq_attend_desc {
  int32_t n_req;            /* requests (>= 0)                                */
  int32_t n_tok;            /* rows of q and o, 0 .. 2^28 (a padded batch may   */
                            /* have more than tok_start[n_req]: left alone;   */
                            /* query tokens past n_tok have no row, but count */
                            /* for the others' positions)                     */
  int32_t n_heads;          /* a multiple of n_kv_heads                       */
  int32_t type;             /* of q and o: STQ_BF16 or STQ_FP16               */
  int32_t table_cols;       /* columns of the block table                     */
  int32_t max_new;          /* at least every request's query tokens: queries  */
                            /* past it are left alone                         */
  int32_t max_len;          /* about the longest len: sets the split of the    */
                            /* work, never the result                         */
  int32_t window, n_sink;   /* >= 0; window 0: none                           */
  float scale;              /* finite                                         */
  int64_t q_stride, o_stride;  /* elements between tokens ([n_heads][d] each)  */
} stq_attend_desc;

/* Bytes of the workspace a call with these descriptors needs (0: none). */
size_t stq_kv_attend_bytes(const stq_kv_desc* desc, const stq_attend_desc* a);

/* Lengths are taken as at most table_cols * block_tokens; blocks whose table
 * entry lies outside [0, n_blocks) hold no visible token.  q and o 16-byte
 * aligned with strides a multiple of 16 bytes, the workspace 16-byte aligned,
 * else STQ_ERR_LAYOUT.  STQ_ERR_UNSUPPORTED for calls larger than a launch:
 * n_req * max_new * n_heads from 2^31 on, or n_req * n_kv_heads (times the
 * query rows' tiles and the splits) from 2^24 on.  A workspace serves one call
 * at a time.  o may be q itself (same pointer and stride), else it must not
 * overlap q (STQ_ERR_ARG).  Products run on the matrix cores in binary16 (cached values and
 * queries exact, the queries scaled by a power of two per row; softmax
 * weights rounded to binary16, for bfloat16 outputs cut to it: off by 2^-10
 * of themselves, or by 2^-31 of the row's largest where they are below 2^-21
 * of it), sums and statistics in binary32. */
stq_status stq_kv_attend(const stq_kv_desc* desc, const void* cache_dev, size_t bytes, const stq_attend_desc* a,
                         const int32_t* table_dev, const int32_t* tok_start_dev, const int32_t* len_dev,
                         const void* q_dev, void* o_dev, void* work_dev, size_t work_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* STQ_H */
