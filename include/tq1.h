/*
 * tq1.h -- C ABI of libtq1: ternary TQ1_0 weights x Q8_1 activations, and the
 * decoder layer between such products (rotary positions, paged key/value
 * cache, attention), on NVIDIA GB300 (sm_103a).
 *
 * Formats (PrismML-Eng/llama.cpp issue #139, "Current behavior": five trits
 * per byte in base 3, chunk c of a 256-element block reading digit c of
 * qs[0..31]; the block specification that accompanies it fixes the rest):
 *
 *   TQ1_0 block, 54 bytes, 256 weights:
 *     bytes  0..47  qs[48]  five trits per byte
 *     bytes 48..51  qh[4]   four trits per byte
 *     bytes 52..53  d       fp16 scale, little-endian
 *   byte b holding trits u0..u4 (u in {0,1,2}, u0 most significant) is
 *   ceil((sum u_i 3^(4-i)) * 256 / 243); digit k of b is ((uint8)(b*3^k)*3)>>8;
 *   trit 0/1/2 means weight -d/0/+d.  Element e of a block is
 *     e <  160: qs[e % 32] digit e / 32
 *     e <  240: qs[32 + (e - 160) % 16] digit (e - 160) / 16
 *     e >= 240: qh[(e - 240) % 4] digit (e - 240) / 4
 *   A matrix of n rows and k columns (k % 256 == 0) is [n][k/256] blocks,
 *   rows contiguous.
 *
 *   Q8_1 block, 36 bytes, 32 activations: fp16 d @0, fp16 s @2, int8 q[32] @4.
 *   A [t][k] activation matrix is [t][k/32] blocks.
 *
 *   TQ2_0 block, 66 bytes, 256 weights (the 2-bit sibling format the same
 *   page names in "Upstream state" without a layout; this library's reading):
 *     bytes  0..63  qs[64]  four 2-bit codes per byte, code = trit + 1
 *     bytes 64..65  d       fp16 scale, little-endian
 *   Element e of a block is field (e/32) % 4 (bits 2f..2f+1) of byte
 *   qs[32 * (e/128) + e % 32]: chunk c reads one field of 32 consecutive
 *   bytes, the chunk pattern above with four codes per byte.  Code 3 is never
 *   written and decodes to +2*d.
 *
 * Conventions shared by every entry point:
 *   - All data pointers are DEVICE pointers owned by the caller and must be
 *     16-byte aligned (TQ1_ERR_ALIGN otherwise).  The library never
 *     synchronises and allocates no device memory; work is enqueued on
 *     `stream` (a cudaStream_t, NULL for the legacy default stream) on the
 *     current device.  Scratch, where a path needs any, is a caller-owned
 *     workspace with a size query (tq1_mmv_ws, tq1_mmv_id).
 *   - Arguments are checked on the host before anything is launched; a
 *     failed check returns its negative code and launches nothing.
 *   - Shapes: k must be a positive multiple of 256; n, t >= 0 (0 means there
 *     is nothing to do and TQ1_OK is returned).
 *   - Errors met while kernels run (a bulk-copy wait that timed out, a
 *     routing id out of range) set a device status word; tq1_sync_status()
 *     synchronises `stream` and returns and clears it.
 *   - Kernels are launched with programmatic dependent launch: the mat-vec
 *     kernels start streaming weight blocks before the previous kernel in the
 *     stream has finished, so weight blocks must not be written by a kernel
 *     that lets its dependents start early (tq1_quantize_rows does not).
 */
#ifndef TQ1_H_
#define TQ1_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

enum tq1_status {
  TQ1_OK = 0,
  TQ1_ERR_NULL = -1,        /* a required pointer is NULL */
  TQ1_ERR_SHAPE = -2,       /* k not a positive multiple of 256, or n/t/top_k negative */
  TQ1_ERR_ALIGN = -3,       /* a pointer is not 16-byte aligned */
  TQ1_ERR_UNSUPPORTED = -4, /* shape beyond the kernels' limits (e.g. k > 62720) */
  TQ1_ERR_WORKSPACE = -5,   /* workspace too small */
  TQ1_ERR_CUDA = -6,        /* a CUDA runtime call failed */
  TQ1_ERR_TIMEOUT = -7,     /* a kernel gave up waiting on a transfer (device status) */
  TQ1_ERR_BAD_ID = -8,      /* a routing, page or sequence id was out of range (device status) */
  TQ1_ERR_NO_PAGES = -9     /* no free pages, or no room in a page-table row (device status) */
};

/* Text for a status code (static storage).  No passage: a convention of this
 * library (the pages define no API). */
const char* tq1_status_string(int status);

/* Library version, e.g. "0.1.0".  No passage: a convention of this library. */
const char* tq1_version(void);

/*
 * Test hook for the error path of the bounded transfer waits.  The next
 * tq1_mmv / tq1_mmv_add / tq2_mmv / tq2_mmv_add call consumes the hook,
 * whichever kernel it runs; when that call runs the decode kernel
 * (1 <= t <= 5), its first CTA issues no copy (and no byte count) for its
 * first 4-row group, so every wait on that group gives up after about 2 s:
 * the call then reports TQ1_ERR_TIMEOUT through tq1_sync_status, its outputs
 * are unspecified, and the device and the library stay usable.  Nothing
 * faults, traps or hangs.  No passage: a convention of this library.
 */
void tq1_debug_inject_wait_timeout(void);

/* Name and text of the last CUDA runtime error this thread saw inside the
 * library (empty if none); explains a TQ1_ERR_CUDA.  No passage: a
 * convention of this library. */
const char* tq1_last_cuda_error(void);

/* Bytes of a TQ1_0 matrix [n][k/256], a TQ2_0 matrix [n][k/256] and a Q8_1
 * matrix [t][k/32] (54, 66 and 36 bytes per block, as the formats at the top
 * of this file lay them out).  No passage: a convention of this library. */
size_t tq1_blocks_bytes(int64_t n, int64_t k);
size_t tq2_blocks_bytes(int64_t n, int64_t k);
size_t tq1_q8_1_bytes(int64_t t, int64_t k);

/*
 * Quantise fp32 weights w[n][k] (row-major) to TQ1_0 blocks.
 * Per 256-weight block: d = fp16(max |w|); trit = clamp(round_half_away(w / max|w|),
 * -1, 1), or 0 when the block is all zero.  Bit-exact, deterministic.
 * Source: PrismML-Eng/llama.cpp issue #139, "Current behavior" (the block
 * format); the rounding is this library's reading (the pages do not state
 * one).
 */
int tq1_quantize_rows(const float* w, void* blocks, int64_t n, int64_t k, void* stream);

/*
 * Quantise fp32 activations x[t][k] to Q8_1 blocks q8[t][k/32].
 * Per 32-value block: d = max|x| / 127 (fp32); q = clamp(round_half_away(x / d),
 * -127, 127), or 0 when d == 0; stored fp16(d), fp16(d * sum q), q.
 * k must be a positive multiple of 32 here.  Bit-exact, deterministic.
 * Source: PrismML-Eng/llama.cpp issue #139, "Current behavior" (the Q8_1
 * activation blocks of 32 values whose per-block dot product the mat-vec
 * computes); the rounding is this library's reading (the pages do not state
 * one).
 */
int q8_1_quantize_acts(const float* x, void* q8, int64_t t, int64_t k, void* stream);

/*
 * Mat-vec for t token columns: y[c][r] = sum_k w[r][k] * x[c][k] with
 * w = d_w * trit and x = d_a * q, accumulated as
 *   sum_blocks d_w * sum_{chunks j} d_a[j] * I_j,   I_j = sum (trit * q) (exact int32)
 * in fp32.  blocks [n][k/256] TQ1_0, q8 [t][k/32] Q8_1, y fp32 [t][n].
 * The ladder: t <= 5 runs the byte-major dp4a decode kernel (rungs of
 * 1/2/4/8 columns); t >= 6 runs the warp-level tensor-core kernel (mma.sync
 * on exact fp16 operands, trit-derived and the int8 q, with an fp32
 * accumulation of each 32-element chunk that is exact) with rungs of
 * 8/16/24/32 token columns,
 * in slices of 32 columns above 32; shapes either cannot stage take a
 * general dp4a kernel.  Nothing
 * is allocated; for prefill-sized t, tq1_mmv_ws with a workspace runs the
 * tcgen05 tile path instead.  Deterministic: repeated calls give identical
 * bits.
 * Source: PrismML-Eng/llama.cpp issue #139, "Proposed approach" (a dedicated
 * whole-block kernel that iterates over packed bytes); laddered column
 * counts: Neroued/ninfer issue #293.
 */
int tq1_mmv(const void* blocks, const void* q8, float* y, int64_t n, int64_t k, int64_t t, void* stream);

/*
 * Workspace bytes tq1_mmv_ws / tq2_mmv_ws need for an n x k matrix and t
 * columns: the tcgen05 tile path's exact fp16 hi/lo split of the activations
 * (2 * 2 * t_pad * k + 4 * t_pad bytes, t_pad = t rounded up to the token
 * tile, rounded up to 256).  0 when the call takes the allocation-free
 * kernels (t below the tile path's threshold, or a row stride that is not a
 * multiple of 16 bytes, i.e. k not a multiple of 2048).
 * Source: PrismML-Eng/llama.cpp issue #139, "Measured impact" (prefill, pp512,
 * is the case the dense tensor-core path serves); the workspace itself is a
 * convention of this library.
 */
size_t tq1_mmv_workspace_size(int64_t n, int64_t k, int64_t t);

/*
 * tq1_mmv / tq1_mmv_add with a caller-owned workspace: where
 * tq1_mmv_workspace_size(n, k, t) > 0 (prefill-sized t), a prep kernel
 * splits the activations into exact fp16 hi/lo rows in `ws` and a tcgen05
 * kernel (A: the weights expanded straight into tensor memory; B: the hi/lo
 * rows by TMA; fp32 accumulators in tensor memory) contracts them; otherwise
 * the call equals tq1_mmv (res == NULL) or tq1_mmv_add.  res may be NULL or
 * y itself.  ws: device, 16-byte aligned, at least
 * tq1_mmv_workspace_size(n, k, t) bytes (TQ1_ERR_WORKSPACE otherwise; checked
 * before any launch), or NULL (then the allocation-free kernels run).  The
 * workspace is in use until the call's kernels finish on `stream`.
 * tq2_mmv_ws: the same for TQ2_0 weights.
 * Source: PrismML-Eng/llama.cpp issue #139, "Measured impact" and
 * "Proposed approach" (prefill through a dedicated whole-block kernel).
 */
int tq1_mmv_ws(const void* blocks, const void* q8, const float* res, float* y, int64_t n, int64_t k, int64_t t,
               void* ws, size_t ws_bytes, void* stream);
int tq2_mmv_ws(const void* blocks, const void* q8, const float* res, float* y, int64_t n, int64_t k, int64_t t,
               void* ws, size_t ws_bytes, void* stream);

/*
 * Decode mat-vec straight from fp32 activations: the Q8_1 quantisation of x
 * (the same operations and rounding as q8_1_quantize_acts) runs in the dp4a
 * decode kernel's prologue, so a decode step needs one launch per mat-vec
 * instead of two.  y equals, bit for bit, q8_1_quantize_acts followed by
 * tq1_mmv (the same decode kernel on the same records).  x: fp32 [t][k],
 * device, 16-byte aligned.  1 <= t <= 4 (larger t: TQ1_ERR_UNSUPPORTED; quantise
 * once and call tq1_mmv).  Errors as tq1_mmv.
 * Source: PrismML-Eng/llama.cpp issue #139, "Current behavior" (activations
 * are quantised to Q8_1 before the MMVQ kernel: here inside it).
 */
int tq1_mmv_f32(const void* blocks, const float* x, float* y, int64_t n, int64_t k, int64_t t, void* stream);

/*
 * Mat-vec with a residual added in the kernel's epilogue:
 *   y[c][r] = res[c][r] + sum_k w[r][k] * x[c][k]
 * (one fp32 add per output after the dot product; the same kernels, rungs and
 * accumulation as tq1_mmv).  res: fp32 [t][n], device, 16-byte aligned; it may
 * be y itself (in-place update).  Errors as tq1_mmv; res == NULL is
 * TQ1_ERR_NULL.
 * Source: Neroued/ninfer issue #293 (the linear_add rungs: a linear layer
 * fused with its residual add).
 */
int tq1_mmv_add(const void* blocks, const void* q8, const float* res, float* y, int64_t n, int64_t k, int64_t t,
                void* stream);

/*
 * Debug entry: the exact integer partials part[c][r][j] = I_j (int32,
 * [t][n][k/32]) that tq1_mmv scales, for any t, from the kernel tq1_mmv runs
 * for that t: the dp4a decode kernel at t <= 5 (its dp4a sums, stored before
 * scaling), the tensor-core rungs at t >= 6 (each chunk's accumulator, which
 * holds exactly I_j when the operands are unscaled); shapes neither can stage
 * take the general kernel.  Bit-exact by construction.
 * Source: PrismML-Eng/llama.cpp issue #139, "Acceptance criteria" (the new
 * kernel checked case by case against a CPU reference), and the per-32-block
 * integer dot product of "Current behavior" that the kernels compute.
 */
int tq1_mmv_partials(const void* blocks, const void* q8, int32_t* part, int64_t n, int64_t k, int64_t t,
                     void* stream);

/*
 * Dequantise TQ1_0 rows: out[r][j] = d_w(r, j/256) * trit(r, j), the value the
 * block encodes (fp32 when out_f16 == 0, else fp16; both exact, since the
 * scale is an fp16 value and the trit is -1, 0 or +1).
 *   blocks: [n][k/256] TQ1_0;  out: [n][k] fp32 or fp16, 16-byte aligned.
 * Source: PrismML-Eng/llama.cpp issue #139, "Current behavior" (the CPU
 * dequantize_row walk: each packed byte amortised over its trits, element
 * order of the block) and "Upstream state" (the dequant shader that ships with
 * the Vulkan mat-vec).
 */
int tq1_dequantize_rows(const void* blocks, void* out, int64_t n, int64_t k, int out_f16, void* stream);

/*
 * Gather dequantised rows (get_rows, e.g. an embedding lookup):
 * out[i][:] = row row_ids[i] of the n x k TQ1_0 matrix, i < n_ids, fp32 or
 * fp16 as in tq1_dequantize_rows.  An id outside [0, n) leaves its output row
 * untouched and sets TQ1_ERR_BAD_ID in the device status (tq1_sync_status).
 *   row_ids: int32 [n_ids] (device);  out: [n_ids][k].
 * Source: PrismML-Eng/llama.cpp issue #139, "Upstream state" (get_rows for the
 * format next to its mat-vec).
 */
int tq1_get_rows(const void* blocks, const int32_t* row_ids, int64_t n_ids, void* out, int64_t n, int64_t k,
                 int out_f16, void* stream);

/*
 * Workspace bytes tq1_mmv_id needs for n_experts experts and t*top_k routed
 * pairs (the compacted routing table: n_active, expert bounds, active
 * experts, sorted pairs, task offsets).  Small routings (four words per
 * expert plus one per pair within 16 KiB) build the table inside the routed
 * kernel and leave the workspace untouched; it is required all the same.
 * Source: AMD-Ecosystem/llama.cpp PR #76, "Summary" (ids -> expert_bounds ->
 * compacted grid: the table this workspace holds).
 */
size_t tq1_mmv_id_workspace_size(int64_t n_experts, int64_t t, int64_t top_k);

/*
 * Expert-routed mat-vec (MoE "mul_mat_id"): y[c][s][r] = expert ids[c][s]'s
 * matrix times token c's activations, for every token c < t and slot s < top_k.
 *   expert_blocks: n_experts matrices [n][k/256] back to back (expert e starts
 *                  at byte e * tq1_blocks_bytes(n, k))
 *   q8:            [t][k/32] Q8_1, one row per token (shared by its slots)
 *   ids:           int32 [t][top_k] expert ids
 *   y:             fp32 [t][top_k][n]
 *   ws, ws_bytes:  caller-owned device workspace of at least
 *                  tq1_mmv_id_workspace_size() bytes (TQ1_ERR_WORKSPACE otherwise);
 *                  it holds the compacted routing table between the two launches.
 * Ids outside [0, n_experts) skip their slot (its output is left untouched) and
 * set TQ1_ERR_BAD_ID in the device status.  n_experts <= 12288.
 * Source: AMD-Ecosystem/llama.cpp PR #76, "Summary" (ids -> expert_bounds ->
 * compacted grid); PrismML-Eng/llama.cpp issue #139, "Acceptance criteria"
 * (MUL_MAT_ID with fewer experts used than available).
 */
int tq1_mmv_id(const void* expert_blocks, int64_t n_experts, const void* q8, const int32_t* ids, float* y,
               int64_t n, int64_t k, int64_t t, int64_t top_k, void* ws, size_t ws_bytes, void* stream);

/*
 * Expert-routed mat-vec with one activation row per routed (token, slot) pair
 * (the down-projection of an expert layer, whose input differs per slot):
 *   y[c][s][r] = expert ids[c][s]'s matrix times activation row (c, s).
 *   q8: [t][top_k][k/32] Q8_1.  Everything else, including the workspace and
 * the error behaviour, as tq1_mmv_id.
 * Source: PrismML-Eng/llama.cpp issue #139, "Acceptance criteria" (MUL_MAT_ID
 * cases); AMD-Ecosystem/llama.cpp PR #76, "Summary" (ids -> expert bounds ->
 * compacted grid).
 */
int tq1_mmv_id_slots(const void* expert_blocks, int64_t n_experts, const void* q8, const int32_t* ids, float* y,
                     int64_t n, int64_t k, int64_t t, int64_t top_k, void* ws, size_t ws_bytes, void* stream);

/*
 * Debug entry: the exact integer partials part[c][s][r][j] = I_j (int32,
 * [t][top_k][n][k/32]) that tq1_mmv_id / tq2_mmv_id scale, from the routed
 * decode kernels themselves (their expansion and dp4a sums, stored before
 * scaling): direct mode for up to 128 routed pairs, the compacted mode above.
 * Arguments, workspace and errors as tq1_mmv_id (part replaces y); shapes
 * that only the general kernel can stage return TQ1_ERR_UNSUPPORTED.
 * Source: AMD-Ecosystem/llama.cpp PR #76, "Summary" (the expert-routed grid
 * these kernels run); PrismML-Eng/llama.cpp issue #139, "Acceptance criteria"
 * (MUL_MAT_ID checked against a CPU reference).
 */
int tq1_mmv_id_partials(const void* expert_blocks, int64_t n_experts, const void* q8, const int32_t* ids,
                        int32_t* part, int64_t n, int64_t k, int64_t t, int64_t top_k, void* ws, size_t ws_bytes,
                        void* stream);
int tq2_mmv_id_partials(const void* expert_blocks, int64_t n_experts, const void* q8, const int32_t* ids,
                        int32_t* part, int64_t n, int64_t k, int64_t t, int64_t top_k, void* ws, size_t ws_bytes,
                        void* stream);

/*
 * tq1_mmv_id without a workspace argument, for callers that cannot allocate
 * device memory (inside a stream capture, under a fixed memory budget, in a
 * latency-critical loop, or from plain C with no allocator at hand).  The
 * routing table lives in a fixed array that is part of the library image
 * (about 76 KiB on every GPU that loads the library, held until exit).
 * Limits: n_experts <= 1024 and t * top_k <= 16384; larger calls return
 * TQ1_ERR_WORKSPACE and launch nothing.  Same arguments, layouts, results
 * and errors as tq1_mmv_id otherwise.
 * The first call on a device looks up the array's device address with that
 * device current; make that first call before any stream capture begins.
 * All calls on a device share the array (each call rewrites what it reads,
 * so nothing needs clearing); calls that may overlap on the GPU race on it.
 * No passage: a convention of this library (the pages have no counterpart
 * to this entry point).
 */
int tq1_mmv_id_noalloc(const void* expert_blocks, int64_t n_experts, const void* q8, const int32_t* ids, float* y,
                       int64_t n, int64_t k, int64_t t, int64_t top_k, void* stream);

/*
 * Synchronise `stream`, then return and clear the device status word:
 * TQ1_OK, TQ1_ERR_TIMEOUT, TQ1_ERR_BAD_ID or TQ1_ERR_NO_PAGES, the first of
 * them that was raised in this order (or TQ1_ERR_CUDA if the stream itself
 * reported an error).  No passage: a convention of this library (the
 * pages define no error reporting).
 */
int tq1_sync_status(void* stream);

/*
 * TQ2_0 weights (2-bit codes; format at the top of this file).
 *
 * tq2_quantize_rows: fp32 w[n][k] -> TQ2_0 blocks, with the same scale and
 * trit rounding as tq1_quantize_rows (so both formats hold the same trits and
 * scales for the same weights).  Bit-exact, deterministic.
 *
 * tq2_mmv: y[c][r] = sum_k w[r][k] * x[c][k] for TQ2_0 blocks [n][k/256] and
 * Q8_1 q8 [t][k/32], accumulated exactly as tq1_mmv (exact int32 per-32
 * partials, fp32 scale-and-sum per block).  The same ladder as tq1_mmv:
 * t <= 5 runs the decode kernel (the codes already are its packed-digit
 * registers: masked dp4a, no expansion), t >= 6 the warp-level tensor-core
 * rungs (the codes become fp16 operands by a byte permute), with the
 * tcgen05 tile path through tq2_mmv_ws.  Deterministic; allocates nothing.
 *
 * tq2_mmv_partials: the exact int32 partials part[c][r][k/32] of tq2_mmv
 * (debug, as tq1_mmv_partials).
 *
 * Arguments, alignment, shapes and errors as the TQ1_0 counterparts.
 * Source: PrismML-Eng/llama.cpp issue #139, "Upstream state" (TQ2_0 as the
 * stalled sibling of the TQ1_0 port) and "Proposed approach" (whole-block
 * kernels that load each packed byte once).
 */
int tq2_quantize_rows(const float* w, void* blocks, int64_t n, int64_t k, void* stream);
int tq2_mmv(const void* blocks, const void* q8, float* y, int64_t n, int64_t k, int64_t t, void* stream);
int tq2_mmv_partials(const void* blocks, const void* q8, int32_t* part, int64_t n, int64_t k, int64_t t,
                     void* stream);

/*
 * TQ2_0 counterparts of tq1_mmv_f32 (Q8_1 quantisation fused into the decode
 * kernel's prologue, 1 <= t <= 4, bit-identical to q8_1_quantize_acts +
 * tq2_mmv) and tq1_mmv_add (y = res + W x, res may be y).  Arguments and
 * errors as those.
 * Source: as tq1_mmv_f32 and tq1_mmv_add, with PrismML-Eng/llama.cpp issue
 * #139, "Upstream state" (the TQ2_0 sibling format).
 */
int tq2_mmv_f32(const void* blocks, const float* x, float* y, int64_t n, int64_t k, int64_t t, void* stream);
int tq2_mmv_add(const void* blocks, const void* q8, const float* res, float* y, int64_t n, int64_t k, int64_t t,
                void* stream);

/*
 * TQ2_0 rows to fp32 (out_f16 == 0) or fp16 values, d * (code - 1) exactly:
 * the whole matrix (tq2_dequantize_rows) or the rows listed in row_ids
 * (tq2_get_rows).  Arguments, layouts, errors and the handling of
 * out-of-range ids as tq1_dequantize_rows / tq1_get_rows.
 * Source: PrismML-Eng/llama.cpp issue #139, "Upstream state" (the TQ2_0
 * sibling format) and "Current behavior" (the dequantise walk of a block).
 */
int tq2_dequantize_rows(const void* blocks, void* out, int64_t n, int64_t k, int out_f16, void* stream);
int tq2_get_rows(const void* blocks, const int32_t* row_ids, int64_t n_ids, void* out, int64_t n, int64_t k,
                 int out_f16, void* stream);

/*
 * Expert-routed mat-vec over TQ2_0 experts (each expert [n][k/256] x 66
 * bytes, back to back): the same routing, workspace
 * (tq1_mmv_id_workspace_size), kernels, layouts and errors as tq1_mmv_id
 * (one activation row per token) and tq1_mmv_id_slots (one per token and
 * slot).
 * Source: AMD-Ecosystem/llama.cpp PR #76, "Summary" (ids -> expert_bounds ->
 * compacted grid); PrismML-Eng/llama.cpp issue #139, "Upstream state" (the
 * TQ2_0 sibling format).
 */
int tq2_mmv_id(const void* expert_blocks, int64_t n_experts, const void* q8, const int32_t* ids, float* y,
               int64_t n, int64_t k, int64_t t, int64_t top_k, void* ws, size_t ws_bytes, void* stream);
int tq2_mmv_id_slots(const void* expert_blocks, int64_t n_experts, const void* q8, const int32_t* ids, float* y,
                     int64_t n, int64_t k, int64_t t, int64_t top_k, void* ws, size_t ws_bytes, void* stream);

/* ------------------------------------------------------------------------
 * The decoder layer between the projections: rotary positions, a paged
 * key/value cache, the attention that reads it, and its page bookkeeping.
 * A layer's step is: tq1_mmv (q, k, v) -> tq1_rope_append -> tq1_paged_attn
 * (fp32 output) -> q8_1_quantize_acts -> tq1_mmv_add (output projection).
 *
 * The cache keeps keys and values in pages of page_size slots (one slot per
 * token and kv head, head_dim 16-bit elements).  Page p, kv head h, slot s
 * starts at element p * page_stride + h * head_stride + s * slot_stride of k
 * and of v; only the head_dim elements of a slot have to be contiguous.
 * Slot j of sequence s (its token at position j) is slot j % page_size of
 * page page_table[s][j / page_size].
 *
 * Conventions beside those at the top of this file:
 *   - page_table, q_start, kv_len and the other index arrays are int32 in
 *     device memory (4-byte aligned; refs 16-byte) and are read when the
 *     kernels run.  Whatever they hold, no kernel leaves the tensors of the
 *     call: lengths are cut to what the page table addresses, and a page or
 *     sequence id out of range is skipped and sets TQ1_ERR_BAD_ID in the
 *     device status.
 *   - The structs are read during the call only; the caller may reuse them.
 *   - Strides are multiples of 8 elements (16 bytes), page_size is 16, 32,
 *     64, 128 or 256, head_dim a multiple of 8 up to 256; n_seqs <= 8192,
 *     max_pages <= 2^20, t <= 2^24.
 * ------------------------------------------------------------------------ */
enum tq1_dtype { TQ1_F32 = 0, TQ1_F16 = 1, TQ1_BF16 = 2 };

typedef struct tq1_kv_cache {
  void* k;              /* 16-byte aligned */
  void* v;
  int64_t n_pages, n_kv, page_size, head_dim;
  int64_t page_stride, head_stride, slot_stride; /* elements */
  int32_t dtype;        /* TQ1_F16 or TQ1_BF16 */
} tq1_kv_cache;

/* A batch of sequences: sequence s has the call's tokens q_start[s] ..
 * q_start[s + 1] - 1 (none is fine) and kv_len[s] tokens in all, these
 * included; so its token i stands at position kv_len[s] - (q_start[s + 1] -
 * i).  Tokens from q_start[n_seqs] on belong to no sequence and are left
 * alone.  Where q_start does not ascend and sequences share tokens, attention
 * may do nothing and set TQ1_ERR_BAD_ID. */
typedef struct tq1_kv_batch {
  const int32_t* page_table; /* [n_seqs][max_pages] */
  const int32_t* q_start;    /* [n_seqs + 1], ascending */
  const int32_t* kv_len;     /* [n_seqs] */
  int64_t n_seqs, max_pages;
} tq1_kv_batch;

/* The pools of a cache (e.g. the keys and the values of every layer) that
 * share one set of tables: pool i's page p is the page_bytes bytes at base +
 * i * pool_stride + p * page_bytes (both multiples of 16).  refs[p] is how
 * many sequences hold page p; a page is free exactly when it is 0. */
typedef struct tq1_page_pool {
  void* base;
  int64_t n_pools, pool_stride, page_bytes, n_pages;
  int32_t* refs;        /* [n_pages] */
  int32_t* page_table;  /* [n_seqs][max_pages], -1 where there is no page */
  int32_t* kv_len;      /* [n_seqs], 0: the sequence is empty */
  int64_t n_seqs, max_pages, page_size;
} tq1_page_pool;

/*
 * Inverse frequencies of rotary positions, inv_freq[i] for the rot_dim / 2
 * rotated pairs: theta_i ((1 - g) / factor + g), theta_i = base^(-2i/rot_dim).
 * factor == 1 gives theta_i.  For contexts `factor` times longer than the
 * orig_len positions a model was trained on, g ramps from 0 (stretched by the
 * factor) to 1 (kept) as the turns orig_len theta_i / 2 pi of a pair go from
 * `low` to `high`; low = high = INFINITY stretches all pairs alike.  (The ramp
 * is linear in the turns.  A model whose ramp is linear in the pair's index
 * between two indexes wants other numbers: fill inv_freq with them instead;
 * tq1_rope_append takes any table.)  fp64, rounded once.  inv_freq: fp32 [rot_dim / 2], device; rot_dim even, <= 256.
 * No passage: a convention of this library.
 */
int tq1_rope_freqs(float* inv_freq, int64_t rot_dim, double base, double factor, double orig_len, double low,
                   double high, void* stream);

/*
 * Rotary positions and cache append.  For every token of the batch: the first
 * rot_dim elements of each q and k head turn by the token's position, the
 * rotated q goes to q_out, the rotated k and the v to the token's cache slot.
 * Pair i, (x, y) = elements (i, i + rot_dim/2), or (2i, 2i + 1) when
 * interleaved != 0, becomes mscale * (x cos a - y sin a, x sin a + y cos a)
 * with a = position * inv_freq[i] (formed in fp64); elements from rot_dim on
 * are copied.  rot_dim is a multiple of 8, 0 <= rot_dim <= head_dim.
 *   q: [t][n_q][head_dim], k and v: [t][n_kv][head_dim], all of type in_dtype
 *      (TQ1_F32, TQ1_F16 or TQ1_BF16), tokens ldq / ldk / ldv elements apart
 *      (multiples of 4): column ranges of one fused projection will do
 *   q_out: [t][n_q][head_dim] of the cache's type, contiguous
 *   positions: int32 [t] (device) to turn by instead of the tokens' positions
 *      in their sequences, or NULL; the slots stay the sequences'
 * Values are rounded once, to the cache's type.  A token whose slot is outside
 * its page-table row, or in no valid page, is not appended (its q row is
 * written) and sets TQ1_ERR_BAD_ID.
 * No passage: a convention of this library.
 */
int tq1_rope_append(const tq1_kv_cache* cache, const tq1_kv_batch* batch, const void* q, int64_t ldq, const void* k,
                    int64_t ldk, const void* v, int64_t ldv, int in_dtype, void* q_out, int64_t t, int64_t n_q,
                    const float* inv_freq, int64_t rot_dim, int interleaved, float mscale, const int32_t* positions,
                    void* stream);

/* Workspace bytes for tq1_paged_attn on t tokens of n_seqs sequences with n_q
 * query heads (0: invalid arguments).  What t tokens need depends on how they
 * are spread over sequences; the bytes returned serve any spread, and fewer
 * tokens too: a workspace for a server's largest t serves all its batches.
 * No passage: a convention of this library. */
size_t tq1_paged_attn_workspace_size(const tq1_kv_cache* cache, int64_t t, int64_t n_q, int64_t n_seqs);

/*
 * Attention of the batch's tokens over their sequences' pages:
 *   out[i][h] = sum_j p_j V[j],  p = softmax over the visible j of scale * q[i][h] . K[j]
 * with K, V of kv head h / (n_q / n_kv).  Visible to the token at position p
 * are the slots j < kv_len with j <= p (causal != 0) and j > p - window
 * (window > 0).  A row that sees nothing is 0.  One call serves decode steps
 * (one token per sequence), prompt chunks and any mix of them.  (The kernel is
 * chosen by the average sequence's rows, t * n_q / n_kv / n_seqs: a long chunk
 * runs faster in a call of its own than with hundreds of steps, and in a batch
 * without the sequences that have no new tokens.)
 *   q: [t][n_q][head_dim] of the cache's type, tokens ldq elements apart
 *   out: [t][n_q][head_dim] of the cache's type, or fp32 when out_f32 != 0
 *      (what q8_1_quantize_acts takes), tokens ldo elements apart; rows of
 *      tokens that belong to no sequence are left alone
 *   ws: device, 16-byte aligned, tq1_paged_attn_workspace_size() bytes
 *      (TQ1_ERR_WORKSPACE otherwise), in use until the call's kernels finish
 * Scores, maxima, sums and outputs are accumulated in fp32; the weights p
 * enter the second product as 16-bit numbers of the cache's type.  Slots at
 * or past kv_len, and slots before the window of a sequence's first new token,
 * may hold anything, NaN included, and the table entries of pages that have no
 * other slots are not read (a cache may free what its window has passed).
 * Keys that are not finite hurt only the rows that see them; values that are
 * not finite, in a chunk of several tokens, also rows of nearby tokens that do
 * not see them (a weight of zero does not silence them).
 * Deterministic.  head_dim 64 or 128, n_q a multiple of n_kv, at most 128
 * query heads per kv head, t * n_q / n_kv <= 2^30 (TQ1_ERR_UNSUPPORTED
 * otherwise); scale > 0; ldq, ldo multiples of 8.
 * No passage: a convention of this library.
 */
int tq1_paged_attn(const tq1_kv_cache* cache, const tq1_kv_batch* batch, const void* q, int64_t ldq, int64_t t,
                   int64_t n_q, float scale, int causal, int64_t window, void* out, int64_t ldo, int out_f32, void* ws,
                   size_t ws_bytes, void* stream);

/* Workspace bytes of tq1_pages_resize, _fork and _compact on this pool (0:
 * invalid arguments).  No passage: a convention of this library. */
size_t tq1_pages_workspace_size(const tq1_page_pool* pool);

/*
 * Copy pages src[i] -> dst[i], i < n, in every pool.  No destination may be a
 * source or occur twice (the copies run in no order); tables and counts are
 * left alone.  No passage: a convention of this library.
 */
int tq1_pages_copy(const tq1_page_pool* pool, const int32_t* src, const int32_t* dst, int64_t n, void* stream);

/*
 * Set the length of sequences seqs[i] (distinct) to new_len[i], i < n <=
 * n_seqs.  First all that shrink let their pages past the new length go (new
 * length 0 frees a sequence).  Then those that grow get the lowest free
 * pages, in the order of the arguments; one whose last page is partly filled
 * and held by other sequences too first gets a copy of that page for itself
 * (free pages and holders as they stand when all shrinking is done).  From
 * the first sequence on that the free pages do not suffice for, none grows;
 * these keep their length and TQ1_ERR_NO_PAGES is set, as it is for a length
 * that is negative or beyond max_pages.  New slots hold whatever their pages
 * held.  No passage: a convention of this library.
 */
int tq1_pages_resize(const tq1_page_pool* pool, const int32_t* seqs, const int32_t* new_len, int64_t n, void* ws,
                     size_t ws_bytes, void* stream);

/*
 * Fork: children[i] (distinct, empty) become copies of parents[i], i < n <=
 * n_seqs (a parent may occur several times, but not as a child).  Full pages
 * are shared; a partly filled last page is copied to the lowest free one, in
 * the order of the arguments.  A child that is not empty is skipped and sets
 * TQ1_ERR_BAD_ID; children from the first one on that there is no page for
 * stay empty and TQ1_ERR_NO_PAGES is set.
 * No passage: a convention of this library.
 */
int tq1_pages_fork(const tq1_page_pool* pool, const int32_t* parents, const int32_t* children, int64_t n, void* ws,
                   size_t ws_bytes, void* stream);

/*
 * Compact: with L pages in use, the j-th page in use at or past L moves to
 * the j-th free page below L, so that afterwards exactly pages 0 .. L-1 are
 * in use; tables and counts follow.
 * No passage: a convention of this library.
 */
int tq1_pages_compact(const tq1_page_pool* pool, void* ws, size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* TQ1_H_ */
