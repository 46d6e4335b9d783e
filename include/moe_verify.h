/*
 * moe_verify.h -- C ABI of the MoE layer of a speculative-decoding verify round,
 * on one NVIDIA GB300 (sm_103a).
 *
 * The layer (sources: "How AlphaInfer makes local decoding fast", sections 2 and 3.1:
 * a decode round over 1..16 token rows replayed as one captured graph with
 * per-request data as ingress buffers, where every extra verified row can route to
 * experts the other rows did not need and so adds weight bytes; "infero", the
 * decoder-block diagram and Design notes: a SwiGLU expert FFN silu(W_g x) * (W_u x)
 * -> W_d, weights consumed in 32-element block encoding, block scales folded in in
 * float; a dedicated top-k routing kernel at decode):
 *
 *   1. logits[r][e] = Wr[e] . x[r]                  fp32, fixed summation order (*)
 *   2. per row: the k largest logits, ordered by (logit desc, id asc);
 *      w_j = exp(l_j - l_1) / sum_i exp(l_i - l_1)   (softmax renormalised over the k)
 *   3. U = ascending distinct ids over all rows (each routed expert's weights are
 *      streamed once per call, however many rows picked it)
 *   4. per (row, routed expert): h = silu(Wg x) * (Wu x), silu(t) = t / (1 + e^-t)
 *   5. out[r] = sum_j w_j * (Wd h_{r,j})            (j in rank order)
 * Expert weights are int4 codes q in [-8, 7] with one fp16 scale per 32 codes;
 * weight = scale * q.  Activations in are bf16; everything after is fp32.
 *
 * (*) The router summation order is part of the definition so that the top-k
 * decision is reproducible bit for bit: 32 lane partials, lane l takes elements
 * 128c + 4l + j (c ascending, j = 0..3), each with one correctly rounded fma; the
 * partials are combined by p_l <- p_l + p_{l^o} for o = 16, 8, 4, 2, 1; logit = p_0.
 *
 * Conventions for every call below:
 *   - Device pointers are caller-owned device memory, 16-byte aligned (256 recommended).
 *     The library never frees caller memory.  Host pointers are plain host memory.
 *   - `stream` is a cudaStream_t (NULL = the legacy default stream).  Compute calls are
 *     asynchronous on that stream and return only argument/launch status; errors a
 *     kernel finds (a bounded wait that gave up) are read with moe_last_device_status.
 *   - Return codes: MOE_OK, or a negative MOE_E* code; moe_strerror names it.
 *   - Rows are independent: a row's outputs do not depend on which other rows share
 *     the call or on its position among them (bitwise).
 *   - Activations must be finite with |x| < 2^40 (and so must the SwiGLU output h);
 *     beyond that range results are undefined.
 *   - Rounds of fewer than 13 rows evaluate each 32-element block dot of steps 4 and 5
 *     exactly in integers, from the block's codes and its activations in block fixed
 *     point (x: 16 bits relative to the block's largest |x|; h: 23 bits), then scale it
 *     in fp32; the rounding of the smaller activations of a block (at most 2^-15 and
 *     2^-22 of the block's largest) stays within the stated output tolerance.  Wider
 *     rounds use bf16 x (exact) and h split into bf16 hi + lo on the tensor cores.
 *   - Every contribution to a row's output (rounds of fewer than 13 rows: one expert
 *     and 32-element slice of the intermediate dimension; wider rounds: one expert and
 *     chunk of up to 768 intermediate elements) is added as round(y * 2^32) into 64-bit
 *     integer accumulators, so the sum is exact and independent of the order of the
 *     adds; every such contribution and every output must stay below 2^31 in magnitude
 *     (beyond that results are undefined).
 */
#ifndef MOE_VERIFY_H
#define MOE_VERIFY_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

enum {
  MOE_OK = 0,
  MOE_EINVAL = -1,       /* bad dimensions, NULL or misaligned pointer, rows out of range */
  MOE_ECUDA = -2,        /* a CUDA runtime call failed (no device, launch failure, ...) */
  MOE_EWORKSPACE = -3,   /* workspace smaller than moe_workspace_bytes() */
  MOE_ETIMEOUT = -4,     /* a device-side bounded wait gave up (moe_last_device_status) */
  MOE_EUNSUPPORTED = -5  /* valid dimensions this build does not handle (see moe_create) */
};

/* which matrix set a packing call refers to */
enum { MOE_GATEUP = 0, MOE_DOWN = 1 };

/* Layer dimensions.  hidden H, n_experts E, top_k k, inter I (expert intermediate),
 * max_rows = the largest row count any call on this handle will pass. */
typedef struct moe_dims {
  int32_t hidden, n_experts, top_k, inter, max_rows;
} moe_dims;

/* One layer's weights, all DEVICE pointers in the packed layout of moe_pack_q4:
 *   router        fp32 [E][H] row-major
 *   gateup_nib    E * moe_packed_bytes(MOE_GATEUP, 0) bytes
 *   gateup_scale  E * moe_packed_bytes(MOE_GATEUP, 1) bytes of fp16 bits
 *   down_nib      E * moe_packed_bytes(MOE_DOWN, 0) bytes
 *   down_scale    E * moe_packed_bytes(MOE_DOWN, 1) bytes of fp16 bits          */
typedef struct moe_layer_w {
  const float* router;
  const uint8_t* gateup_nib;
  const uint16_t* gateup_scale;
  const uint8_t* down_nib;
  const uint16_t* down_scale;
  /* Expert -> slot indirection (AlphaInfer docs, section 2: "which expert lives where"
   * is per-round ingress data written into fixed buffers; section 5.1: one shared slot
   * bank across layers).  NULL: expert e's packed weights are entry e of the four
   * arrays above (as moe_pack_q4 writes them for a layer).  Otherwise a DEVICE int32
   * array [n_experts]: expert e's weights are entry slot_of_expert[e] of a bank of
   * n_slots entries that the four pointers address (one moe_pack_q4 entry per slot;
   * several layers may share one bank).  The kernel reads the table during the call,
   * so a captured round (moe_round with use_graph) picks up new table contents
   * without being rebuilt.  A slot outside [0, n_slots) is not read: the layer
   * computes with slot 0 instead and moe_last_device_status returns MOE_EINVAL. */
  const int32_t* slot_of_expert;
  int32_t n_slots;
} moe_layer_w;

typedef struct moe_handle moe_handle;

/* Validates dims and binds a handle to `device` (queries its SM count, allocates a
 * 4-byte device status word -- the only device allocation the library makes).
 * Supported: hidden a multiple of 256 in [256, 2048], inter a multiple of 256 in
 * [256, 4096], 1 <= top_k <= min(n_experts, 32), n_experts <= 512, 1 <= max_rows <= 32
 * (and the shared-memory plan must fit one SM).
 * MOE_EINVAL for dims that make no sense, MOE_EUNSUPPORTED for sizes outside those
 * ranges, MOE_ECUDA if the device cannot be used.  *out is NULL on failure. */
int moe_create(const moe_dims* dims, int device, moe_handle** out);
void moe_destroy(moe_handle* h);

/* Device workspace (bytes) a call with `rows` rows needs: barrier words, router logits,
 * the SwiGLU outputs exchanged between CTAs by the tensor-core path and the output
 * accumulators (2 x 8 copies x rows x H int64; the tensor-core path uses one copy).  It depends only on
 * the dimensions and the row count, so it takes the dimensions rather than a handle and
 * can be sized before any handle exists.  0 for invalid dims/rows. */
size_t moe_workspace_bytes(const moe_dims* dims, int32_t rows);

/* Packed size of ONE expert: part 0 = code bytes, part 1 = scale bytes (codes and scales
 * are separate device arrays, so each has its own size).  0 if invalid. */
size_t moe_packed_bytes(const moe_dims* dims, int which, int part);

/* Host-side packer (HOST buffers).  Packs n_experts consecutive experts:
 *   MOE_GATEUP: q_a = gate codes [n][I][H], s_a = gate scales [n][I][H/32],
 *               q_b = up codes [n][I][H],   s_b = up scales [n][I][H/32]
 *   MOE_DOWN:   q_a = down codes [n][H][I], s_a = down scales [n][H][I/32]; q_b, s_b unused
 * into nib_out / scale_out (n * moe_packed_bytes(which, 0 / 1) bytes).  Codes outside
 * [-8, 7] give MOE_EINVAL.  Layout (32-element blocks, code q stored as the nibble
 * q + 8, element 2t in the low nibble of byte t of its block):
 *   gate/up codes  [E][I][2: gate, up][H/32 blocks][16 B]   (intermediate row i of an
 *   gate/up scales [E][I][2][H/32]                           expert: gate, then up)
 *   down codes     [E][I/32 blocks][H rows][16 B]            (block-major: block b of all
 *   down scales    [E][I/32][H]                               H output rows is one run)
 * where, within each gate/up row, the code block and the scale of logical block b are
 * stored at position b ^ (i & 7) (i the row's intermediate index; gate and up alike).
 * Down block b of output row o is at b * H + o. */
int moe_pack_q4(const moe_dims* dims, int which, int32_t n_experts, const int8_t* q_a,
                const uint16_t* s_a, const int8_t* q_b, const uint16_t* s_b, uint8_t* nib_out,
                uint16_t* scale_out);

/* Steps 1-3 only (router GEMV, top-k + renormalised weights, union).
 * x_bf16 [rows][H] device; topk_ids [rows][k] int32 (rank order), topk_w [rows][k]
 * fp32, union_ids [E] int32 (first *n_union valid, ascending), n_union: device int32.
 * Any of the four outputs may be NULL.  ws: device workspace of ws_bytes. */
int moe_route(moe_handle* h, const moe_layer_w* w, const uint16_t* x_bf16, int32_t rows,
              int32_t* topk_ids, float* topk_w, int32_t* union_ids, int32_t* n_union, void* ws,
              size_t ws_bytes, void* stream);

/* Steps 1-5 for one layer.  x_bf16 [rows][H] device, out [rows][H] fp32 device. */
int moe_decode_layer(moe_handle* h, const moe_layer_w* w, const uint16_t* x_bf16, int32_t rows,
                     float* out, void* ws, size_t ws_bytes, void* stream);

/* A round over an L-layer stack, layer after layer in stream order (layer l+1's
 * routing starts only after layer l's output is complete).  layers: HOST array [L] of
 * device weight sets; x_bf16 [L][rows][H] device (layer l reads its own rows);
 * out [L][rows][H] fp32 device; stats: device int32 [L] receiving |U| per layer, or
 * NULL.  use_graph != 0 captures the round once per (handle, argument set) into a
 * CUDA graph and replays it on later calls with the same arguments; the buffers
 * are ingress: write new rows into the same x buffer and call again.  use_graph
 * needs a non-default stream. */
int moe_round(moe_handle* h, const moe_layer_w* layers, int32_t L, const uint16_t* x_bf16,
              int32_t rows, float* out, int32_t* stats, void* ws, size_t ws_bytes, int use_graph,
              void* stream);

/* moe_round with the rows in and the outputs out in HOST memory: on `stream`, in this
 * order, the copy of x_host into x_dev, the round (moe_round on x_dev / out_dev), and the
 * copy of out_dev into out_host -- what a caller holding the draft rows on the host runs
 * once per verify round (AlphaInfer docs §2: the round's rows are ingress into one
 * captured round).
 *   - dims: the dims the handle was created with (the copies move L * rows * hidden
 *     elements); call with the handle's device current.
 *   - x_host [L][rows][H] bf16 bits and out_host [L][rows][H] fp32, host memory owned
 *     by the caller.  Page-locked memory makes both copies asynchronous; with pageable
 *     memory the calling thread waits for each copy.
 *   - x_dev [L][rows][H] and out_dev [L][rows][H]: the caller's device staging buffers
 *     (16-byte aligned); they are moe_round's x_bf16 and out, so with use_graph the
 *     round replays while they, ws and stream stay the same.
 *   - stats, ws, ws_bytes, use_graph, stream: as for moe_round.
 *   - sync != 0: returns after the stream has finished, with out_host written, and with
 *     moe_last_device_status's answer (MOE_ETIMEOUT or MOE_EINVAL if the kernel raised
 *     one, the status word cleared).  sync == 0: returns once the work is enqueued; the
 *     caller synchronizes the stream before reading out_host and may read the status
 *     with moe_last_device_status.
 * Allocates nothing.  Nothing is enqueued when an argument is wrong: MOE_EINVAL for a
 * NULL handle, dims, layers or buffer, L outside [1, 128] or rows outside [1, max_rows],
 * moe_create's code for dims it would reject.  Otherwise moe_round's codes for the
 * round (the rows' copy is then already enqueued) and MOE_ECUDA if a copy fails. */
int moe_round_host(moe_handle* h, const moe_dims* dims, const moe_layer_w* layers, int32_t L,
                   const uint16_t* x_host, int32_t rows, float* out_host, uint16_t* x_dev,
                   float* out_dev, int32_t* stats, void* ws, size_t ws_bytes, int use_graph, int sync,
                   void* stream);

/* Prefill-width layer: steps 1-5 for many token rows at once (a prompt's tokens), the
 * infero README's MoE prefill path ("Beyond plain text decode": a counting sort of the
 * (token, expert) picks by expert, then one GEMM per expert).  Same weights, routing
 * (canonical router order, ties to the lower id, renormalised top-k weights) and
 * output definition as moe_decode_layer, for 1 <= tokens <= 65536:
 *   out[t] = sum_j w_{t,j} Wd_{e_j} (silu(Wg_{e_j} x_t) * (Wu_{e_j} x_t)).
 * Gate/up and down run on the tensor cores (bf16 operands that are exact for the int4
 * codes and the bf16 rows, fp32 accumulation per 32-element block, h' split into bf16
 * hi + lo), so a token's output equals moe_decode_layer's within the layer tolerance,
 * not bitwise; it does not depend on the other tokens of the call.
 * x_bf16 [tokens][H] device, out [tokens][H] fp32 device (both 16-byte aligned);
 * expert_counts: device int32 [E] receiving the picks per expert, or NULL.
 * ws: device workspace (16-byte aligned) of at least moe_prefill_workspace_bytes.
 * The handle's max_rows does not limit tokens.  MOE_EINVAL for bad arguments,
 * MOE_EWORKSPACE for a short workspace; slot-table entries outside the bank are
 * reported by moe_last_device_status.  Enqueues 7 kernels and one memset. */
size_t moe_prefill_workspace_bytes(const moe_dims* dims, int32_t tokens);
int moe_prefill_layer(moe_handle* h, const moe_layer_w* w, const uint16_t* x_bf16, int32_t tokens,
                      float* out, int32_t* expert_counts, void* ws, size_t ws_bytes, void* stream);

/* Synchronizes `stream`, reads and clears the handle's device status word.
 * MOE_OK, MOE_ETIMEOUT (a bounded device wait gave up), MOE_EINVAL (a slot table entry
 * was outside [0, n_slots)), or MOE_ECUDA. */
int moe_last_device_status(moe_handle* h, void* stream);

/* Number of kernel launches the most recent moe_route / moe_decode_layer /
 * moe_round / moe_prefill_layer call enqueued (a graph replay counts the kernels
 * inside it). */
int32_t moe_last_launch_count(const moe_handle* h);

/* Bound on every device-side wait of this handle's kernels (default 2 s; 0 restores
 * the default).  A tiny bound makes the waits give up at once: the kernels then set
 * the timeout bit, drain their copies in flight under the default bound, and return,
 * so tests can exercise the MOE_ETIMEOUT path without any hang. */
int moe_set_wait_limit_ns(moe_handle* h, uint64_t ns);

/* Routing tail skip (an approximation; off by default).  Avalon README, "Numbers" (RX
 * 7900 XT): experts that every token of a verification routes only at rank 7 or lower
 * are skipped.  With rank = T > 0, every later moe_route / moe_decode_layer / moe_round
 * call of this handle drops a union expert when each row that picked it has it at
 * 1-based rank >= T (T = 7 is the page's setting): the expert leaves the union
 * (union_ids, n_union and stats shrink), its picks contribute nothing to the output,
 * and the remaining weights are not renormalised (the page does not say; this is the
 * reading taken).  topk_ids / topk_w still report every row's k picks.  rank = 0 turns
 * it off; T = 1 drops every expert (output 0); T > k drops none.  Returns MOE_EINVAL for
 * a NULL handle or rank < 0.  moe_decode_layer_noalloc never skips. */
int moe_set_tail_skip(moe_handle* h, int32_t rank);

/* Timing of eager (non-graph) calls.  moe_profile(h, 1) starts recording a CUDA event
 * pair around every kernel launch the handle makes on the caller's stream, and
 * per-phase device timestamps inside moe_round (first use allocates a small device
 * buffer for them); earlier records are discarded.  moe_profile(h, 0) stops.
 * moe_profile_read synchronizes the events and returns the summed device time in ms
 * and the launch count (kind must be 0: the fused round kernel).
 * moe_profile_phases writes, for the last profiled moe_round, the mean over CTAs and
 * layers (mean_us) and the per-layer maximum over CTAs averaged over layers (max_us)
 * of its phases and returns how many it wrote (or a negative MOE_E* code); n_phases
 * >= 12 always suffices.  Rounds of fewer than 13 rows (10 phases): router GEMV,
 * logits barrier (and the previous layer's output written), routing, piece issue, wait
 * for the first gate/up bytes, units before the last, the last unit's gate/up, its
 * SwiGLU and the wait for its down bytes, its down products, layer-end barrier.  Wider rounds (12 phases): router GEMV,
 * barrier 1 (and the previous layer's output written), routing, wait for the first
 * staged gate/up chunk, gate/up until the last chunk has landed, gate/up after it,
 * barrier 2, (zero), down pass, (zero), (zero), barrier 3. */
int moe_profile(moe_handle* h, int enable);
int moe_profile_read(moe_handle* h, int kind, double* total_ms, int32_t* launches);
int moe_profile_phases(moe_handle* h, double* mean_us, double* max_us, int32_t n_phases);

/* Allocation-free moe_decode_layer, for callers that may not allocate device memory at
 * all (allocation disabled by a surrounding memory pool, allocation-free real-time
 * loops, hosts that forbid cudaMalloc after start-up).  There is no counterpart on the
 * pages this layer follows; it is an integration convenience.
 *   - Needs no handle and no workspace: the scratch (barrier words, logits, exchanged
 *     SwiGLU outputs, output accumulators) is one static device array of
 *     MOE_NOALLOC_SCRATCH_BYTES that every device loading this library holds until the
 *     process exits.
 *   - Runs on the current device.  Its first call on a device sets that device up
 *     (looks up the array's device address, the SM count, the kernels' shared-memory
 *     limits); make that first call before any stream capture on the device.
 *   - Arguments as for moe_decode_layer, plus dev_status: a caller-owned device word
 *     (required; NULL gives MOE_EINVAL) into which the kernel ORs what it finds: bit 1
 *     (value 1) if a bounded device wait gave up (the output is then incomplete), bit 2
 *     (value 2) if an expert-table entry was outside [0, n_slots) (slot 0 was used
 *     instead).  The caller clears the word and reads it after the stream has finished.
 *     Returns MOE_EWORKSPACE if the layer needs more scratch than the array holds
 *     (moe_workspace_bytes(dims, rows) > MOE_NOALLOC_SCRATCH_BYTES).
 *   - Calls no cudaMalloc, cudaFree or allocating routine.  Every call shares the one
 *     array: calls whose executions overlap on the GPU (different streams, or different
 *     host threads without ordering) race on it and give wrong results. */
#define MOE_NOALLOC_SCRATCH_BYTES ((size_t)8 << 20)
int moe_decode_layer_noalloc(const moe_dims* dims, const moe_layer_w* w, const uint16_t* x_bf16,
                             int32_t rows, float* out, unsigned* dev_status, void* stream);

/* ======================================================================================
 * The attention side of a verify round
 *
 * What a round runs around its expert layers: the page and slot map of the rows to come
 * (moe_round_map), the norms and rotation of their queries and keys with the write into
 * the paged cache (moe_qk_rope_cache), the attention of the drafted rows over that cache
 * (moe_tree_attention), the log probabilities of the drafted tokens under the logits
 * (moe_token_logprobs), and which of them stand (moe_verify_drafts).  The cache may be in 8
 * bits (moe_cache8_append, moe_cache8_read, moe_tree_attention8).  The pages leave these steps
 * to the surrounding engine; their definitions here are this library's own.
 *
 * Conventions, besides those at the top of this file:
 *   - No handle.  A call runs on the current device and takes one descriptor struct that
 *     a caller fills once and may reuse for every round; the struct itself is host
 *     memory, read during the call, and its pointers are device memory.  Lengths, maps
 *     and masks are read on the device, so a captured graph follows their contents.
 *   - Device pointers are 16-byte aligned except where a field says otherwise.
 *   - Strides are below 2^40 elements, and such that a buffer's last row or slot begins less
 *     than 2^60 elements behind its first.
 *   - dev_status: a caller-owned device word, required, 4-byte aligned.  A kernel ORs
 *     MOE_DEV_* bits into it and never clears it; the caller does.
 *   - Nothing outside the described buffers is read or written whatever the device-side
 *     maps hold: an entry that does not fit is skipped and raises its bit.
 *   - The calls allocate nothing and synchronise with nothing; workspaces are passed in, set
 *     to zero once before their first use.  One buffer may serve any calls that are not
 *     under way at the same time, of other shapes and of either kind, if it is as large as
 *     the largest needs.
 *   - Outputs do not depend on the order in which thread blocks finish (bitwise).
 *   - Outputs overlap neither inputs nor each other, except where a call says that they may.
 *   - Element types: MOE_BF16, MOE_F16, and MOE_F32 where a call says so.  Sums, softmax
 *     statistics and norms are held in 32 bits; results are rounded once.
 * ====================================================================================== */

enum { MOE_BF16 = 0, MOE_F16 = 1, MOE_F32 = 2 };
enum { MOE_E4M3 = 3, MOE_I8 = 4 }; /* codes of a cache in 8 bits (moe_kv_cache8) */

enum {
  MOE_DEV_TIMEOUT = 1, /* a bounded device wait gave up: outputs are incomplete */
  MOE_DEV_SLOT = 2,    /* an expert table entry outside the bank (expert layer calls) */
  MOE_DEV_PAGES = 4,   /* free pages or table columns ran out */
  MOE_DEV_LENGTH = 8,  /* a length that is negative, too long or does not fit the rest */
  MOE_DEV_INDEX = 16,  /* a page, slot, parent or token index outside its range */
  MOE_DEV_VALUE = 32   /* a value that is not finite, or a scale that is not one, where the call says so */
};

/* A paged cache of keys and values, DEVICE pointers.  The element (page, slot in page,
 * head, e) of either is at page * page_stride + slot * slot_stride + head * head_stride
 * + e, strides in elements (multiples of 8, not negative), so both [page][slot][head][D]
 * and [page][head][slot][D] orders and slices of larger buffers can be described.  A
 * position p of a request lives in page block_table[request][p / page_size] at slot
 * p % page_size; its flat slot number is page * page_size + p % page_size, and
 * n_pages * page_size must stay below 2^31.  page_size: 1..65536. */
typedef struct moe_kv_cache {
  void* k;
  void* v;
  int64_t page_stride, slot_stride, head_stride;
  int32_t n_pages, page_size;
} moe_kv_cache;

/* Block tables, slots and tree masks of a round, from the requests' lengths alone.
 * Request b has ctx_len[b] cached positions and brings new_len[b] rows (0 allowed),
 * which take the positions after the context in the cache.  Rows are numbered request
 * after request.  With P = page_size, held_b = pages_held[b] (ceil(ctx_len[b] / P) where
 * pages_held is NULL) and need_b = ceil((ctx_len[b] + new_len[b]) / P), each request
 * takes max(0, need_b - held_b) pages from free_pages, in request order, and they are
 * written behind its held ones: block_table[b][held_b ..].  Other table entries stay.
 *   row_start [n_req + 1]  first row of each request; row_start[n_req] = all rows
 *   pages     [n_req]      pages the request holds now (the next call's pages_held; the two
 *                          may be one array, for which a second small launch is made)
 *   n_taken   [1]          pages taken: free_pages[0 .. n_taken) are in use now
 *   row_req   [n_rows]     request of the row
 *   row_pos   [n_rows]     ctx_len + depth of the row in its tree (the rotation's position)
 *   row_slot  [n_rows]     flat cache slot of the row's key and value
 *   tree_mask [n_rows]     bit j: row j of the same request is the row itself or one of
 *                          its ancestors (may be NULL)
 * parents [n_rows]: index within the request of the row's parent, less than the row's
 * own, or -1 for a row that follows the context directly (several may); requests then
 * bring at most 64 rows.  NULL: each row follows the one before it (a chain, or a
 * prompt); tree_mask is then the chain's, for at most 64 rows.
 * n_rows is the capacity of the row arrays: rows that no request brings get row_req -1,
 * row_pos 0, row_slot -1 and an empty mask, so a captured round can keep its width.  No
 * output may overlap an input or another output otherwise.
 * Raised bits: MOE_DEV_PAGES (too few free pages, or more than table_width columns
 * needed: rows without a page get slot -1, fresh table entries without one -1);
 * MOE_DEV_LENGTH (a negative length, or lengths past 2^31 - 1 together: the request brings no
 * rows, and a negative context counts as 0; pages_held below what the context needs or
 * outside the table; more rows than n_rows, the rest is left out; a tree of more than 64
 * rows, its later rows get an empty mask); MOE_DEV_INDEX (a page outside [0, n_pages),
 * treated as none; a parent outside [-1, row), treated as -1).
 * Limits: 1 <= n_req <= 16384, 0 <= n_rows <= 2^30, 1 <= table_width, n_req * table_width
 * below 2^31, 0 <= n_free. */
typedef struct moe_map_args {
  const int32_t* ctx_len;
  const int32_t* new_len;
  const int32_t* pages_held;
  const int32_t* free_pages;
  const int32_t* parents;
  int32_t* block_table; /* [n_req][table_width] */
  int32_t* row_start;
  int32_t* pages;
  int32_t* n_taken;
  int32_t* row_req;
  int32_t* row_pos;
  int32_t* row_slot;
  uint64_t* tree_mask;
  unsigned* dev_status;
  int32_t n_req, n_rows, n_free, page_size, n_pages, table_width;
} moe_map_args;
int moe_round_map(const moe_map_args* args, void* stream);

/* Norm and rotation of queries and keys, and the cache write, in one pass.  Per row and
 * head, in 32 bits: y = x * gain / sqrt(mean(x^2) + eps) (y = x where the gain is NULL);
 * then the first rot_dim elements are rotated in pairs (a, b) by the angle
 * row_pos * inv_freq[i]: (a cos - b sin, b cos + a sin) * rot_scale.  Pair i is elements
 * (i, i + rot_dim / 2), or (2i, 2i + 1) with interleaved.  inv_freq, in 64 bits, is taken
 * modulo one turn a position and multiplied in fixed point, so whole turns drop out without a
 * rounding; the angle is off by at most |row_pos| * 2^-52 turns for frequencies below one turn
 * (1.4e-9 rad at 10^6, 3e-6 at 2^31) and 1e-7 rad of its 32-bit form.  Queries go to
 * q_out; keys go to the cache at the row's slot, and so do the values, as they are.  A row with slot -1 has its queries written and nothing cached;
 * other slots outside the cache raise MOE_DEV_INDEX and are skipped.  Two rows must not
 * share a slot.
 *   q [n_rows][q_heads][D], k and v [n_rows][kv_heads][D]: the strides are from row to
 *   row, in elements (multiples of 8), so the three may lie in one projection's output.
 *   q_out may be q itself (same stride); k and v must not lie in the cache.
 * dtype: MOE_BF16 or MOE_F16, of every element array.  head_dim 64, 128 or 256; rot_dim a
 * multiple of 16, 16..head_dim, or 0 (no rotation); q_heads and kv_heads 1..256; n_rows
 * 0..2^24; eps >= 0. */
typedef struct moe_qk_rope_args {
  const void* q;
  const void* k;
  const void* v;
  void* q_out;
  const void* q_gain;     /* [D] or NULL */
  const void* k_gain;     /* [D] or NULL */
  const double* inv_freq; /* [rot_dim / 2] */
  const int32_t* row_pos;
  const int32_t* row_slot;
  unsigned* dev_status;
  moe_kv_cache cache;
  int64_t q_stride, k_stride, v_stride, q_out_stride;
  int32_t n_rows, q_heads, kv_heads, head_dim, rot_dim, interleaved, dtype;
  float eps, rot_scale;
} moe_qk_rope_args;
int moe_qk_rope_cache(const moe_qk_rope_args* args, void* stream);

/* Attention of drafted rows over the paged cache.  Request b brings the rows
 * [row_start[b], row_start[b + 1]), n_b of them, at most max_tree; the keys and values of
 * its ctx_len[b] context positions and then of its own rows lie in the cache.  Row i sees
 * every context position, and row j of its request where bit j of tree_mask[row] is set
 * (tree_mask NULL: where j <= i).  Query head h reads key/value head h / (q_heads /
 * kv_heads).  In 32 bits: s = scale * (q . k), out = sum softmax(s) v over what is seen;
 * lse = log(sum exp(s)).  A row that sees nothing gets out 0 and lse -infinity.  Positions
 * that are not seen have no influence, whatever their cached bits hold (infinities and
 * NaN included).  With n_b = 1 this is the decode step of a single token.
 * The softmax weights are rounded to the element type for the product with v (their sum
 * is not); everything else stays in 32 bits until out is rounded.
 * How the keys of a head are cut up follows the lengths of the whole call, so a row's last
 * bits may change with the lengths of other requests; not with anything else of them, and
 * the same call gives the same bits again.
 *   q, out [n_rows][q_heads][D], the strides from row to row in elements (multiples of
 *   8); lse fp32 [n_rows][q_heads] or NULL; row_start [n_req + 1] and ctx_len [n_req] as
 *   moe_round_map writes and reads them (4-byte aligned is enough).  Rows that belong to
 *   no request are not written.
 * dtype MOE_BF16 or MOE_F16; head_dim 64, 128 or 256; kv_heads a divisor of q_heads with
 * a quotient of at most 64; q_heads 1..1024; max_tree 1..64; n_req 1..16384; n_rows
 * 0..2^20; the last head of either cache's last slot less than 2^35 - 256 elements behind
 * its first element; n_req * kv_heads * (table_width * page_size / 64, rounded up, + 4)
 * below 2^31.
 * MOE_DEV_LENGTH: a negative context, row_start not ascending within n_rows, more rows
 * than max_tree, or a length beyond the table: that request's rows are not computed (out
 * 0, lse -infinity where the rows themselves are valid).  MOE_DEV_INDEX: a needed page
 * outside the cache; its positions count as not seen.  MOE_DEV_TIMEOUT: a wait inside a
 * thread block, or between blocks that share a request's context, gave up after 2 s; the
 * outputs are incomplete, and ws has to be set to zero before its next use.
 * ws: moe_tree_attention_workspace_bytes (it goes by head_dim and, up to a bound, by
 * max_tree * q_heads / kv_heads; 0 for arguments that the call would refuse), 16-byte
 * aligned, set to zero once before its first use; a call that ends without
 * MOE_DEV_TIMEOUT leaves it ready for the next, whatever its shape. */
typedef struct moe_tree_attention_args {
  const void* q;
  void* out;
  float* lse;
  const int32_t* row_start;
  const int32_t* ctx_len;
  const int32_t* block_table; /* [n_req][table_width] */
  const uint64_t* tree_mask;  /* [n_rows] or NULL */
  unsigned* dev_status;
  moe_kv_cache cache;
  int64_t q_stride, out_stride;
  int32_t n_req, n_rows, max_tree, table_width, q_heads, kv_heads, head_dim, dtype;
  float scale;
} moe_tree_attention_args;
/* Bound on the device-side waits of every later moe_tree_attention call of the process
 * (default 2 s; 0 restores it; a captured call keeps the bound of its capture).  As with
 * moe_set_wait_limit_ns a tiny bound makes waits give up at once, and the call ends its
 * products in flight under the default bound and returns, so tests can see
 * MOE_DEV_TIMEOUT without any hang. */
int moe_set_attention_wait_limit_ns(uint64_t ns);
size_t moe_tree_attention_workspace_bytes(const moe_tree_attention_args* args);
int moe_tree_attention(const moe_tree_attention_args* args, void* ws, size_t ws_bytes, void* stream);

/* A paged cache of keys and values in 8 bits, DEVICE pointers: codes, and a scale for each
 * block of block_size tokens and head, of keys and of values apart.  A value is the 32-bit
 * product code * scale.  The code (page, slot in page, head, e) of either is at the byte
 * page * page_stride + slot * slot_stride + head * head_stride + e (strides multiples of
 * 16, not negative), its scale at the float page * scale_page_stride + (slot /
 * block_size) * scale_block_stride + head * scale_head_stride (not negative).  block_size: a
 * power of two, 1..128, that divides page_size; 1 is a scale a token.
 *   format MOE_E4M3: 1 sign, 4 exponent (bias 7) and 3 mantissa bits, 0x7f and 0xff NaN (the
 *   calls never write those).  MOE_I8: two's complement; the calls write -127..127.
 * A scale is 0 or a finite positive normal number; any other counts as 0 and raises
 * MOE_DEV_VALUE where a position that a call reads goes by it.  moe_cache8_append writes
 * powers of two; a program's own calibrated scales may be any.  Strides of scales may be 0, for one
 * scale over pages, blocks or heads, where a cache is only read; moe_cache8_append wants codes and a
 * scale for each block and head, of keys and of values, that no other shares (MOE_EINVAL for strides
 * of 0 and for one array of scales for both).  Pages are numbered as in moe_kv_cache. */
typedef struct moe_kv_cache8 {
  void* k;
  void* v;
  float* k_scale;
  float* v_scale;
  int64_t page_stride, slot_stride, head_stride;
  int64_t scale_page_stride, scale_block_stride, scale_head_stride;
  int32_t n_pages, page_size, block_size, format;
} moe_kv_cache8;

/* Rows into a cache of 8 bits (moe_cache8_append) and out of it (moe_cache8_read).  Row
 * i of request b, row_start[b] + i, is its position ctx_len[b] + i: behind the context
 * where rows are appended, anywhere (0 for a whole prefix) where they are read.
 *   append: per block of tokens that rows fall into, and per head, of keys and of values, let
 *   a be the largest magnitude, finite ones only, of the block's new rows and of what it holds
 *   from before (the positions of the block that are below ctx_len[b]; codes behind them, as
 *   of drafts that were rejected, are not looked at).  The block's scale becomes 2^e
 *   with the least e >= -126 for which a <= Q * 2^e, Q = 448 (MOE_E4M3) or 127 (MOE_I8).
 *   Rows are rounded to the nearest code (ties to even) of x / 2^e; what the block holds
 *   is rounded again from its values where the scale has changed.  So a value carries the
 *   rounding of every scale that its block has had since it was written, also of one that came
 *   with rows that were rejected since: a scale that falls again does not bring back what was
 *   lost under it.  Let S be the largest of them.  With MOE_I8 a value is off by less than S, one
 *   step (rounded once: half a step); with MOE_E4M3 by less than 2^-9 S, one step of its smallest
 *   codes, beside the first rounding (2^-4 of it), and not at all further while its code is a
 *   normal one.  A held scale that is no power of two adds a rounding of its own when it is
 *   replaced.  Where rows that may be rejected are far larger than the context, blocks of one
 *   token keep them apart from it.
 *   Infinities become the largest code with their sign, NaN 0 (rows and what is held alike), and
 *   both raise MOE_DEV_VALUE.  The last block of a context is written as a whole, so it must not
 *   be shared with another request (a shared prefix ends with a block);
 *   no two rows of a call may fall into one slot.
 *   read: k, v = code * scale, rounded once to dtype.
 *   k, v [n_rows][kv_heads][D] of MOE_BF16, MOE_F16 or MOE_F32, the strides from row to row in
 *   elements (multiples of 8); they must not lie in the cache.  Rows that belong to no request
 *   are neither read nor written.
 * head_dim 64, 128 or 256; kv_heads 1..256; n_req 1..16384; n_rows 0..2^24;
 * MOE_DEV_LENGTH: a negative context, row_start not ascending within n_rows, or a length
 * beyond the table: that request is left out (its rows are not written).  MOE_DEV_INDEX: a
 * page outside the cache: what would lie there is not cached, and read as 0. */
typedef struct moe_cache8_args {
  void* k; /* append: read; read: written */
  void* v;
  const int32_t* row_start;
  const int32_t* ctx_len;
  const int32_t* block_table; /* [n_req][table_width] */
  unsigned* dev_status;
  moe_kv_cache8 cache;
  int64_t k_stride, v_stride;
  int32_t n_req, n_rows, table_width, kv_heads, head_dim, dtype;
} moe_cache8_args;
int moe_cache8_append(const moe_cache8_args* args, void* stream);
int moe_cache8_read(const moe_cache8_args* args, void* stream);

/* moe_tree_attention over a cache of 8 bits: the same rows, masks, lengths, outputs, limits,
 * raised bits and workspace rules, with keys and values code * scale (a scale that is not
 * one counts as 0 and raises MOE_DEV_VALUE).  dtype is that of q and out.  Inside, codes are
 * 16-bit numbers (exactly), queries fp16 numbers with a power of two for each row and
 * head (exactly, but for elements below 2^-31, of fp16 queries 2^-28, of its largest, which
 * are off by 2^-39 of that at most, where that is 2^-112 or more), and the softmax weights,
 * with the values' scale in them, are rounded to fp16 for the product with the codes (what is
 * lost are weights times scale under 2^-32 of the largest); the rest is in 32 bits.  Among it is
 * the product of a key's scale, |scale| and a power of two near a query row's largest element:
 * where the three together (or |scale| alone) pass 2^127, scores are past 32 bits but for codes
 * that cancel, and the row may be NaN where those would have given a number.  Scales of
 * values are taken between 2^-48 and 2^48: smaller ones count as 0 (their values are below
 * 1.6e-12), and so do larger ones, which raise MOE_DEV_VALUE.  A code that is NaN is NaN under any
 * scale, 0 too, for the rows that see it.  The span of either cache is below 2^36 - 2048 bytes here.
 * Positions that are not seen have no influence, whatever codes and scales are cached there.
 * Waits go by moe_set_attention_wait_limit_ns. */
typedef struct moe_tree_attention8_args {
  const void* q;
  void* out;
  float* lse;
  const int32_t* row_start;
  const int32_t* ctx_len;
  const int32_t* block_table; /* [n_req][table_width] */
  const uint64_t* tree_mask;  /* [n_rows] or NULL */
  unsigned* dev_status;
  moe_kv_cache8 cache;
  int64_t q_stride, out_stride;
  int32_t n_req, n_rows, max_tree, table_width, q_heads, kv_heads, head_dim, dtype;
  float scale;
} moe_tree_attention8_args;
size_t moe_tree_attention8_workspace_bytes(const moe_tree_attention8_args* args);
int moe_tree_attention8(const moe_tree_attention8_args* args, void* ws, size_t ws_bytes, void* stream);

/* Log probabilities of given tokens under rows of logits.  With z = logit *
 * inv_temperature and lse = log(sum exp(z)) over the row:
 *   logp     [n_rows]         z[token] - lse
 *   entropy  [n_rows]         -sum p log p, p = exp(z - lse), 0 log 0 = 0
 *   rank     [n_rows] int32   entries before the token by (logit descending, id ascending)
 *   top_ids  [n_rows][top_k] int32, top_logp [n_rows][top_k]: the first top_k entries in
 *                             that order and their log probabilities
 * Any output may be NULL, top_ids and top_logp only where top_k is 0.  A logit of
 * -infinity is an entry that cannot occur: it has log probability -infinity and never is
 * a top entry; where fewer than top_k entries can occur the rest is id -1 and -infinity.
 * A row without any entry that can occur: logp -infinity, entropy 0.  A token of -1 stands
 * for no token: logp -infinity, rank -1; other tokens outside the vocabulary do the same
 * and raise MOE_DEV_INDEX.  NaN or +infinity in a row makes its logp and entropy NaN, its
 * top_logp NaN or -infinity, and its rank and ids unspecified.
 * The top entries cost least where the largest logits are not all late in the row: after a
 * masked or low start, or with logits that rise along it, parts of the row are read again,
 * top_k times at worst (2,000 rows of 129,283 with the first half masked take nine times
 * as long as without a mask).  top_k 0 does not depend on the order.
 *   logits [n_rows][vocab] of MOE_F32, MOE_BF16 or MOE_F16, stride from row to row in
 *   elements, any alignment of the element type; tokens [n_rows] (NULL if neither logp nor
 *   rank is asked for).  n_rows 0..2^24, vocab 1..2^24, top_k 0..32, inv_temperature > 0
 *   and finite.
 * ws: moe_token_logprobs_workspace_bytes (some 84 KB, the same for all arguments; 0 for those
 * that the call would refuse), 16-byte aligned, set to zero once before its first use;
 * every call leaves it ready for the next, whatever its shape. */
typedef struct moe_logprob_args {
  const void* logits;
  const int32_t* tokens;
  float* logp;
  float* entropy;
  int32_t* rank;
  int32_t* top_ids;
  float* top_logp;
  unsigned* dev_status;
  int64_t stride;
  int32_t n_rows, vocab, top_k, dtype;
  float inv_temperature;
} moe_logprob_args;
size_t moe_token_logprobs_workspace_bytes(const moe_logprob_args* args);
int moe_token_logprobs(const moe_logprob_args* args, void* ws, size_t ws_bytes, void* stream);

/* Which drafted tokens stand, and which token follows.  Request b's rows are row_start[b] ..
 * row_start[b + 1] - 1, at most 64: row 0 is the token that was there before (its own
 * token is not read), the others are drafts, each behind its parent (parents[row], an index
 * within the request less than the row's own; NULL: the row before it).  logits[r] is what
 * the target says behind row r, p_r = softmax(logits[r] * inv_temperature).  From r = row
 * 0 on, the children of r are tried in the order of their rows:
 *   without draft_probs (the drafts were looked up, or are a drafter's likeliest): child c
 *   with token x is taken if p_r(x) > 0 and uniform[c] * (1 - the sum of p_r over the tokens
 *   of the children rejected before it) < p_r(x); a token that was rejected already is not
 *   taken.  After the last rejection the rest is p_r without their tokens;
 *   with draft_probs (chains only, parents NULL; draft_probs[c] the probabilities q_c that
 *   c's token was drawn from): c is taken if uniform[c] * q_c(x) < p_r(x), the rest after
 *   a rejection is max(p_r - q_c, 0);
 *   inv_temperature = +infinity (greedy): c is taken if x is the largest logit's token (of
 *   equal ones the lowest; a row of -infinity alone has none); the token that follows is that
 *   token; uniform, noise and draft_probs are not read and may be anything.
 * r goes on with the child that was taken; where none was, or there is none (the rest is
 * p_r then), the token that follows is the one with the largest rest(x) / noise[b][x], of
 * equal ones the lowest: a draw from rest if noise is exponentially distributed, entries
 * that are not positive cannot be drawn.  Where nothing of the rest is left, p_r is drawn
 * from.  So, with uniform in [0, 1), the tokens are distributed as the target's own.
 *   accepted   [n_req]   drafts that stand
 *   path       [n_rows]  path[row_start[b] + i]: the i-th row that stands (path[row_start[b]]
 *                        is 0), as an index within the request; -1 behind the last
 *   next_token [n_req]   the token that follows
 * The rows of a chain that stand lie in the cache as the next round needs them.  Those of a tree lie
 * apart: before the next round they are cached once more behind the same context
 * (moe_cache8_append with the same ctx_len, the rows gathered by path from the round's own).
 * A request without rows gets accepted 0 and next_token -1.  A draft of token -1 stands for
 * none and is not taken (its draft_probs are not read); other tokens outside the
 * vocabulary are not taken either and raise MOE_DEV_INDEX, as does a parent outside
 * [-1, row), taken as -1: such rows, but for row 0, hang on nothing and are not tried.  Logits of
 * -infinity are tokens that cannot occur.  Where the row that is drawn from has no other or
 * holds NaN or +infinity, next_token is -1; the latter raise MOE_DEV_VALUE, and no child of a
 * row with them is taken.  MOE_DEV_LENGTH: row_start not ascending within n_rows, or more
 * than 64 rows: the request gets accepted 0, next_token -1, and its path is not written.
 * Decisions come from sums in 32 bits joined in 64; a uniform number within some 1e-6 of
 * its border may fall on either side of it.
 *   logits [n_rows][vocab] of MOE_F32, MOE_BF16 or MOE_F16, stride from row to row in
 *   elements; draft_probs [n_rows][vocab] of draft_dtype, draft_stride; uniform [n_rows] and
 *   noise [n_req][vocab] (noise_stride) fp32; any alignment of their element types.  n_req
 *   1..16384, n_rows 0..2^20, vocab 1..2^24, inv_temperature > 0.
 * ws: moe_verify_drafts_workspace_bytes (it goes by n_req, n_rows and vocab alone and does not
 * fall as they grow; 0 for arguments that the call would refuse), 16-byte aligned, set to zero
 * once before its first use; every call leaves it ready for the next, whatever its shape. */
typedef struct moe_verify_args {
  const void* logits;
  const void* draft_probs; /* or NULL */
  const int32_t* row_start;
  const int32_t* parents; /* or NULL */
  const int32_t* tokens;
  const float* uniform;
  const float* noise;
  int32_t* accepted;
  int32_t* path;
  int32_t* next_token;
  unsigned* dev_status;
  int64_t stride, draft_stride, noise_stride;
  int32_t n_req, n_rows, vocab, dtype, draft_dtype;
  float inv_temperature;
} moe_verify_args;
size_t moe_verify_drafts_workspace_bytes(const moe_verify_args* args);
int moe_verify_drafts(const moe_verify_args* args, void* ws, size_t ws_bytes, void* stream);

const char* moe_strerror(int code);

#ifdef __cplusplus
}
#endif

#endif /* MOE_VERIFY_H */
