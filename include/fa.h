/*
 * fa.h -- C ABI of the GB300 (sm_103a) fused exact attention library (libfa.so).
 *
 * The operation (FlashAttention-4 blog, opening section and "Forward pass"
 * section; FlashAttention-4 paper summary, notation table):
 *
 *   S = alpha * Q K^T  (+ causal mask: key j visible to query i iff j <= i)
 *   P = softmax(S) row-wise,   O = P V,   LSE_i = ln sum_j exp(S_ij)
 *
 * and its gradients (FlashAttention-4 blog, "Backward pass" section: the five
 * products S, dP, dV, dK, dQ plus the elementwise work for P and dS):
 *
 *   dV = P^T dO,  dP = dO V^T,  D_i = sum_j P_ij dP_ij,  dS = P * (dP - D),
 *   dQ = alpha dS K,  dK = alpha dS^T Q.
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 * - Element types: q, k, v, o, do, dq, dk, dv are bfloat16 (raw 16-bit
 *   storage, passed as void*); lse is float32; cu_seqlens is int32.
 * - Head dimension d is 64, 128 or 256 (the pages' balance point moves with
 *   d: FlashAttention-4 paper summary, "Roofline" remarks).  Hq must be a multiple of Hkv; query head h reads
 *   key/value head h / (Hq / Hkv).
 * - Fixed-length layout (cu_seqlens == NULL): q, o, do, dq are [B, N, Hq, d]
 *   row-major, k, v, dk, dv are [B, N, Hkv, d]; lse is [B, Hq, N].
 * - Variable-length layout (cu_seqlens != NULL): B sequences packed along
 *   the token axis; N is then the TOTAL token count T; q, o are [T, Hq, d],
 *   k, v are [T, Hkv, d], lse is [Hq, T].  cu_seqlens is a DEVICE array of
 *   B+1 non-decreasing offsets with cu_seqlens[0] = 0 and cu_seqlens[B] = T;
 *   max_seqlen is an upper bound on every sequence length.  Malformed
 *   offsets are sanitised by one rule in every kernel: c'_0 = clamp(c_0, 0,
 *   T), c'_s = max(c'_{s-1}, clamp(c_s, 0, T)), and sequence s is rows
 *   [c'_s, c'_{s+1}).  Sequences thus never overlap and never leave the
 *   tensors; rows outside every sequence are not written (o, lse, dk, dv)
 *   or written as zero (dq).  A sanitised sequence longer than 131072
 *   tokens (possible only when max_seqlen understates the lengths) makes a
 *   d = 64/128 call compute nothing and report FA_ERR_INVALID through
 *   fa_get_device_status; the d = 256 forward has no such limit.
 * - Causal masks are top-left aligned within each sequence (query and key
 *   lengths are equal).
 * - Pointers are device pointers owned by the caller; the library allocates
 *   no device memory.  Every tensor must be 16-byte aligned and contiguous.
 * - Calls are asynchronous: they validate arguments on the host, enqueue
 *   kernels on `stream` and return.  They never synchronise (except
 *   fa_get_device_status).  No exception crosses the ABI.
 * - Return value: FA_OK, or a negative fa_status for invalid arguments
 *   (nothing is launched) or a launch error.  Device-side faults of the
 *   pipeline's own bounded waits are reported through fa_get_device_status.
 */
#ifndef FA_H_
#define FA_H_

#include <stddef.h>
#include <stdint.h>
#include <cuda_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    FA_OK = 0,
    FA_ERR_INVALID = -1,      /* null pointer, bad size, bad scale           */
    FA_ERR_UNSUPPORTED = -2,  /* legal but not built: d not 64/128/256, ... */
    FA_ERR_ALIGN = -3,        /* a tensor is not 16-byte aligned            */
    FA_ERR_LAUNCH = -4,       /* CUDA reported an error at launch           */
    FA_ERR_TIMEOUT = -5,      /* a device-side wait gave up (see status)    */
    FA_ERR_WORKSPACE = -6     /* workspace missing or too small             */
} fa_status;

/* Human-readable name of a status code (static string, never NULL). */
const char *fa_status_string(int status);

/* Number of streaming multiprocessors the kernels size their persistent
 * grids by on the current device (>0), or a negative fa_status. */
int fa_num_sms(void);

/*
 * Process-wide tuning of the forward kernel (affects later fa_fwd calls):
 *   exp2_emu_sixteenths: share of the softmax exponentials evaluated on the
 *     FMA pipe by the polynomial (fa_exp2_emu) instead of MUFU.EX2, in
 *     sixteenths (0 to 4, i.e. up to 25 %; FlashAttention-4 paper summary
 *     §3.1.3 uses 10-25 %).  Both d = 128 forward kernels and the d = 64 one
 *     apply it.
 *   tau: conditional-rescale threshold in log2 units, 0 <= tau <= 64
 *     (default log2(256) = 8; tau = 0 rescales whenever the max grows).
 * At d = 256 only tau applies: that forward evaluates every exponential on
 * MUFU (its exponentials are off the critical path; the products set the
 * pace).  Every setting gives the same attention up to rounding.  Not thread-safe
 * with concurrent fa_fwd calls.  Errors: FA_ERR_UNSUPPORTED, FA_ERR_INVALID.
 */
int fa_set_tuning(int exp2_emu_sixteenths, float tau);

/*
 * Process-wide choice of the forward kernel (affects later fa_fwd calls):
 *   0 -- two 128-row query tiles per CTA in ping-pong, 128-key tiles: the
 *        pipeline of the FlashAttention-4 blog, "Forward pass";
 *   2 -- (default) CTA pairs (clusters of two): 256 query rows per pair and
 *        256-key blocks, each product one M = 256 UMMA over both SMs, so each
 *        SM loads and reads only half of every K and V block.
 * Kernel 2 serves fixed-length and packed varlen inputs with d = 128; d = 64
 * calls use kernel 0.
 * Both compute the same attention up to rounding.
 * Errors: FA_ERR_INVALID (any other value).
 */
int fa_set_fwd_kernel(int kernel);

/*
 * Number of CTA pairs forward kernel 2 keeps resident (its persistent grid is
 * that many clusters of two; a cluster must fit inside one GPC, so this can be
 * below half the SM count).  0 until the kernel has been launched once in
 * this process.  Never fails.
 */
int fa_fwd_pairs_resident(void);

/*
 * Process-wide choice of the backward main kernel (affects later fa_bwd
 * calls; FlashAttention-4 blog, "2-CTA backward"):
 *   0 -- (default) one CTA per 128-key tile;
 *   1 -- CTA pairs per 256-key block: S^T, dP^T, dV and dK are
 *        M = 256 products over both SMs (each stages half of every B
 *        operand), dQ an M = 128 pair product after an exchange of half of
 *        dS through distributed shared memory; the dQ of a tile is computed
 *        during the next tile, in the S columns beside P^T ("2-CTA
 *        backward": the previous tile's dQ before the current dP).
 * Kernel 1 serves d = 128 inputs, fixed length or packed varlen, atomic or
 * deterministic; other head dims use kernel 0 (d = 256 its own kernel).
 * Both compute the same gradients up to the order of the fp32 dQ
 * additions; kernel 0 is the faster on GB300.  Errors: FA_ERR_INVALID.
 */
int fa_set_bwd_kernel(int kernel);

/*
 * Number of CTA pairs backward kernel 1 keeps resident; 0 until it has been
 * launched once in this process.  Never fails.
 */
int fa_bwd_pairs_resident(void);

/*
 * Process-wide order in which the kernels take their work units (affects
 * later fa_fwd and fa_bwd calls), for testing the scheduler:
 *   0 -- (default) the cost-ordered schedule (FlashAttention-4 blog,
 *        "Scheduling"): longest-processing-time first under a causal mask
 *        and for packed varlen batches (sequences sorted by length),
 *        L2-sized (batch, head) sections, zig-zag couples of query blocks;
 *   1 -- plain enumeration: (sequence, head) major, query tiles (forward)
 *        or key tiles (backward) ascending, sequences in index order.
 * Each work unit's arithmetic does not depend on the order, so the forward's
 * O and LSE and the deterministic backward's gradients are bitwise the same
 * under both; the atomic backward's dQ differs by the order of its fp32
 * additions only.  Order 1 is slower under a causal mask or with unequal
 * sequence lengths.  Not thread-safe with concurrent calls.
 * Errors: FA_ERR_INVALID (any other value).
 */
int fa_set_schedule_order(int order);

/*
 * Debug counters for the scheduler's exactly-once property (FlashAttention-4
 * blog, "Scheduling": every work tile is handed out once) and for the
 * conditional rescale (paper summary §3.1.4: how often tau = 8 skips).
 * Process-wide; affects later fa_fwd / fa_bwd calls; all NULL (the default)
 * turns counting off.  The caller owns and zeroes the device buffers; the
 * kernels only add to them (atomically), so calls accumulate.  With T the
 * token count (B * N fixed length, the packed total for varlen):
 *   visits (int [Hq * T] for fa_fwd, [Hkv * T] for fa_bwd; may be NULL):
 *     fa_fwd adds 1 at [h * T + r] when it finishes the 128-row query tile
 *     of head h starting at token row r; fa_bwd adds 1 at [hk * T + r] when
 *     it finishes the work unit of key/value head hk whose 128-key tile
 *     starts at row r (its dK, dV written; units split by query-head group
 *     count once per group);
 *   inner (int [Hq * T], fa_bwd; may be NULL): 1 at [h * T + r] each time a
 *     128-key tile's dQ contribution to the query tile of head h starting at
 *     row r has been added (so the count is the number of key tiles that see
 *     the query tile; at d = 256 the query tiles are the kernel's 64-row
 *     steps, counted by the first head-dim half's pass);
 *   rescales (unsigned long long [2], fa_fwd; may be NULL): [1] counts the
 *     per-warp rescale decisions after each row block's first key block,
 *     [0] those that took the rescale branch (tau exceeded).
 * Tile starts are the sequence start plus multiples of 128.  Counting costs
 * an atomic per tile (and per warp decision): a debugging aid, not for
 * timed runs.  While any counter is armed, the CTA-pair forward, the CTA-pair
 * backward and both d = 256 kernels run a separate build that counts; the
 * build without the counters has no trace of them.
 * Errors: FA_ERR_ALIGN (misaligned pointer).
 */
int fa_set_debug_counters(int *visits, int *inner, unsigned long long *rescales);

/*
 * Forward: O and LSE of exact attention (FlashAttention-4 blog, "Forward
 * pass: a new softmax pipeline with conditional rescaling").
 *
 * q [B,N,Hq,d], k/v [B,N,Hkv,d] bf16 in; o [B,N,Hq,d] bf16 out,
 * lse [B,Hq,N] float32 out (natural log, includes alpha).  Varlen: see
 * above.  alpha > 0 is the logit scale (normally 1/sqrt(d)).
 * causal: 0 or 1.  N == 0 (or T == 0) is a no-op returning FA_OK.
 * Errors: FA_ERR_INVALID (null pointer, B<1, N<0, Hq/Hkv<1, Hq % Hkv,
 * alpha not finite and > 0, varlen without max_seqlen>0),
 * FA_ERR_UNSUPPORTED (d not 64, 128 or 256; varlen with B > 1024 or
 * max_seqlen > 131072),
 * FA_ERR_ALIGN, FA_ERR_LAUNCH.  d = 256 runs on a kernel of its own (one
 * 128-row query tile per CTA, 64-key blocks) whatever fa_set_fwd_kernel says.
 */
int fa_fwd(const void *q, const void *k, const void *v, void *o, float *lse,
           int B, int Hq, int Hkv, int N, int d, float alpha, int causal,
           const int *cu_seqlens, int max_seqlen, cudaStream_t stream);

/*
 * Bytes of device workspace fa_bwd needs (the library allocates none):
 * D (rowsum(dO*O), fp32), the fp32 dQ accumulator, the deterministic-mode
 * semaphores, the varlen work list and, for varlen at d = 64 or 128, room
 * for fp32 dK and dV partial sums (Hq * T * d / 2 bytes; used when the work
 * is split by query-head group, see fa_bwd).  N is the sequence length
 * (fixed length) or the total token count T (varlen = 1).  Returns 0 for
 * invalid sizes (d not 64, 128 or 256 among them).  About (4 d + 4) * Hq * T
 * bytes (varlen at d = 64 / 128: (4.5 d + 4) * Hq * T).
 */
size_t fa_bwd_workspace_size(int B, int Hq, int N, int d, int deterministic, int varlen);

/*
 * Backward: dQ, dK, dV of exact attention (FlashAttention-4 blog, "Backward
 * pass", "Deterministic mode").  Inputs q, k, v, the forward's o and lse,
 * and the upstream gradient dout (layouts as in fa_fwd); outputs dq like q,
 * dk and dv like k (bf16; for Hkv < Hq, dk/dv sum over the query heads of
 * each group).  deterministic = 1 adds dQ contributions in a fixed order
 * (bit-identical across runs); 0 uses unordered fp32 reductions.
 * workspace: device memory of at least fa_bwd_workspace_size(...) bytes,
 * 256-byte aligned, owned by the caller; its contents need no
 * initialisation and are overwritten.  Calls that share a workspace must not
 * overlap on the GPU.
 * d = 256 runs on a kernel of its own: the dK / dV accumulators of a
 * 128-key tile would fill all of tensor memory, so each tile is processed
 * once per head-dim half of the gradients (recomputing S and dP for each),
 * with queries in 64-row steps (fa_set_bwd_kernel does not apply).
 * Packed varlen batches in atomic mode whose key/value heads each serve at
 * least 16 query heads (a multiple of 8; MQA-like) run, on the one-CTA
 * kernel at d = 64 or 128, as work units of 8 query heads each: the CTAs of
 * a wave then share one head group's rows of Q, dO and the dQ accumulator
 * in L2 (FlashAttention-4 blog, "Scheduling": L2-sized sections), and each
 * unit adds its group's share of dK and dV into fp32 sums in the workspace
 * that the last stage converts to bf16 (dK times alpha).
 * Errors: as fa_fwd, plus FA_ERR_WORKSPACE (NULL, misaligned or too small)
 * and FA_ERR_UNSUPPORTED (varlen with max_seqlen > 131072 or B > 1024).
 */
int fa_bwd(const void *q, const void *k, const void *v, const void *o, const float *lse,
           const void *dout, void *dq, void *dk, void *dv,
           int B, int Hq, int Hkv, int N, int d, float alpha, int causal,
           const int *cu_seqlens, int max_seqlen, int deterministic,
           void *workspace, size_t workspace_bytes, cudaStream_t stream);

/*
 * fa_bwd split into its three launches, for callers that time or schedule
 * them separately: stages is a bit mask, 1 = preprocess (D, zero the dQ
 * accumulator and semaphores, varlen work list), 2 = main kernel (dK, dV and
 * the dQ accumulator), 4 = dQ postprocess (dq = bf16(alpha * accumulator)).
 * Stages must run in this order on one workspace; fa_bwd == stages 7.  For
 * a packed varlen batch, stage 1 plans the work list for the backward kernel
 * selected at that time (fa_set_bwd_kernel) and for the call's mode (units
 * split by query-head group or not, see fa_bwd): a stage 2 run with the
 * other selection or the other mode computes nothing and reports
 * FA_ERR_INVALID through fa_get_device_status.  With split units, stage 4
 * also writes dk and dv.
 */
int fa_bwd_stages(int stages, const void *q, const void *k, const void *v, const void *o,
                  const float *lse, const void *dout, void *dq, void *dk, void *dv,
                  int B, int Hq, int Hkv, int N, int d, float alpha, int causal,
                  const int *cu_seqlens, int max_seqlen, int deterministic,
                  void *workspace, size_t workspace_bytes, cudaStream_t stream);

/*
 * fa_bwd without a workspace argument, for callers that cannot allocate
 * device memory when they need gradients (for example code running under a
 * framework that owns every device allocation, or a plugin whose host
 * application forbids allocation after start-up).  The FlashAttention-4 pages
 * have no counterpart: this is a library convenience.
 *
 * It computes exactly what fa_bwd computes (same arguments, minus the
 * workspace) and allocates nothing: its scratch is a 64 MiB array of static
 * device storage inside the library, reserved on every GPU that loads the
 * library until the process exits.  Sizes whose workspace
 * (fa_bwd_workspace_size) exceeds 64 MiB -- about Hq * T > 130000 -- are
 * rejected with FA_ERR_WORKSPACE before anything is launched; other errors
 * as fa_bwd.
 * - The first call on each device looks up the array's device address
 *   (cudaGetSymbolAddress) with that device current; make that first call
 *   before any stream capture.
 * - All calls on a device share the one scratch array, which keeps the last
 *   call's contents (each call re-zeroes what must start at zero).  Calls
 *   that overlap on the GPU (different streams, or concurrent host threads)
 *   race on it and produce wrong gradients: serialise them.
 * - A device-side wait timeout (or an offset table the plan stage rejects)
 *   is recorded in the scratch area's own status word;
 *   fa_get_device_status reports and clears it on this device, as it does
 *   for a workspace passed to it.
 * Argument errors are fa_bwd's, checked in fa_bwd's order (FA_ERR_UNSUPPORTED
 * for an unbuilt head dim, ...); a call with no tokens returns FA_OK.
 */
int fa_bwd_noalloc(const void *q, const void *k, const void *v, const void *o, const float *lse,
                   const void *dout, void *dq, void *dk, void *dv,
                   int B, int Hq, int Hkv, int N, int d, float alpha, int causal,
                   const int *cu_seqlens, int max_seqlen, int deterministic, cudaStream_t stream);

/*
 * Serving: a paged key/value cache and attention over it
 * ------------------------------------------------------
 * One step of a serving loop is fa_page_plan (pages and slots for the step's
 * new tokens), fa_kv_store (their keys and values into the cache) and
 * fa_prefix_fwd (attention of the new tokens).  fa_fwd serves prompts that
 * have nothing in the cache.
 * - The cache: k_pages and v_pages are bf16 [num_pages, Hkv, page_size, d];
 *   page_size is 16, 32, 64, 128 or 256 tokens.  Slot s is row s % page_size
 *   of page s / page_size, of every head.
 * - A block table [B, table_width] (int32) lists each request's pages in the
 *   order of its tokens.  An entry outside [0, num_pages) is "no page":
 *   nothing is read or written there, and the keys it would hold are absent.
 * - At most 1024 requests a call.  The requests' lengths are read on the device,
 *   so a captured graph serves later steps with other lengths.  What the host
 *   passes stays as captured: prefix_len, max_seqlen, the numbers of rows and
 *   requests, the table's width.
 */

/*
 * Block tables and slot maps of one step, from request lengths on the device.
 *
 *   have_b = ceil(c_b / page_size),  need_b = ceil((c_b + n_b) / page_size)
 *
 * ctx_lens [B]: c_b, request b's tokens in the cache (below 0 counts as 0,
 * above the row's capacity table_width * page_size as that); new_lens [B]:
 * n_b, tokens it adds in this step, or any negative number when it leaves.
 * block_table [B, table_width], in and out: the first have_b entries of row b
 * are read; entries have_b .. need_b - 1 are written; others are left alone.
 * Free pages wait in a queue: ring [num_pages] with the counters
 * pool = {head, tail, -}; position i (head <= i < tail) is ring[i %
 * num_pages].  New pages come off its head, requests in order and each
 * request's in order; pages of requests that leave go behind its tail in the
 * same order (their entries as they stand, table rows untouched), and can be
 * handed out from the next call on.  pool_out [3] receives the new {head,
 * tail, missing}: missing counts the pages that the queue (or the row's
 * width) could not give, entries of the queue that are no pages among them (a
 * request that leaves with absent pages puts them there).  Their table entries
 * are -1 (past the width: none), their tokens' slots -1; the caller looks at
 * missing before the step counts as done.  (The same step repeated meets entries
 * that are no pages again; they are gone once pool_out is taken over.  Tokens
 * that go on in a page that the request itself lacks have slots -1, too, and
 * are not counted.)  Pages coming back beyond num_pages in the queue are
 * dropped.
 * cu_new [B+1]: prefix sums of the n_b that are >= 0 (the cu_seqlens of the
 * step's packed rows); kv_lens [B]: c_b + n_b (at most the row's capacity), 0
 * for a request that leaves; slots [num_slots]: the slot of packed row t, -1
 * where it has no page and for rows t >= cu_new[B]; rows t >= num_slots get
 * none.
 * A call writes nothing that it reads, so the same call again gives the same.
 * One launch, no workspace.  An array that is written must not overlap another
 * (kv_lens is not written over ctx_lens, nor pool_out over pool).
 * Errors: FA_ERR_INVALID (null pointer, B, table_width or num_pages < 1,
 * num_slots < 0, arrays that overlap), FA_ERR_UNSUPPORTED (B > 1024, page_size,
 * B * table_width, table_width * page_size or num_pages * page_size above
 * 2^31 - 1), FA_ERR_ALIGN (an array not aligned to its element),
 * FA_ERR_LAUNCH.
 */
int fa_page_plan(const int *ctx_lens, const int *new_lens, int B, int page_size, int *block_table, int table_width,
                 int *ring, int num_pages, const int64_t *pool, int64_t *pool_out, int *cu_new, int *kv_lens,
                 int *slots, int num_slots, cudaStream_t stream);

/*
 * Writes a step's keys and values into the cache: row t of k and v ([T, Hkv,
 * d] bf16; k_stride and v_stride elements between tokens, at least Hkv * d and
 * multiples of 8, so both may be cut from one projection's output) goes to
 * slot slots[t].  Slots outside [0, num_pages * page_size) are skipped, every
 * other slot is left as it was.  The slots of one call must be distinct: where
 * two rows share one, the slot holds parts of either.  k and v may be rows of
 * the cache itself, other ones than the call writes.  k_pages and v_pages must
 * not overlap, but may be one array when k and v are one, too.
 * d is 64, 128 or 256.  T == 0 is a no-op.
 * Errors: FA_ERR_INVALID (null pointer, T < 0, Hkv, d or num_pages < 1, stride below Hkv
 * * d, page arrays that overlap each other or slots), FA_ERR_UNSUPPORTED (d, page_size, num_pages * page_size above 2^31 -
 * 1), FA_ERR_ALIGN (k, v or a page array not 16-byte aligned, a stride not a
 * multiple of 8), FA_ERR_LAUNCH.
 */
int fa_kv_store(const void *k, const void *v, int64_t k_stride, int64_t v_stride, const int *slots, int T, int Hkv,
                int d, void *k_pages, void *v_pages, int num_pages, int page_size, cudaStream_t stream);

/*
 * Attention of a step's tokens for a batch whose requests share a prefix:
 * query i (of n_b) of request b sees all prefix_len keys of the prefix and
 * keys j <= s_b - n_b + i of its own s_b (its last n_b keys are the new
 * tokens'; with s_b < n_b the first queries see none of them):
 *
 *   x_j = alpha q . k_j,  O = softmax(x) V,  LSE = ln sum_j exp(x_j)
 *
 * The prefix's part is computed once for the rows of all requests (each key
 * and value of it is read once for up to 256 rows of its head), every
 * request's own part from its pages; the two are joined by their maxima and
 * sums.  A request with four such blocks of rows of its own (128 rows each at
 * d = 256) reads the prefix for itself.  Equal calls give equal results, bit for bit.
 * Scores, sums and the output's accumulator are 32 bits wide, the weights bf16
 * for the product with V.
 * q: bf16 [T, Hq, d], q_stride elements between tokens (>= Hq * d, a multiple
 * of 8); o: bf16 [T, Hq, d]; lse: float32 [Hq, T].
 * cu_seqlens [B+1] (device) delimits the requests' rows as in fa_fwd, each of
 * at most max_seqlen rows; NULL: one row a request, T == B.  Rows outside
 * every request are not written.  A request with more rows than max_seqlen
 * makes the call compute nothing and report FA_ERR_INVALID through
 * fa_get_device_status.  max_seqlen decides one shape of the kernel for all
 * requests: right for any mixture, but a chunk of 512 rows among 63 single
 * tokens (32 / 8 heads of 128) takes 4 to 12 % longer than the two apart.
 * block_table [B, table_width] and kv_lens [B] (s_b, taken as at least 0 and
 * at most table_width * page_size): the requests' own keys; prefix_table: the
 * prefix's pages (ceil(prefix_len / page_size) entries), NULL when prefix_len
 * is 0.  Keys of absent pages (see above) are not seen.  A row that sees no
 * key at all gives O = 0 and LSE = -inf.  What the cache holds behind the
 * lengths does not matter, NaN and infinities included; a NaN in a query or in
 * a key gives NaN in the rows that see it, one in a value (or an infinity) may
 * also reach the request's rows before it, whose weight for it is 0.
 * o, lse and the workspace must not overlap an input or one another (o between
 * the tokens of a strided q does not).  workspace: at least
 * fa_prefix_workspace_size(...) bytes, 256-byte aligned, no initialisation
 * needed; calls that share one must not overlap on the GPU (captured graphs
 * that hold the same one included).  A call whose kernel gives up a wait (2 s)
 * reports FA_ERR_TIMEOUT through fa_get_device_status; one that was not read
 * does not stop later calls.
 * T == 0 is a no-op.
 * Errors: FA_ERR_INVALID (null pointer, T < 0, B, Hq, Hkv, num_pages or
 * table_width < 1, Hq % Hkv, prefix_len < 0, alpha not finite and > 0,
 * max_seqlen < 1, q_stride below Hq * d, T != B without cu_seqlens, arrays that
 * overlap),
 * FA_ERR_UNSUPPORTED (d not 64, 128 or 256; Hq / Hkv > 128; B > 1024;
 * page_size; prefix_len or table_width * page_size above 2^29; Hq * T, B *
 * table_width or num_pages * Hkv * page_size above 2^31 - 1; row blocks times
 * tiles of 64 keys that the lengths allow above 2^30), FA_ERR_ALIGN,
 * FA_ERR_WORKSPACE, FA_ERR_LAUNCH.
 */
int fa_prefix_fwd(const void *q, int64_t q_stride, const void *k_pages, const void *v_pages, void *o, float *lse,
                  int T, int B, int Hq, int Hkv, int d, float alpha, int num_pages, int page_size,
                  const int *block_table, int table_width, const int *kv_lens, const int *cu_seqlens, int max_seqlen,
                  const int *prefix_table, int prefix_len, void *workspace, size_t workspace_bytes,
                  cudaStream_t stream);

/*
 * Bytes of device workspace fa_prefix_fwd needs for T rows of B requests of at
 * most max_seqlen rows each (the current device's SM count enters: call it
 * with the device current); 0 for invalid sizes.  Enough for every call with
 * at most these T and B, and this max_seqlen or one below it; max_seqlen above
 * T counts as T.
 */
size_t fa_prefix_workspace_size(int T, int B, int Hq, int Hkv, int d, int max_seqlen);

/*
 * Reads (and clears) the library's device status word on the current
 * device after synchronising `stream`: FA_OK, or FA_ERR_TIMEOUT when a
 * kernel's bounded wait gave up (the kernel then skipped its remaining work,
 * drained its own copies, freed its tensor memory and returned), or
 * FA_ERR_INVALID when a kernel rejected a device-side table (a varlen batch
 * whose sanitised offsets hold a sequence longer than the 131072-token
 * limit: nothing is computed for that call).
 * `workspace` may be NULL; when it is a backward workspace its status word
 * is read (and cleared) too, and after a reported failure the main stage's
 * unit claim counter in the workspace is rewound, so that a later
 * fa_bwd_stages call with stages == 2 alone starts from the first unit.
 * The status word of fa_bwd_noalloc's scratch area on this device is read,
 * cleared and rewound the same way once a no-allocation call has run here.
 * The first non-OK code found is returned (device word, then workspace,
 * then scratch area); all of them are cleared.
 */
int fa_get_device_status(const void *workspace, cudaStream_t stream);

/*
 * The forward kernel's FMA-pipe exponential, exposed for testing: y[i] =
 * 2^x[i] by Cody-Waite range reduction (n = floor(x), f = x - n) and a
 * degree-3 Horner polynomial in f with p0 = 1, scaled by adding n to the
 * exponent bits (FlashAttention-4 blog, "Faster exponential" section;
 * paper summary §3.1.3: max relative error 8.77e-5 on [0,1)).  Inputs below
 * -127 (and -inf) give 0 or a value below 2^-126.  Each element is
 * evaluated both in the scalar form (ping-pong forward) and in the packed
 * two-lane form (CTA-pair forward); where the two differ in any bit, y[i] is
 * NaN.  x, y: device float32 arrays of n elements.
 * Errors: FA_ERR_INVALID, FA_ERR_LAUNCH.
 */
int fa_exp2_emu(const float *x, float *y, int64_t n, cudaStream_t stream);

/*
 * Diagnostic for the failure-detection path, for tests: enqueues a one-block
 * kernel on `stream` whose warp waits, through the same bounded mbarrier
 * wait every kernel here uses, on a barrier nothing ever arrives at.  After
 * the wait limit (about 2 s) it records FA_ERR_TIMEOUT in the current
 * device's status word and returns; the context stays usable, and
 * fa_get_device_status(NULL, stream) then reports (and clears) the timeout.
 * Errors: FA_ERR_LAUNCH.
 */
int fa_selftest_timeout(cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* FA_H_ */
