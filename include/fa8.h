/*
 * fa8.h -- C ABI of the GB300 (sm_103a) fused FP8 attention forward.
 *
 *   O   = softmax( softmax_scale * dq * dk * Q K^T  [+ causal / left-window mask]
 *                  [+ learnable sink in the denominator] ) * V * dv
 *   LSE = natural-log log-sum-exp of the masked, scaled scores (and the sink)
 *
 * with Q, K, V in E4M3, O in bf16 or fp16 and LSE in fp32.
 *
 * Where the operation is defined (page title, section):
 *  - "PyTorch ... FlashAttention-4 MXFP8", 2.1 Attention Forward: S = Q K^T,
 *    P = softmax(S), O = P V.
 *  - "[Cute,Fwd,Sm90] Native FP8 (E4M3 Q/K/V) forward for Hopper":
 *    Design/"Descales" (q/k descales fold into the softmax scale, v descale into the
 *    final normalisation; each 0-d or (batch, kv_heads)); Design/"Paged K/V";
 *    Design/"Decode launches" (host-known launch choices); "Supported" (head dims,
 *    causal, sliding window, varlen, paged K/V, PackGQA, SplitKV, learnable sink,
 *    fp16/bf16 output) and "Rejected with an error" (E5M2, mixed dtypes).
 *  - "tml-fa4 PR #4", Summary: P carries a 2^8 bias that cancels in the O
 *    normalisation and is removed from the LSE.
 *
 * Every pointer argument is owned by the caller.  The library keeps no pointer after
 * a call returns other than inside the work it enqueued on `stream`.  Arguments are
 * validated on the host before anything is enqueued; on an error nothing is enqueued,
 * a status code is returned and fa8_last_error() gives a one-line reason.
 */
#ifndef FA8_H_
#define FA8_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define FA8_VERSION 100 /* 1.0.0 */

#if defined(__GNUC__)
#define FA8_API __attribute__((visibility("default")))
#else
#define FA8_API
#endif

typedef enum {
    FA8_SUCCESS = 0,
    FA8_ERR_INVALID_ARG = 1,    /* malformed shape, stride, pointer or flag           */
    FA8_ERR_UNSUPPORTED = 2,    /* well-formed but not implemented (e.g. E5M2, d=80)  */
    FA8_ERR_WORKSPACE = 3,      /* split-KV workspace missing or too small            */
    FA8_ERR_CUDA = 4,           /* a CUDA runtime/driver call failed                  */
    FA8_ERR_DEVICE_TIMEOUT = 5, /* a kernel gave up a bounded wait (see fa8_check)    */
    FA8_ERR_DEVICE_BOUNDS = 6   /* a kernel saw a block-table entry out of range      */
} fa8_status;

typedef enum {
    FA8_DTYPE_E4M3 = 1, /* float8_e4m3fn */
    FA8_DTYPE_E5M2 = 2, /* float8_e5m2 (rejected as Q/K/V) */
    FA8_DTYPE_BF16 = 3,
    FA8_DTYPE_F16 = 4,
    FA8_DTYPE_F32 = 5,
    FA8_DTYPE_I32 = 6,
    FA8_DTYPE_F64 = 7
} fa8_dtype;

/*
 * A strided view of device memory.  `stride` is in elements; unused trailing entries of
 * `shape`/`stride` are ignored.  A 0-d tensor has ndim == 0.
 */
typedef struct {
    void *data;
    int32_t dtype; /* fa8_dtype */
    int32_t ndim;  /* 0..4 */
    int64_t shape[4];
    int64_t stride[4];
} fa8_tensor;

/*
 * fa8_fwd -- enqueue the fused FP8 attention forward on `stream` (a cudaStream_t).
 *
 * Layouts (the last dimension is always contiguous):
 *   q   batched (B, Sq, Hq, D)            or varlen (total_q, Hq, D) with cu_seqlens_q
 *   k   batched (B, Sk, Hkv, D)           or varlen (total_k, Hkv, D) with cu_seqlens_k
 *       or paged (num_pages, page_size, Hkv, D) with block_table and cu_seqlens_k
 *   v   as k with DV in place of D
 *   out like q with DV in place of D; bf16 or fp16
 *   lse batched (B, Hq, Sq) or varlen (Hq, total_q); fp32; may be NULL
 * Q/K/V are E4M3 (E5M2 or mixed dtypes -> FA8_ERR_UNSUPPORTED).  (D, DV) is one of
 * (64,64), (96,96), (128,128), (192,128), (192,192), (256,256).  Hq % Hkv == 0 and Hq/Hkv <= 128;
 * q-head h reads kv-head h / (Hq/Hkv).  Row strides of q/k/v must be multiples of 16
 * bytes and their base pointers 16-byte aligned (they are read by TMA).
 *
 * cu_seqlens_q / cu_seqlens_k: int32 (B+1) prefix sums of the per-request query / key
 *   lengths.  For paged K/V, cu_seqlens_k gives each request's key count (its
 *   differences); keys are read only from the first ceil(len/page_size) entries of the
 *   request's block_table row.
 * block_table: int32 (B, max_pages), stride(1) == 1, entries are page indices into
 *   k/v dim 0.  page_size must equal k.shape[1] and be a multiple of 8.
 *   Entries out of range read as zeros (TMA bounds) and raise FA8_ERR_DEVICE_BOUNDS in
 *   fa8_check; they never make the kernel touch memory outside k/v.
 * descale_q/k/v: fp32, 0-d or (B, Hkv) with any strides (0 = broadcast); NULL = 1.0.
 *   They must be positive.
 * sink: fp32 (Hq,) natural-log logits added to every row's denominator; NULL = none.
 * causal: 0/1, bottom-right aligned (key j visible to query i when j <= i + Lk - Lq).
 * window_left: -1 = unbounded, else keys j >= i + Lk - Lq - window_left stay visible.
 * softmax_scale: <= 0 selects 1/sqrt(D).
 * num_splits: 0 = heuristic, 1 = no split, n > 1 = launch n splits of each tile's key
 *   range and merge them with a second kernel.  The launch depends only on shapes and the
 *   device's SM count, never on device values, so a call can be graph-captured.  On the
 *   device, a tile whose visible keys span t KV tiles of 128 keys runs
 *   min(n, max(1, ceil(t / cap))) of the launched splits; the other splits exit at once and
 *   the merge does not read them.  cap (2 to 512 KV tiles per split) is chosen once per
 *   call from the requests' key counts: the choice that minimises a model of the run time
 *   (a fixed cost per work unit, the units spread over the CTAs that run at once, and the
 *   longest unit's tail).  The heuristic launches about eight waves of CTAs, or one wave
 *   when there are few (query tile, kv-head) pairs; when every launched split fits in one
 *   wave the finest cap is used, and with dense K/V and batched q (every length known from
 *   the shapes) the host chooses the cap and launches only the splits that run.
 * workspace / workspace_bytes: device scratch for the split partials and the split cap the
 *   forward kernel passes to the merge kernel, at least fa8_fwd_workspace_size() bytes
 *   (may be NULL/0 when that size is 0).
 */
FA8_API fa8_status fa8_fwd(const fa8_tensor *q, const fa8_tensor *k, const fa8_tensor *v,
                   const fa8_tensor *descale_q, const fa8_tensor *descale_k,
                   const fa8_tensor *descale_v, fa8_tensor *out, fa8_tensor *lse,
                   const fa8_tensor *cu_seqlens_q, const fa8_tensor *cu_seqlens_k,
                   const fa8_tensor *block_table, int page_size, int causal, int window_left,
                   const fa8_tensor *sink, float softmax_scale, int num_splits,
                   void *workspace, size_t workspace_bytes, void *stream);

/*
 * fa8_fwd_workspace_size -- validates the shape arguments of fa8_fwd (no data is read)
 * and reports the split count fa8_fwd would use and the workspace it needs.
 * Either output pointer may be NULL.
 */
FA8_API fa8_status fa8_fwd_workspace_size(const fa8_tensor *q, const fa8_tensor *k,
                                  const fa8_tensor *v, const fa8_tensor *cu_seqlens_q,
                                  const fa8_tensor *cu_seqlens_k, const fa8_tensor *block_table,
                                  int page_size, int num_splits, int *splits_out,
                                  size_t *bytes_out);

/*
 * fa8_fwd_plan -- the launch plan fa8_fwd would use on a device with `sm_count` SMs,
 * computed on the host only (no CUDA call): the split count, the workspace bytes and the
 * forward's work grid (grid_out[0] = Q-tile slots, grid_out[1] = kv_heads x splits; the
 * prefill kernel for dv <= 128 is persistent and walks these units with min(units, SMs)
 * CTAs).  It runs the same shape validation as fa8_fwd.  Any output pointer may be NULL.
 */
FA8_API fa8_status fa8_fwd_plan(const fa8_tensor *q, const fa8_tensor *k, const fa8_tensor *v,
                                const fa8_tensor *cu_seqlens_q, const fa8_tensor *cu_seqlens_k,
                                const fa8_tensor *block_table, int page_size, int num_splits,
                                int sm_count, int *splits_out, size_t *bytes_out,
                                int64_t *grid_out);

/*
 * fa8_fwd_static_scratch -- fa8_fwd without a caller-provided workspace.  The attention
 * it computes is fa8_fwd's, argument for argument; nothing in the published method
 * corresponds to this entry point, which only changes where the split partials live.
 *
 * Who it is for: callers that cannot hand the library a device buffer -- a runtime whose
 * device memory is carved up once at start-up and that may not allocate afterwards, or
 * plain C code that links only this library and has no allocator of its own.  Neither
 * this function nor anything it calls allocates or frees device memory.
 *
 * Where the partials go: one array of FA8_STATIC_SCRATCH_BYTES (32 MiB) of device memory
 * that the library declares statically, so it exists once per device for as long as the
 * library is loaded.  A call whose split plan (see fa8_fwd_workspace_size) needs more
 * than that returns FA8_ERR_WORKSPACE before anything is enqueued; lower num_splits or
 * use fa8_fwd with a workspace of your own.  Calls whose plan has one split do not touch
 * the array.  Nothing in it has to start at zero: every call writes each partial before
 * the merge kernel reads it.
 *
 * Sharing: every call on a device uses the same array.  Two calls that can run at the
 * same time on one device (different streams without an event between them, or different
 * host threads) overwrite each other's partials and give wrong results; order them on one
 * stream, or use fa8_fwd with separate workspaces.
 *
 * Set-up: the first call on each device, made with that device current, looks up the
 * array's device address (cudaGetSymbolAddress) and keeps it; make that first call
 * before capturing a stream.  A failure there returns FA8_ERR_CUDA.
 */
#define FA8_STATIC_SCRATCH_BYTES ((size_t)32 * 1024 * 1024)
FA8_API fa8_status fa8_fwd_static_scratch(const fa8_tensor *q, const fa8_tensor *k,
                                          const fa8_tensor *v, const fa8_tensor *descale_q,
                                          const fa8_tensor *descale_k,
                                          const fa8_tensor *descale_v, fa8_tensor *out,
                                          fa8_tensor *lse, const fa8_tensor *cu_seqlens_q,
                                          const fa8_tensor *cu_seqlens_k,
                                          const fa8_tensor *block_table, int page_size,
                                          int causal, int window_left, const fa8_tensor *sink,
                                          float softmax_scale, int num_splits, void *stream);

/* ------------------------------------------------------------------------------------
 * Around the paged cache: filling it, summarising its pages, choosing pages for each query,
 * and attention over the chosen pages.
 *
 * Shared conventions.  "New tokens" are the last Lq keys of each request: batched
 * (B, Sq, ...) or packed (total_q, ...) with cu_seqlens_q, as q in fa8_fwd; token i of a
 * request with Lk keys is its key Lk - Lq + i.  Where Lk < Lq (a padded slot may have no key)
 * the first tokens have no key: nothing is appended for them, and they see nothing when
 * causal = 1.  Output rows of a packed tensor behind the last sequence stay as they were.  A
 * tensor that a call writes must not have expanded dims.  A cu_seqlens_k or block_table entry
 * out of range raises FA8_ERR_DEVICE_BOUNDS in fa8_check and is never followed.  Every call
 * enqueues one kernel on `stream`, needs no workspace, allocates nothing, and its launch
 * depends on shapes and the SM count only, so it can be graph-captured.  Results do not depend
 * on timing: equal inputs give equal bits.
 * ------------------------------------------------------------------------------------ */

/* How fa8_rope_inv_freq stretches the frequencies w_i = base^(-2 i / rotary_dim). */
typedef enum {
    FA8_ROPE_PLAIN = 0,  /* w_i                                                            */
    FA8_ROPE_LINEAR = 1, /* w_i / factor (position interpolation)                          */
    FA8_ROPE_NTK = 2,    /* base * factor^(rotary_dim / (rotary_dim - 2)) in place of base */
    FA8_ROPE_YARN = 3,   /* w_i / factor where w_i makes fewer than `low` turns over
                            original_len, w_i above `high` turns, a ramp over the index i
                            between (YaRN; customary low = 1, high = 32)                   */
    FA8_ROPE_BANDS = 4   /* as YARN, with the ramp over the number of turns itself
                            (customary low = 1, high = 4)                                  */
} fa8_rope_scaling;

/*
 * fa8_rope_inv_freq -- host only: writes the rotary_dim / 2 frequencies (radians per
 * position) to inv_freq in host memory.  factor >= 1 is read by every scaling but PLAIN;
 * original_len, low and high by YARN and BANDS.
 */
FA8_API fa8_status fa8_rope_inv_freq(int rotary_dim, double base, int scaling, double factor,
                                     double original_len, double low, double high,
                                     double *inv_freq);

/*
 * fa8_rope_append -- rotates Q and K, rounds Q, K and V to E4M3 and stores them: Q in
 * q_out, K and V as the new tokens' keys in k_out / v_out.
 *   q (B, Sq, Hq, D) or (total_q, Hq, D); k (.., Hkv, D) and v (.., Hkv, DV) with the same
 *     leading dims; all bf16 or all fp16; last dim contiguous, strides multiples of 8
 *     elements (views of one projection output will do), 16-byte aligned.  (D, DV) as in
 *     fa8_fwd.
 *   q_out: E4M3, q's shape.  k_out / v_out: E4M3, in any of fa8_fwd's K/V layouts; with
 *     batched k_out (B, Sk, ..) the new tokens are the last Sq of Sk.
 *   inv_freq: fp64 or fp32, (rotary_dim / 2) on the device; rotary_dim a multiple of 16.
 *     Dims [rotary_offset, rotary_offset + rotary_dim) of every head are rotated, the rest
 *     pass through; rotary_offset is a multiple of 8.  Pair i is dims (i, i + rotary_dim/2)
 *     of that range, or (2 i, 2 i + 1) when interleaved = 1.
 *   positions: int32, one per token, any strides; NULL = the token's key index.  The angle
 *     of pair i is position * inv_freq[i], reduced exactly at every position.
 *   rot_scale multiplies the rotated dims (YaRN's attention factor; 1 otherwise).
 *   descale_q/k/v: as in fa8_fwd, 2^-124 or more; out = e4m3(x / descale), round to nearest
 *     even (of the fp32 quotient, which keeps what is halfway between two values while the
 *     descale is below 2^100), saturating at +-448 (infinities too); NaN stays NaN.
 * The outputs must not overlap the inputs, and no two tokens may share a cache slot.
 */
FA8_API fa8_status fa8_rope_append(const fa8_tensor *q, const fa8_tensor *k, const fa8_tensor *v,
                                   const fa8_tensor *inv_freq, const fa8_tensor *positions,
                                   int interleaved, int rotary_offset, float rot_scale,
                                   const fa8_tensor *descale_q, const fa8_tensor *descale_k,
                                   const fa8_tensor *descale_v, fa8_tensor *q_out,
                                   fa8_tensor *k_out, fa8_tensor *v_out,
                                   const fa8_tensor *cu_seqlens_q, const fa8_tensor *cu_seqlens_k,
                                   const fa8_tensor *block_table, int page_size, void *stream);

/*
 * fa8_page_bounds -- per page, kv-head and channel, the smallest and the largest key:
 * bounds[page, h, 0, c] = min and bounds[page, h, 1, c] = max over the page's keys of the
 * request (rows past its Lk are ignored).  Exact: E4M3 values in, E4M3 values out.  A
 * channel with a NaN key has NaN bounds.
 *   k: paged (num_pages, page_size, Hkv, D); D a multiple of 16 up to 256.
 *   bounds: E4M3 (num_pages, Hkv, 2, D), last two dims contiguous, 16-byte strides.
 *   Updated are the pages that hold a new key: of each request's last Lq keys when
 *   cu_seqlens_q is given, else of its last `new_tokens` keys, or all its pages when
 *   new_tokens < 0.  A page is recomputed whole.  Other pages keep what they hold.
 * Requests that share a page (a common prefix) must both fill it.
 */
FA8_API fa8_status fa8_page_bounds(const fa8_tensor *k, fa8_tensor *bounds,
                                   const fa8_tensor *cu_seqlens_q, const fa8_tensor *cu_seqlens_k,
                                   const fa8_tensor *block_table, int page_size, int new_tokens,
                                   void *stream);

/*
 * fa8_select_pages -- for every new token and kv-head, the top_k pages that can hold the
 * largest scores: score(page) = max over the kv-head's q-heads of
 * sum_c max(q_c * lo_c, q_c * hi_c), an upper bound of q . key over the page.
 *   q: E4M3 (B, Sq, Hq, D) or (total_q, Hq, D); D in {64, 96, 128, 192, 256}.
 *   bounds: as fa8_page_bounds writes them.
 *   pages: int32 (B, Sq, Hkv, top_k) or (total_q, Hkv, top_k), last dim contiguous: page
 *     indices of the request (positions in its block_table row), ascending, -1 behind the
 *     last.
 * Candidates are the n pages with a key the token sees (all of the request's when
 * causal = 0, keys up to its own when causal = 1); n <= top_k lists them all.  The first
 * keep_first and the last keep_last of them are always listed (their sum is at most
 * top_k); the rest goes by score.  Scores are compared exactly, as the real numbers that
 * the formula gives, and ties go to the lower page; a NaN score ranks above all others.
 * At most 16384 block_table columns; top_k 1 to 4096.
 */
FA8_API fa8_status fa8_select_pages(const fa8_tensor *q, const fa8_tensor *bounds,
                                    fa8_tensor *pages, const fa8_tensor *cu_seqlens_q,
                                    const fa8_tensor *cu_seqlens_k, const fa8_tensor *block_table,
                                    int page_size, int causal, int keep_first, int keep_last,
                                    void *stream);

/*
 * fa8_fwd_pages -- fa8_fwd over the keys of listed pages only: token t's q-heads of kv-head
 * h attend to the keys of pages[t, h, :] that the token sees (causal or all, below Lk).
 *   q, k, v (paged), descales, out, lse, sink, softmax_scale, causal: as in fa8_fwd.
 *   pages: int32, as fa8_select_pages writes them.  Any order will do; entries below 0 are
 *     skipped, a page listed twice counts twice, and a page with no visible key adds
 *     nothing.  At most 4096 per token and kv-head.
 *   page_size: a multiple of 8 up to 4096.
 * Tokens with no visible listed key get O = 0 and LSE = -inf (the sink's logit with a
 * sink).  What the pool holds in rows that are not visible does not matter.
 */
FA8_API fa8_status fa8_fwd_pages(const fa8_tensor *q, const fa8_tensor *k, const fa8_tensor *v,
                                 const fa8_tensor *pages, const fa8_tensor *descale_q,
                                 const fa8_tensor *descale_k, const fa8_tensor *descale_v,
                                 fa8_tensor *out, fa8_tensor *lse, const fa8_tensor *cu_seqlens_q,
                                 const fa8_tensor *cu_seqlens_k, const fa8_tensor *block_table,
                                 int page_size, int causal, const fa8_tensor *sink,
                                 float softmax_scale, void *stream);

/*
 * fa8_check -- reads the library's device status word of the current device on `stream`
 * (ordered after the work enqueued there), waits for that read, and clears the word if it
 * was set: FA8_SUCCESS, FA8_ERR_DEVICE_TIMEOUT (a kernel gave up a bounded wait and
 * returned early; its outputs are undefined) or FA8_ERR_DEVICE_BOUNDS.
 *
 * The status word is one per device, shared by every stream and host thread that calls the
 * library on that device: a kernel on any stream sets its bits, and a check on any stream
 * reads and clears them all.  So a check may report (and clear) an error raised by another
 * stream's work, and work still running on another stream may set the word after the read.
 * Callers that run forwards on several streams at once and need to know which call failed
 * should check from one place after joining the streams.
 */
FA8_API fa8_status fa8_check(void *stream);

/*
 * fa8_set_decode_kernel -- 1 (the default): shapes with batched q and at most 16 query rows
 * per kv-head (Sq x Hq/Hkv <= 16, Hq/Hkv dividing 16, dv a multiple of 128) run the decode
 * kernel, which puts the keys of a tile on the MMA's M dimension and the few query rows on
 * N; 0: every shape runs the 128-row forward kernel.  Both compute the same attention (not
 * bit-identically).  A process-wide setting, safe to change from any host thread: each
 * fa8_fwd call reads it once, so one call uses one setting throughout.
 */
FA8_API fa8_status fa8_set_decode_kernel(int enable);

/* Sets the bound on every in-kernel wait (nanoseconds; default 2e9, minimum 1e5); a
 * process-wide setting, read once by each later fa8_fwd call, safe from any host thread. */
FA8_API fa8_status fa8_set_wait_timeout_ns(uint64_t ns);

/*
 * fa8_debug_wait_probe -- DEBUG ONLY.  Launches a one-CTA kernel whose only work is a bounded wait on a
 * barrier that nothing completes, then returns fa8_check(stream).  It exists to test the
 * timeout path: with the default bound it returns FA8_ERR_DEVICE_TIMEOUT after ~2 s.
 */
FA8_API fa8_status fa8_debug_wait_probe(void *stream);

/*
 * fa8_debug_set_trace_buffer -- in a library built with -DFA8_TRACE, later forward launches
 * record clock64() at each pipeline event (TMA issue, MMA issue, softmax and fold
 * hand-offs) of the first 8 CTAs into `device_buffer`, laid out [cta 8][event 16][tile 64]
 * as uint64 (needs 65536 bytes); NULL turns it off.  Other builds return
 * FA8_ERR_UNSUPPORTED.  DEBUG ONLY: for pipeline tuning with a trace build; production
 * builds do not record anything.
 */
FA8_API fa8_status fa8_debug_set_trace_buffer(void *device_buffer, size_t bytes);

FA8_API const char *fa8_status_string(fa8_status s);
/* Reason for the last error returned on the calling thread ("" if none). */
FA8_API const char *fa8_last_error(void);
FA8_API int fa8_version(void);

#ifdef __cplusplus
}
#endif

#endif /* FA8_H_ */
