/*
 * fa.h -- C ABI of the GB300 (sm_103a) FlashAttention-2 forward library.
 *
 * The operation is exact scaled-dot-product attention with an optional
 * causal mask and the per-row log-sum-exp:
 *
 *   O[b,h,i,:] = sum_j softmax_j( scale * Q[b,h,i,:] . K[b,h,j,:] ) V[b,h,j,:]
 *   LSE[b,h,i] = log sum_j exp( scale * Q[b,h,i,:] . K[b,h,j,:] )
 *
 * where j runs over all N keys, or over j <= i when causal.  It is computed
 * with the FlashAttention-2 forward recurrence: K/V tiles stream past an
 * on-chip Q tile, a running row max m and row sum l rescale an fp32 output
 * accumulator by exp(m_old - m_new), and the accumulator is divided by l once
 * at the end; the N x N score matrix is never written to memory.
 *
 * Sources (page title, section):
 *  - "FlashAttention 2 from PyTorch to Triton", What I am building: the
 *    recurrence, L = m + log(l) in natural-log units.
 *  - "A09 - Advanced Triton & FlashAttention", 3. Deep Dive: the rescaling
 *    update and its exactness; causal masking by block skipping.
 *  - "Building a Verifiable FlashAttention Forward from PyTorch to Triton",
 *    Scope: contiguous [B, H, N, D] self-attention, FP16/BF16, causal and
 *    non-causal, head dimension 64 or 128.
 *
 * Every call is asynchronous on the caller's stream and stream-ordered like a
 * kernel launch.  Nothing in this header throws.
 *
 * Device memory: calls that use the balanced schedule (below) need a
 * workspace for partial results -- per CTA two slots of [256, D] fp32 plus
 * (m, l) per row, and one int counter per (CTA tile, Q tile) -- about
 * 2 x 152 x 256 x (D + 2) x 4 bytes plus 8 bytes per 256 query rows per head.
 * It is allocated once per (device, stream) on the first such call, kept for
 * the life of the process, and reallocated larger (after synchronising that
 * stream) when a later call needs more; the counters are cleared with an
 * asynchronous memset when the buffer is new.  Calls on one stream share its
 * workspace in stream order; calls on different streams never share one.
 * Calls with the whole-tile schedule allocate nothing.
 */
#ifndef FA_GB300_H
#define FA_GB300_H

/* The library is built with hidden symbol visibility; only these entry
 * points are exported. */
#if defined(__GNUC__)
#define FA_API __attribute__((visibility("default")))
#else
#define FA_API
#endif

#include <stddef.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same type as cudaStream_t; 0 is the legacy default stream. */
struct CUstream_st;
typedef struct CUstream_st *fa_stream_t;

/* Element type of Q, K, V and O. */
typedef enum {
    FA_BF16 = 0,   /* bfloat16 */
    FA_FP16 = 1    /* IEEE binary16 */
} fa_dtype;

/*
 * Work decomposition over the persistent CTAs (one per SM).  A CTA tile is
 * 256 query rows of one head; a step is one 128-key tile of K and V.
 *  - FA_SCHEDULE_WHOLE_TILES: CTA c computes whole CTA tiles c, c + G, ...
 *  - FA_SCHEDULE_BALANCED: every CTA gets an equal share of all (tile, step)
 *    units; a tile cut by a share boundary is computed in parts whose partial
 *    results (O normalised per part, row max and sum) are merged by the last
 *    part to finish with the same rescaling rule the recurrence uses between
 *    key tiles ("A09 - Advanced Triton & FlashAttention", 3. Deep Dive).  This
 *    removes the idle SMs of a last partial wave of tiles.
 *  - FA_SCHEDULE_AUTO: the balanced schedule where it is expected to pay
 *    (non-causal calls whose shares span at least two tiles and whose last
 *    wave would leave SMs idle), whole tiles otherwise.
 * All three compute the same function; results agree to rounding.  The
 * pages describe one CTA per (Q tile, head) on a grid; these schedules are
 * this library's own.
 */
typedef enum {
    FA_SCHEDULE_AUTO = 0,
    FA_SCHEDULE_WHOLE_TILES = 1,
    FA_SCHEDULE_BALANCED = 2
} fa_schedule;

typedef enum {
    FA_OK = 0,
    FA_ERR_INVALID_VALUE = 1,      /* bad size, dtype, flag, scale, NULL, host pointer or overlapping output */
    FA_ERR_MISALIGNED = 2,         /* a pointer is not 16-byte aligned (the tensor-copy engine needs it) */
    FA_ERR_UNSUPPORTED_DEVICE = 3, /* no device, or the current device is not compute capability 10.3 */
    FA_ERR_CUDA = 4,               /* a CUDA runtime call or the launch failed */
    FA_ERR_DEVICE_TIMEOUT = 5,     /* a bounded in-kernel wait expired (reported by fa_sync_status) */
    FA_ERR_NO_ALLOC_LIMIT = 6      /* fa_fwd_noalloc: the call needs more than its static workspace */
} fa_status;

/*
 * fa_fwd -- attention forward for B*H independent heads.
 *
 * Q, K, V : device pointers to contiguous [B, H, N, D] tensors of `dtype`.
 *           They may alias one another (they are only read).
 * O       : device pointer to a contiguous [B, H, N, D] tensor of `dtype`;
 *           every element is written.  Must not overlap Q, K, V or LSE.
 * LSE     : device pointer to a contiguous [B, H, N] float32 tensor; row i
 *           receives log sum_j exp(scale * q_i . k_j) (natural log) over its
 *           visible keys.  Must not overlap Q, K, V or O.
 * B, H, N : batch, heads, sequence length (queries = keys = N); each >= 1 and
 *           B*H*N < 2^31.
 * D       : head dimension, 64 or 128.
 * causal  : 0 = every query sees all N keys; 1 = query i sees keys j <= i.
 *           Key tiles wholly above the diagonal are skipped, not masked.
 * scale   : softmax scale applied to q.k (usually 1/sqrt(D)); must be finite
 *           and > 0 (the kernel takes row maxima on unscaled scores).
 * stream  : CUDA stream the work is ordered on.
 *
 * All pointers belong to the caller and must stay valid until the work on
 * `stream` completes.  The device is the caller's current CUDA device.
 *
 * Returns FA_OK once the kernel is enqueued.  Argument errors are detected
 * before anything is enqueued and leave O and LSE untouched; FA_ERR_CUDA is
 * returned if a needed workspace cannot be allocated.  Errors raised inside
 * the kernel (a bounded wait that expired) are recorded in a per-device
 * status word and returned by fa_sync_status().
 *
 * fa_fwd uses FA_SCHEDULE_AUTO.
 */
FA_API fa_status fa_fwd(const void *Q, const void *K, const void *V, void *O, float *LSE,
                 int B, int H, int N, int D, int causal, float scale,
                 fa_dtype dtype, fa_stream_t stream);

/*
 * fa_fwd_ex -- fa_fwd with an explicit work decomposition `schedule` (see
 * fa_schedule); any other value returns FA_ERR_INVALID_VALUE.  A balanced
 * request the shape cannot take (more than 2^30 units of work) runs whole
 * tiles.
 */
FA_API fa_status fa_fwd_ex(const void *Q, const void *K, const void *V, void *O, float *LSE,
                    int B, int H, int N, int D, int causal, float scale,
                    fa_dtype dtype, fa_schedule schedule, fa_stream_t stream);

/*
 * fa_fwd_qkv -- fa_fwd_ex for Nq queries against Nkv keys per head: cross
 * attention, and decoding the last Nq positions of a longer sequence.
 *
 * Q, O : contiguous [B, H, Nq, D]; K, V : contiguous [B, H, Nkv, D];
 * LSE  : contiguous [B, H, Nq] float32.  Nq, Nkv >= 1, B*H*Nq < 2^31 and
 *        B*H*Nkv < 2^31; other arguments as for fa_fwd_ex.
 * causal: query i sees keys j <= i + (Nkv - Nq) -- aligned bottom-right, so
 *        the last query sees every key; with Nq = Nkv this is fa_fwd's mask.
 *        A query that sees no key (possible when Nq > Nkv) gets O = 0 and
 *        LSE = -inf.
 *
 * With few queries and many keys (decode) the balanced schedule splits each
 * head's keys over many CTAs and merges the partial results by their
 * log-sum-exp -- split-KV decoding; FA_SCHEDULE_AUTO picks it where it pays.
 * The pages fix only the square case; the bottom-right alignment is this
 * library's reading of the general one.
 */
FA_API fa_status fa_fwd_qkv(const void *Q, const void *K, const void *V, void *O, float *LSE,
                            int B, int H, int Nq, int Nkv, int D, int causal, float scale,
                            fa_dtype dtype, fa_schedule schedule, fa_stream_t stream);

/*
 * fa_fwd_band -- fa_fwd_qkv with a sliding-window (band) mask: with
 * i' = i + (Nkv - Nq), query i sees keys j in [i' - window_left,
 * i' + window_right]; a negative bound is unbounded on that side.  Causal is
 * (-1, 0), no mask (-1, -1), a causal window of W keys (W - 1, 0).  A query
 * whose band holds no key gets O = 0 and LSE = -inf.  Key tiles wholly
 * outside every row's band are skipped, not masked.  Other arguments as for
 * fa_fwd_qkv.
 */
FA_API fa_status fa_fwd_band(const void *Q, const void *K, const void *V, void *O, float *LSE,
                             int B, int H, int Nq, int Nkv, int D, int window_left, int window_right,
                             float scale, fa_dtype dtype, fa_schedule schedule, fa_stream_t stream);

/*
 * fa_fwd_sink -- causal attention in a sliding window whose first tokens stay
 * visible ("sinks"), with query heads that may share key heads.
 *
 * Q, O : contiguous [B, H, Nq, D];  K, V : contiguous [B, Hkv, Nkv, D], H a
 * multiple of Hkv, query head h reading key head floor(h / (H / Hkv));  LSE :
 * [B, H, Nq] float32.  With i' = i + (Nkv - Nq), query i sees the keys
 * j <= i' with j >= i' - window_left (window_left < 0: no bound) or
 * j < sinks.  A query that sees no key (i' < 0) gets O = 0 and LSE = -inf.
 * Key tiles (128 keys) that hold neither a sink nor a key of some row's window
 * are skipped, not masked.  What K holds at a key does not reach the queries
 * that do not see it; V must be finite in every tile that is visited, as a
 * hidden key's weight 0 still multiplies it.
 *
 * workspace : device memory, 16-byte aligned, of at least the bytes that
 *             fa_fwd_sink_workspace gives for the same arguments (0 where the
 *             schedule needs none; NULL is then fine).  It is the caller's:
 *             calls that may overlap, captured graphs among them, take
 *             different ones.  Its contents need no set-up.
 * Other arguments and errors as for fa_fwd_ex; B*H*Nq and B*Hkv*Nkv at most
 * 2^31 - 65536.
 */
FA_API fa_status fa_fwd_sink(const void *Q, const void *K, const void *V, void *O, float *LSE, int B, int H,
                             int Hkv, int Nq, int Nkv, int D, int window_left, int sinks, float scale,
                             fa_dtype dtype, fa_schedule schedule, void *workspace, size_t workspace_bytes,
                             fa_stream_t stream);

/* fa_fwd_sink_workspace -- bytes of workspace that fa_fwd_sink needs on the
 * current device for these arguments. */
FA_API fa_status fa_fwd_sink_workspace(int B, int H, int Hkv, int Nq, int Nkv, int D, int window_left, int sinks,
                                       fa_schedule schedule, size_t *bytes);

/*
 * fa_fwd_noalloc -- fa_fwd_ex that allocates no memory, device or host, at
 * any call.  The pages describe nothing like it: the method itself needs no
 * scratch, and this entry point only concerns where this library's balanced
 * schedule keeps its partial results.
 *
 * Who needs it: callers that cannot let a library allocate device memory on
 * their behalf -- a serving loop whose latency budget has no room for the
 * implicit device-wide synchronisation cudaMalloc / cudaFree may perform, or
 * a framework that owns every byte of device memory through its own pool and
 * forbids allocations behind its back.  fa_fwd_ex would allocate its
 * per-stream workspace on the first balanced call; this entry point instead
 * uses a workspace compiled into the library: a static device array of
 * FA_NOALLOC_WORKSPACE_BYTES per device.
 *
 * Set-up: the first call on a device looks up that array's address
 * (cudaGetSymbolAddress, which may load the library's code onto the device)
 * and keeps it; make that first call before any stream capture.  Every call
 * clears the partial-result counters (which must start at zero) with an
 * asynchronous memset on `stream`.
 *
 * Limit: with FA_SCHEDULE_AUTO, where the automatic plan would split tiles
 * into more partial results than the array holds, the call runs whole tiles
 * instead, which need no workspace.  A call with FA_SCHEDULE_BALANCED whose
 * schedule needs more workspace than the array holds returns
 * FA_ERR_NO_ALLOC_LIMIT before anything is enqueued.  The partial-result
 * slots always fit; the counters take 8 bytes per 256 query rows per head,
 * so B*H*ceil(N/256) may reach
 * 966,656 -- e.g. B*H = 256 at N = 965,000.  Whole-tile calls need no
 * workspace and have no limit.
 *
 * Overlapping calls race: there is one workspace per device, so two calls
 * whose work can overlap (on different streams, without ordering between
 * them) must not both run the balanced schedule; calls on one stream are
 * ordered and safe.  Arguments, results and other errors are as for
 * fa_fwd_ex.
 */
#define FA_NOALLOC_WORKSPACE_BYTES (48u << 20)
FA_API fa_status fa_fwd_noalloc(const void *Q, const void *K, const void *V, void *O, float *LSE,
                                int B, int H, int N, int D, int causal, float scale,
                                fa_dtype dtype, fa_schedule schedule, fa_stream_t stream);

/*
 * fa_bwd -- attention backward: the gradients of fa_fwd's O with respect to
 * Q, K and V for an upstream gradient dO, from the forward's O and LSE.
 *
 * Q, K, V, O, dO : device pointers to contiguous [B, H, N, D] tensors of
 *                  `dtype` (O and LSE as fa_fwd wrote them for the same Q, K,
 *                  V, causal and scale).  Only read; they may alias one
 *                  another.
 * LSE            : device pointer to contiguous [B, H, N] float32.
 * dQ, dK, dV     : device pointers to contiguous [B, H, N, D] tensors of
 *                  `dtype`; every element is written.  None may overlap an
 *                  input or another output.
 * B, H, N, D, causal, scale, dtype, stream : as for fa_fwd; B*H*ceil(N/128)*128
 *                  must stay below 2^31.
 *
 * With P = exp(scale * Q K^T - LSE) (0 where causal hides key j > query i)
 * and delta = rowsum(dO o O):  dV = P^T dO,  dS = P o (dO V^T - delta),
 * dQ = scale * dS K,  dK = scale * dS^T Q.  P and dS are rounded to `dtype`
 * for the tensor-core products, which accumulate in fp32.  P is recomputed
 * from LSE ("FlashAttention 2 from PyTorch to Triton", What I am building);
 * dK and dV are accumulated per key tile over the query tiles.  dQ (the
 * page's list of limitations: "by atomics or a second pass"):
 *  - D = 64: in the same pass, each key tile's dQ products added into an
 *    fp32 accumulator in global memory by tensor reductions (fp32 adds in
 *    L2), then scaled and rounded to `dtype`.  The order of those adds varies
 *    from call to call, so dQ may differ in its last bits between calls;
 *    dK and dV do not.
 *  - D = 128, and any call through fa_bwd_ex with FA_BWD_DETERMINISTIC: in a
 *    second pass over the key tiles, without atomics; bit for bit the same
 *    on every call.
 *
 * Scratch: 8 bytes per query row (rounded up to 128 rows per head) for delta
 * and LSE * log2(e), plus 4 * D bytes per such row for the dQ accumulator on
 * the D = 64 single pass, allocated per (device, stream) on first use like
 * the balanced schedule's workspace.  Errors as for fa_fwd; FA_ERR_CUDA if
 * the scratch cannot be allocated.
 */
FA_API fa_status fa_bwd(const void *Q, const void *K, const void *V, const void *O, const void *dO,
                        const float *LSE, void *dQ, void *dK, void *dV, int B, int H, int N, int D, int causal,
                        float scale, fa_dtype dtype, fa_stream_t stream);

/*
 * fa_bwd_band -- fa_bwd for Nq queries against Nkv keys under the band mask
 * of fa_fwd_band (window_left, window_right; a negative bound is unbounded;
 * causal = (-1, 0), no mask = (-1, -1)), from that call's O and LSE.
 *
 * Q, O, dO, dQ : contiguous [B, H, Nq, D];  K, V, dK, dV : contiguous
 * [B, H, Nkv, D];  LSE : [B, H, Nq] float32.  A query that sees no key
 * (LSE = -inf) contributes nothing and gets dQ = 0; a key that no query sees
 * gets dK = dV = 0.  Each key tile visits only the query tiles whose bands
 * reach it, and each query tile only the key tiles its rows' bands reach.
 * Other arguments as for fa_bwd; B*H*Nkv must stay below 2^31 as well.
 */
FA_API fa_status fa_bwd_band(const void *Q, const void *K, const void *V, const void *O, const void *dO,
                             const float *LSE, void *dQ, void *dK, void *dV, int B, int H, int Nq, int Nkv, int D,
                             int window_left, int window_right, float scale, fa_dtype dtype, fa_stream_t stream);

/* fa_bwd_ex flags. */
#define FA_BWD_DETERMINISTIC 1u /* dQ by the second pass at every D: the same bits on every call */

/*
 * fa_bwd_ex -- fa_bwd_band with `flags` (0 or FA_BWD_DETERMINISTIC; any other
 * bit: FA_ERR_INVALID_VALUE).  fa_bwd and fa_bwd_band are fa_bwd_ex with
 * flags = 0.
 */
FA_API fa_status fa_bwd_ex(const void *Q, const void *K, const void *V, const void *O, const void *dO,
                           const float *LSE, void *dQ, void *dK, void *dV, int B, int H, int Nq, int Nkv, int D,
                           int window_left, int window_right, float scale, fa_dtype dtype, unsigned int flags,
                           fa_stream_t stream);

/*
 * fa_bwd_sink -- the gradients of fa_fwd_sink, from that call's O and LSE.
 *
 * Q, O, dO, dQ : contiguous [B, H, Nq, D];  K, V, dK, dV : contiguous
 * [B, Hkv, Nkv, D], the gradients of a shared key head summed over its query
 * heads in fp32;  LSE : [B, H, Nq] float32.  A query that sees no key gets
 * dQ = 0; a key that no query sees dK = dV = 0.  Q, K, V, O and dO must be
 * finite in every tile that is visited.
 * flags : 0 or FA_BWD_DETERMINISTIC, as for fa_bwd_ex (dK and dV are the same
 *         bits on every call either way: a sink tile's query tiles are summed
 *         in parts, the parts added in a fixed order).
 * workspace : at least fa_bwd_sink_workspace bytes of device memory, 16-byte
 *         aligned, under the rules of fa_fwd_sink's.
 * Other arguments and errors as for fa_bwd.
 */
FA_API fa_status fa_bwd_sink(const void *Q, const void *K, const void *V, const void *O, const void *dO,
                             const float *LSE, void *dQ, void *dK, void *dV, int B, int H, int Hkv, int Nq, int Nkv,
                             int D, int window_left, int sinks, float scale, fa_dtype dtype, unsigned int flags,
                             void *workspace, size_t workspace_bytes, fa_stream_t stream);

/* fa_bwd_sink_workspace -- bytes of workspace that fa_bwd_sink needs on the
 * current device for these arguments. */
FA_API fa_status fa_bwd_sink_workspace(int B, int H, int Hkv, int Nq, int Nkv, int D, int window_left, int sinks,
                                       unsigned int flags, size_t *bytes);

/*
 * ---- A key/value cache held in 4 bits ----
 *
 * A cache holds, for K and for V, one packed row per token and key head:
 *   codes   [B, Hkv, C, D/2] bytes: D codes of 4 bits, the even channel in
 *           the low half of its byte;
 *   params  [B, Hkv, C, 2] of `dtype`: scale, minimum.
 * C is the capacity.  A row x of D values of type t = `dtype` is held as
 *   min = min_d x_d,  scale = t((max_d x_d - min) / 15),
 *   code_d = clamp(round_half_even((x_d - min) / scale), 0, 15), 0 if scale = 0
 * and stands for min + code_d * scale: D/2 + 4 bytes for 2 D, the values off
 * by at most half a scale, plus 15 roundings of the scale to t at the row's
 * upper end.  A row that holds an infinity or NaN stands for NaN throughout.
 * Kc and Vc are the codes, Kp and Vp the params.
 *
 * lens [B] (int32, device memory) gives each sequence's tokens in the cache;
 * values outside [0, C] are clamped to it.  It is read on the device, so a
 * captured graph follows its changes; rows behind a sequence's last token are
 * neither read nor written unless said otherwise.
 *
 * Arguments of all cache calls: device pointers to contiguous tensors;
 * B, Hkv, C >= 1; B*Hkv*C (B*Hkv*N, B*H*Nq) at most 2^31 - 65536; D = 64 or 128; codes, Q, K, V, O and
 * workspaces 16-byte aligned, everything else to its element (params 4).
 * Outputs overlap no other argument.  Errors as for fa_fwd, nothing enqueued
 * on any of them.  The calls allocate nothing and keep nothing between calls:
 * a workspace is the caller's, so calls that may overlap (other streams,
 * other captured graphs) take different ones.
 */

/*
 * fa_cache_append -- pack N new tokens per sequence into the cache.
 *
 * K, V  : [B, Hkv, N, D] of `dtype`; token i of sequence b becomes cache
 *         token start[b] + i.
 * start : [B] int32, device memory.
 * count : [B] int32, device memory, or NULL: token i of sequence b counts
 *         only if i < count[b] (a padded batch).  Tokens that do not count,
 *         or whose place lies outside [0, C), are not written.
 */
FA_API fa_status fa_cache_append(void *Kc, void *Kp, void *Vc, void *Vp, const void *K, const void *V,
                                 const int *start, const int *count, int B, int Hkv, int N, int C, int D,
                                 fa_dtype dtype, fa_stream_t stream);

/*
 * fa_cache_read -- the values that cache tokens start[b] .. start[b] + N - 1
 * stand for, rounded once to `dtype`, into K and V [B, Hkv, N, D].  Rows that
 * do not count (i >= count[b]) or lie outside [0, C) become zeros.
 */
FA_API fa_status fa_cache_read(const void *Kc, const void *Kp, const void *Vc, const void *Vp, void *K, void *V,
                               const int *start, const int *count, int B, int Hkv, int N, int C, int D,
                               fa_dtype dtype, fa_stream_t stream);

/* fa_cache_workspace -- bytes of workspace that fa_cache_fwd needs on the
 * current device for these sizes (0 for short caches). */
FA_API fa_status fa_cache_workspace(int B, int H, int Hkv, int Nq, int C, int D, size_t *bytes);

/*
 * fa_cache_fwd -- attention of each sequence's last Nq tokens against the
 * cache: decoding (Nq = 1), speculative decoding, or the end of a prompt.
 *
 * Q, O : [B, H, Nq, D] of `dtype`; H a multiple of Hkv, query head h reading
 *        key head floor(h / (H / Hkv)).  LSE : [B, H, Nq] float32.
 * Query i of sequence b sits at position p = lens[b] - Nq + i (its own key is
 * in the cache) and sees the tokens j <= p with j >= p - window_left
 * (window_left < 0: no bound) or j < sinks.  A query that sees no token
 * (p < 0) gets O = 0 and LSE = -inf.
 * workspace : fa_cache_workspace bytes (NULL where they are 0); its contents
 *        need no set-up.
 * The (H / Hkv) Nq query rows of a key head are taken 16 at a time, each block
 * with a pass of its own over the cache.
 *
 * K and V enter the products as their integer codes, exact in 16 bits, with
 * scale and minimum applied outside them in fp32; the softmax weight times V's
 * scale is rounded to 11 bits for the product with V's codes, to 22 for an
 * fp16 result.
 */
FA_API fa_status fa_cache_fwd(const void *Q, const void *Kc, const void *Kp, const void *Vc, const void *Vp,
                              const int *lens, void *O, float *LSE, int B, int H, int Hkv, int Nq, int C, int D,
                              int window_left, int sinks, float scale, fa_dtype dtype, void *workspace,
                              size_t workspace_bytes, fa_stream_t stream);

/*
 * fa_cache_weights -- what each cached token weighs in that attention, from
 * the LSE that fa_cache_fwd returned for the same arguments:
 *   w[b, h, j] = sum over the H/Hkv query heads of key head h and their Nq
 *                queries that see token j of exp(scale * q . k_j - LSE).
 * accumulate = 0: acc [B, Hkv, C] = w, every entry written (0 for tokens
 * that no query sees and behind lens[b]).  accumulate = 1: acc += w at the
 * tokens before lens[b]; the others are left as they are.  The sums have a
 * fixed order: the same bits on every call.
 */
FA_API fa_status fa_cache_weights(const void *Q, const void *Kc, const void *Kp, const float *LSE, const int *lens,
                                  float *acc, int accumulate, int B, int H, int Hkv, int Nq, int C, int D,
                                  int window_left, int sinks, float scale, fa_dtype dtype, fa_stream_t stream);

/*
 * fa_cache_evict -- bring every sequence down to at most `keep` tokens, in
 * another cache of capacity C2 >= keep: per key head the first `sinks`, the
 * last `recent` (sinks + recent <= keep) and, of those between them, the ones
 * with the largest acc [B, Hkv, C] (equal weights: the lowest position first;
 * -0 equals 0; NaN is below every number), in order of position.  A sequence
 * of at most `keep` tokens keeps them all.
 *
 * The kept tokens move together: the j-th of them is token j of the other
 * cache, and every later call counts positions, lengths, windows and sinks
 * there.  window_left then reaches back over that many kept tokens, however
 * far apart they once were, and hides the heavy ones before them: attention
 * that is to see every kept token takes no window.  To append
 * further tokens C2 must have room for them: a sequence that was cut fills the
 * first `keep` rows.
 *
 * Kc2, Kp2, Vc2, Vp2 : the other cache; rows behind the last kept token are
 *                      left as they are.
 * acc2  : [B, Hkv, C2] float32: the kept tokens' weights, then zeros.
 * lens2 : [B] int32: min(lens[b], keep).
 * index : [B, Hkv, keep] int32: the kept tokens' positions in the first
 *         cache, then -1.
 */
FA_API fa_status fa_cache_evict(const void *Kc, const void *Kp, const void *Vc, const void *Vp, const float *acc,
                                const int *lens, void *Kc2, void *Kp2, void *Vc2, void *Vp2, float *acc2,
                                int *lens2, int *index, int B, int Hkv, int C, int C2, int D, int keep, int sinks,
                                int recent, fa_stream_t stream);

/*
 * fa_sync_status -- synchronise `stream`, then return and clear the device
 * status word of the current device: FA_OK, FA_ERR_DEVICE_TIMEOUT if a kernel
 * gave up on a wait since the last call, or FA_ERR_CUDA if the synchronise
 * itself failed.
 *
 * The word is read and cleared in one atomic exchange by a one-thread kernel
 * on `stream`, so a timeout recorded meanwhile is never lost.  (One launch, one
 * copy and one wait a call.)  There is one word per device, shared by all
 * streams: a timeout from a kernel on another
 * stream is reported by whichever call reads the word first, and a timeout
 * from a kernel on another stream that has not finished yet is reported only
 * by a later call.  To attribute a timeout to a stream, synchronise the
 * others first.
 *
 * Device resets: the library keeps, per device, a lazily created workspace,
 * the status word and the static workspace's address.  A call that follows
 * cudaDeviceReset() on that device in the same process is not supported.
 */
FA_API fa_status fa_sync_status(fa_stream_t stream);

/* Static, NUL-terminated description of a status code. */
FA_API const char *fa_status_string(fa_status s);

#ifdef __cplusplus
}
#endif

#endif /* FA_GB300_H */
