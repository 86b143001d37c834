/*
 * kivi.h -- C ABI of libkivi: a KIVI-style quantized KV cache and its
 * decode-attention step, on one GB300 (sm_103a).
 *
 * Method (source: "Literature audit -- Group 2 (KV-cache compression primary
 * sources)", section 1 "KIVI -- kivi2024", list "Core algorithm
 * (implementation-grade)"):
 *   item 1  asymmetric round-to-nearest group quantizer, z = min,
 *           s = (max - min) / (2^B - 1), code = round((x - z) / s),
 *           B = 2 or 4 chosen separately for keys and values;
 *   item 2  keys quantized per channel in groups of G consecutive tokens;
 *   item 3  values quantized per token in groups of G channels;
 *   item 4  fp16 residual window of R tokens: prefill keeps the last t mod R
 *           keys and the last R values in fp16; during decode the fp16 key
 *           block is quantized whole when it holds R keys (R % G == 0) and
 *           the fp16 value queue pops and quantizes its oldest token when it
 *           holds R + 1;
 *   item 5  decode attention = softmax((q K_quant^T || q K_full^T) / sqrt(d))
 *           (V_quant || V_full).
 *
 * Conventions for every call:
 *   - tensor pointers are DEVICE pointers owned by the caller, read or
 *     written in stream order on `stream` (a cudaStream_t; 0 = legacy
 *     default stream).  Host-side arrays are named as such.
 *   - fp16 means IEEE binary16; tensors are dense, row-major, no padding.
 *   - every call validates all arguments before it changes anything; on an
 *     error nothing is launched and the cache is unchanged.
 *   - a CUDA error inside a call poisons the handle: later calls return
 *     KIVI_ERR_STATE (destroy still works).
 *   - calls on one handle are not thread-safe, and must not overlap on the GPU
 *     (two streams without an event between them, two captured graphs replayed
 *     at once): also the read-only ones share the handle's buffers.  Different
 *     handles are independent.
 *   - no call allocates device memory except kivi_cache_create,
 *     kivi_latent_create and a cache's first kivi_chunk_attn,
 *     kivi_prefill_attn_window or kivi_latent_attn that splits its work (see
 *     there).
 * Supported shapes: k_bits, v_bits in {2, 4}; G in {16, 32, 64, 128};
 * d in {64, 128, 256} with d % G == 0; R % G == 0 (item 4's assertion);
 * 1 <= b <= 1024; h_q a multiple of h_kv with h_q / h_kv <= 8.
 * Anything else returns KIVI_ERR_UNSUPPORTED.
 */
#ifndef KIVI_H
#define KIVI_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define KIVI_ABI_VERSION 6

typedef struct kivi_cache *kivi_cache_t;   /* opaque, library-owned */
typedef struct kivi_latent *kivi_latent_t; /* the same: a latent cache */
typedef struct CUstream_st *kivi_stream_t; /* the same type as cudaStream_t */

typedef enum {
    KIVI_OK = 0,
    KIVI_ERR_INVALID_ARG = 1,  /* null pointer, negative size, bad handle */
    KIVI_ERR_UNSUPPORTED = 2,  /* shape or bit width outside the list above */
    KIVI_ERR_CAPACITY = 3,     /* a sequence would exceed max_tokens */
    KIVI_ERR_STATE = 4,        /* handle poisoned by an earlier CUDA error */
    KIVI_ERR_CUDA = 5,         /* a CUDA call failed (see kivi_last_error) */
    KIVI_ERR_OOM = 6           /* device or host allocation failed */
} kivi_status;

/* Create an empty cache for b sequences of h_kv KV heads of dimension d,
 * holding up to max_tokens tokens per sequence; k_bits / v_bits per item 1,
 * group size G per items 2-3, residual length R per item 4.  All device
 * memory of the cache is allocated here (packed codes, fp16 scale/zero,
 * fp16 residual windows, counters, decode partials), but for the chunk
 * attention's partials.  *out receives the handle; release it with
 * kivi_cache_destroy. */
kivi_status kivi_cache_create(int b, int h_kv, int d, int k_bits, int v_bits, int G, int R,
                              int max_tokens, kivi_cache_t *out);

/* Free every resource of the cache.  The handle is invalid afterwards;
 * passing it to any call returns KIVI_ERR_INVALID_ARG. */
kivi_status kivi_cache_destroy(kivi_cache_t c);

/* Prefill (item 4): reset every sequence and fill it from K and V, fp16
 * [b][h_kv][t_stride][d] (device).  Sequence i takes its first t[i] tokens
 * (t: HOST array of b int32, 0 <= t[i] <= t_stride, t[i] <= max_tokens).
 * Keys [0, t - t mod R) and values [0, max(t - R, 0)) are quantized; the
 * rest stays fp16.  Reads K and V in stream order; they may be freed or
 * reused once the stream has passed this call. */
kivi_status kivi_prefill(kivi_cache_t c, const void *K, const void *V, const int32_t *t,
                         int t_stride, kivi_stream_t stream);

/* Prefill with its attention: kivi_prefill(K, V, t, t_stride) and, from
 * the same pass over K and V, the prompt's causal attention in full
 * precision ("Literature audit -- Group 2", section 1 KIVI: its backends
 * list runs the prefill's attention on the unquantized K/V and quantizes
 * the cache after it; its limitations paragraph lists that unfused
 * quantization as open).  For sequence i, query head h (kv head
 * h / (h_q / h_kv)) and token tau < t[i]:
 *   out[i][h][tau] = sum_{s <= tau} softmax_s(q[i][h][tau] . K[i][j][s] / sqrt(d)) V[i][j][s]
 * q and out: fp16 [b][h_q][t_stride][d] (device, 16-byte aligned); rows
 * tau >= t[i] of out are not written.  The cache afterwards is bitwise the
 * one kivi_prefill leaves.  Scores accumulate in fp32; the softmax weights
 * enter the weighted sum of values rounded to fp16.  One launch.  Supports
 * d 64 or 128 and G <= 64 (KIVI_ERR_UNSUPPORTED otherwise); h_q a multiple
 * of h_kv, at most 8 times it. */
kivi_status kivi_prefill_attn(kivi_cache_t c, const void *q, const void *K, const void *V, const int32_t *t,
                              int t_stride, int h_q, void *out, kivi_stream_t stream);

/* Sliding windows with sinks (kivi_prefill_attn_window,
 * kivi_decode_attn_window, kivi_chunk_attn): with window > 0 the query at
 * position p sees, of the tokens s <= p, those with p - s < window and the
 * sequence's first `sinks` tokens (s < sinks).  window == 0: every token
 * s <= p, whatever sinks says.  A token always sees itself.  Neither may be
 * negative (KIVI_ERR_INVALID_ARG).  Inputs are finite also where they are
 * hidden. */

/* kivi_prefill_attn with a sliding window: out is the windowed attention of
 * the prompt; the cache afterwards is the same (it takes every token).  Key
 * tiles that no query of a tile sees are neither read nor multiplied.  With
 * window > 0 several launches, which use the cache's buffer as
 * kivi_chunk_attn's do, and its limits: any G; t_stride <= 2^26, b h_kv
 * t_stride below 2^31. */
kivi_status kivi_prefill_attn_window(kivi_cache_t c, const void *q, const void *K, const void *V, const int32_t *t,
                                     int t_stride, int h_q, int window, int sinks, void *out,
                                     kivi_stream_t stream);

/* Attention of a chunk of new tokens over the cache as it stands and over
 * the chunk itself: the next piece of a long prompt, or the tokens of a
 * speculative step.  Sequence i brings n[i] tokens (n: HOST array of b
 * int32, 0 <= n[i] <= n_stride) at positions T_i, T_i + 1, ...: K and V fp16
 * [b][h_kv][n_stride][d], q and out fp16 [b][h_q][n_stride][d] (device,
 * 16-byte aligned).  For token r < n[i], query head h (kv head
 * h / (h_q / h_kv)):
 *   out[i][h][r] = softmax over the visible tokens s <= T_i + r of the cache
 *                  (quantized, then fp16: item 5) and the chunk (fp16)
 * Rows r >= n[i] of out are not written; a sequence with n[i] = 0 is left
 * out.  Read-only on the cache: kivi_append_chunk appends the tokens, so a
 * rejected draft needs no undoing.  Scores accumulate in fp32; the restored
 * keys and values (scale code + zero) and the softmax weights are rounded to
 * fp16 before the products (|K|, |V| <= 32768, so that they stay finite; a
 * weight by 2^-11 of itself, or by 2^-32 of the row's largest): relative L2
 * error 4e-4 on even keys, up to 1.2e-3 where some channels are 8 times the
 * others (kivi_decode_attn 2e-4).
 * out overlaps no input.  One launch, or two when row tiles are split over
 * CTAs and joined (a call's result is repeatable bit for bit).
 * Splitting uses a buffer of the cache, which the first such call allocates
 * (2 x SMs x 256 rows of d + 2 floats, 40 MB at d = 128, or with up to 16 rows
 * a kv head a sixteenth of that; also while its stream is captured; without
 * the memory KIVI_ERR_OOM, and nothing changes) and the cache keeps.  A
 * captured call replays with the counts and positions it was captured with.
 * Supports d 64 or 128, n_stride <= 2^26 and b h_kv n_stride
 * below 2^31, while an SM's share of the work is below 2^31 key tiles (64
 * tokens for 256 rows; KIVI_ERR_UNSUPPORTED otherwise); h_q a multiple of
 * h_kv, at most 8 times it; the cache's device must be current
 * (KIVI_ERR_INVALID_ARG). */
kivi_status kivi_chunk_attn(kivi_cache_t c, const void *q, const void *K, const void *V, const int32_t *n,
                            int n_stride, int h_q, int window, int sinks, void *out, kivi_stream_t stream);

/* Append n[i] tokens to sequence i (0 leaves it as it is): K, V, n and
 * n_stride as for kivi_chunk_attn, any d.  The cache afterwards is bitwise
 * the one that n[i] calls of kivi_append for sequence i alone would leave.
 * KIVI_ERR_CAPACITY (and nothing changes) if a sequence would exceed
 * max_tokens.  K and V lie outside the cache.  Two launches at most, on
 * `stream`.  A captured call writes, when replayed, the tokens and counts of
 * the state that it was captured in: replay it only there. */
kivi_status kivi_append_chunk(kivi_cache_t c, const void *K, const void *V, const int32_t *n, int n_stride,
                              kivi_stream_t stream);

/* Rotary positions of queries and keys, before they enter the calls above.
 * Channel pair m < rot_dim / 2 of a token at position p turns by the angle
 * p w_m: (x, y) -> factor (x cos - y sin, y cos + x sin).  interleaved == 0:
 * pair m is channels (m, m + rot_dim / 2); else (2 m, 2 m + 1).  Channels
 * from rot_dim on are copied.  inverse != 0 applies the transposed map (the
 * angle negated): the gradient with respect to the input.
 * q, q_out fp16 [b][h_q][n_stride][d], k, k_out fp16 [b][h_kv][n_stride][d]
 * (device, 16-byte aligned; an output may be its input, but not overlap it
 * otherwise; h_q or h_kv may be 0, its pointers are then not used).  Rows
 * r >= n[i] (n: HOST array of b int32) are not written.  The position of
 * token r of sequence i is pos0[i] + r (pos0: HOST array of b int32) or
 * pos[i][r] (pos: DEVICE int32 [b][n_stride]); one of the two is NULL.  Any
 * int32 position is valid.
 * turns (HOST, rot_dim / 2 entries): w_m as a fraction of a full turn in
 * fixed point, round(w_m / (2 pi) 2^64) mod 2^64; the angle is formed in
 * 64-bit integers, so far positions lose nothing.  Frequency scaling for
 * long contexts is a choice of the table (kivi.py: rope_frequencies).
 * Sines and products in fp32, results rounded once.  One launch on the
 * current device, no state.  Supports d 64, 128 or 256 and rot_dim a
 * multiple of 16, at most d (KIVI_ERR_UNSUPPORTED otherwise). */
kivi_status kivi_rope(const void *q, const void *k, int b, int h_q, int h_kv, int n_stride, int d, const int32_t *n,
                      const int32_t *pos0, const int32_t *pos, const uint64_t *turns, int rot_dim, int interleaved,
                      float factor, int inverse, void *q_out, void *k_out, kivi_stream_t stream);

/* kivi_rope with several axes (an image's or a film's tokens: time, height,
 * width): channel pair m turns by the angle p w_m with p the token's position on
 * axis[m] (axis: HOST, rot_dim / 2 entries below axes).  pos: DEVICE int32
 * [axes][b][n_stride]; any int32 position is valid.  1 <= axes <= 255; the rest
 * as there, inverse (the gradient) included.  Tokens that stand at the same
 * position on every axis (text) may go through kivi_rope. */
kivi_status kivi_rope_axes(const void *q, const void *k, int b, int h_q, int h_kv, int n_stride, int d,
                           const int32_t *n, const int32_t *pos, int axes, const uint8_t *axis, const uint64_t *turns,
                           int rot_dim, int interleaved, float factor, int inverse, void *q_out, void *k_out,
                           kivi_stream_t stream);

/* Verification of drafted tokens against the target's probabilities, after the
 * attention of a speculative step (kivi_chunk_attn, kivi_latent_attn) and before
 * the kept tokens are appended.  Sequence i drafted n[i] tokens (n: HOST array of
 * b int32, 0 <= n[i] <= n_stride), draft[i][r], from its own probabilities
 * q[i][r][:]; p[i][r][:] are the target's at the same place, p[i][n[i]][:] those
 * after the whole draft.  p: DEVICE [b][n_stride + 1][vocab], q: DEVICE
 * [b][n_stride][vocab], fp32 or fp16 (bytes = 4 or 2); q == NULL: a draft without
 * probabilities, each token certain.  u: DEVICE fp32 [b][n_stride + 1], uniform
 * numbers in [0, 1).
 *   Token r is kept while u[i][r] q[i][r][x] < p[i][r][x] (x = draft[i][r];
 *   exact; never for a token outside the vocabulary).  At the first that is not,
 *   one token is drawn from the weights max(p[i][r] - q[i][r], 0), or after n[i]
 *   kept ones from p[i][n[i]], by u[i][n_stride].  Probabilities count in units
 *   of 2^-40, rounded down (negative ones and NaN as 0, above 1 as 1); with W the
 *   sum of the weights the token is the lowest whose weights up to and with it
 *   exceed floor(floor(2^30 u) W / 2^30).  No weight left: drawn from p; none
 *   there either: no token, -1.
 * accepted[i] (DEVICE int32 [b]) is the number of kept tokens; tokens[i] (DEVICE
 * int32 [b][n_stride + 1]) they, the drawn one behind them, then -1.  Only the
 * row that is drawn from is read whole.  Outputs overlap no input.  One launch on
 * the current device, no state.  vocab and n_stride up to 2^20. */
kivi_status kivi_verify(const void *p, const void *q, int bytes, const int32_t *draft, const float *u, int b,
                        int n_stride, int vocab, const int32_t *n, int32_t *tokens, int32_t *accepted,
                        kivi_stream_t stream);

/* Latent attention: keys and values of every head are products of one latent
 * vector c_s [r] a token, and a rotary key kr_s [64] is shared by the heads.  Head
 * e has Wk_e, Wv_e [128][r]; a query is qn [128] and qr [64]:
 *   out_p = Wv_e sum_{s <= p} softmax_s(scale (qn . Wk_e c_s + qr . kr_s)) c_s.
 * The cache holds c and kr; the newest R tokens' c in fp16, older ones' quantized
 * as the KIVI values are (items 1 and 3: per token in groups of G channels), kr in
 * fp16.  Two forms, the same sums:
 *   absorbed (steps and chunks over the cache):
 *     ql = kivi_head_product(qn, Wk, transposed), kivi_latent_attn(ql, qr) -> ol,
 *     out = kivi_head_product(ol, Wv);
 *   expanded (whole prompts): K, V = kivi_head_product(c of all heads, Wk, Wv),
 *     kivi_latent_prompt_attn(qn, qr, K, kr, V), and kivi_latent_prefill.
 * (Or kivi_latent_product and kivi_latent_expanded, which kivi_latent_check covers.)
 * ql, ol, K and V are fp16: a query's Wk_e^T qn, or a token's Wk_e c_s and Wv_e c_s,
 * must stay below 65504, or the output is not finite (no flag tells).
 * Handles are as kivi_cache_t: not thread-safe, no two calls on one at once on the
 * GPU, poisoned by a CUDA error; the cache's device must be current
 * (KIVI_ERR_INVALID_ARG).
 *
 * kivi_latent_create: an empty cache for b sequences of up to max_tokens tokens.
 * r 256 or 512; bits 2 or 4; G 32, 64 or 128; R a positive multiple of 64 (R >=
 * max_tokens: nothing is quantized); b <= 1024 (KIVI_ERR_UNSUPPORTED
 * otherwise).  All device memory is allocated here but for kivi_latent_attn's
 * partials. */
kivi_status kivi_latent_create(int b, int r, int bits, int G, int R, int max_tokens, kivi_latent_t *out);
kivi_status kivi_latent_destroy(kivi_latent_t c);

/* Fill (every sequence starts anew with t[i] tokens) and append (n[i] more, 0
 * leaves a sequence as it is): C fp16 [b][stride][r], Kr fp16 [b][stride][64]
 * (device, 16-byte aligned), t and n HOST arrays of b int32 in [0, stride].
 * Afterwards tokens [0, T - R) are quantized, whatever calls brought them.  Inputs
 * finite.  KIVI_ERR_CAPACITY (and nothing changes) if a sequence would exceed
 * max_tokens; stride <= 2^26.  One launch.  A captured append writes, when
 * replayed, at the positions of the state that it was captured in: replay it only
 * there. */
kivi_status kivi_latent_prefill(kivi_latent_t c, const void *C, const void *Kr, const int32_t *t, int t_stride,
                                kivi_stream_t stream);
kivi_status kivi_latent_append(kivi_latent_t c, const void *C, const void *Kr, const int32_t *n, int n_stride,
                               kivi_stream_t stream);

/* The absorbed attention of n[i] new tokens of each sequence (positions T_i,
 * T_i + 1, ...) over the cache as it stands and over themselves; read-only on the
 * cache.  q fp16 [b][h][n_stride][r] (absorbed), q_rope fp16 [b][h][n_stride][64],
 * C, Kr, n as for kivi_latent_append; out fp16 [b][h][n_stride][r] = sum of the
 * weights times c, rows past n[i] not written; out overlaps no input.  scale is
 * positive.  Restored latent vectors and weights are rounded to fp16 before the
 * products (2^-11 of themselves, a weight or 2^-32 of the row's largest), sums in
 * fp32, |restored c| below 65504.  One launch, or two where row tiles are cut and
 * joined (repeatable bit for bit): the first such call allocates a buffer that the
 * cache keeps (2 x SMs x 64 rows of r + 2 floats, 40 MB at r = 512; also while its
 * stream is captured; without the memory KIVI_ERR_OOM).  A captured call replays
 * with the counts it was captured with.  1 <= h <= 128, n_stride h < 2^24,
 * b n_stride < 2^31 (KIVI_ERR_UNSUPPORTED otherwise). */
kivi_status kivi_latent_attn(kivi_latent_t c, const void *q, const void *q_rope, const void *C, const void *Kr,
                             const int32_t *n, int n_stride, int h, float scale, void *out, kivi_stream_t stream);

/* The expanded form over a cache, for long chunks: kivi_latent_rows writes, of each
 * sequence with new tokens (n[i] > 0), the cached rows as attention sees them and the
 * new ones behind them, into C_out fp16 [b][s_stride][r] and Kr_out fp16
 * [b][s_stride][64] (device; either may be NULL; T_i + n[i] <= s_stride; other rows
 * not written); heads' keys and values are then formed of C_out, and
 * kivi_latent_expanded_attn attends to them.  C, Kr, n as for kivi_latent_append. */
kivi_status kivi_latent_rows(kivi_latent_t c, const void *C, const void *Kr, const int32_t *n, int n_stride, void *C_out,
                             void *Kr_out, int s_stride, kivi_stream_t stream);

/* Tokens of each sequence, and how many of them are quantized (HOST arrays of b
 * int32; either may be NULL); the cache's rows as attention sees them, into C fp16
 * [b][t_stride][r] and Kr fp16 [b][t_stride][64] (device; either may be NULL; rows
 * past T_i not written); the status word, as kivi_cache_check. */
kivi_status kivi_latent_lengths(kivi_latent_t c, int32_t *T, int32_t *Tq);
kivi_status kivi_latent_restore(kivi_latent_t c, void *C, void *Kr, int t_stride, kivi_stream_t stream);
kivi_status kivi_latent_check(kivi_latent_t c, uint32_t *flags, kivi_stream_t stream);

/* A matrix of each head times rows of its own (h_x = h) or of all heads alike
 * (h_x = 1): x fp16 [b][h_x][n_stride][K], out fp16 [b][h][n_stride][N], for the
 * tokens s < n[i] (n: HOST array of b int32):
 *   out[i][e][s] = W_e x[i][e or 0][s],
 * w fp16 [h][N][K], or with transposed != 0 [h][K][N] (device, all 16-byte
 * aligned).  Sums in fp32, rounded once (beyond 65504: infinite).  Rows past n[i] are
 * neither read nor written; out overlaps no input.  One launch on the current device, no
 * state.  K a multiple of 64, N of 128, up to 16384; h <= 1024, b <= 1024, up to 2^30
 * tokens in all (KIVI_ERR_UNSUPPORTED otherwise). */
kivi_status kivi_head_product(const void *x, const void *w, int b, int h_x, int h, int n_stride, const int32_t *n,
                              int K, int N, int transposed, void *out, kivi_stream_t stream);

/* The expanded attention of prompts: q fp16 [b][h][t_stride][128], q_rope fp16
 * [b][h][t_stride][64], K and V fp16 [b][h][t_stride][128], Kr fp16
 * [b][t_stride][64], out fp16 [b][h][t_stride][128]; for token p < t[i] (t: HOST
 * array of b int32) causal over the tokens s <= p, scale as above.  Rows past t[i]
 * of out are not written, of the inputs may hold anything.  Weights are rounded to
 * fp16 (2^-11, or 2^-32 of the row's largest), sums in fp32.  out overlaps no input.
 * One launch on the current device, no state.  h <= 1024, t_stride <= 2^26, b h
 * t_stride < 2^31 (KIVI_ERR_UNSUPPORTED otherwise). */
kivi_status kivi_latent_prompt_attn(const void *q, const void *q_rope, const void *K, const void *Kr, const void *V,
                                    int b, int h, const int32_t *t, int t_stride, float scale, void *out,
                                    kivi_stream_t stream);

/* The same for n[i] queries of each sequence behind T[i] tokens (T, n: HOST arrays of
 * b int32): q, q_rope and out [b][h][n_stride][..], K and V [b][h][s_stride][128], Kr
 * [b][s_stride][64]; the query r < n[i] stands at position T[i] + r, T[i] + n[i] <=
 * s_stride.  Limits as above, for both strides. */
kivi_status kivi_latent_expanded_attn(const void *q, const void *q_rope, const void *K, const void *Kr, const void *V,
                                      int b, int h, const int32_t *T, const int32_t *n, int n_stride, int s_stride,
                                      float scale, void *out, kivi_stream_t stream);

/* kivi_head_product and kivi_latent_expanded_attn (T NULL: none, as
 * kivi_latent_prompt_attn with t = n) for the b sequences of a cache: the same, but a
 * wait that runs out shows in kivi_latent_check of the cache, not in kivi_device_check,
 * and the cache's device must be current. */
kivi_status kivi_latent_product(kivi_latent_t c, const void *x, const void *w, int h_x, int h, int n_stride,
                                const int32_t *n, int K, int N, int transposed, void *out, kivi_stream_t stream);
kivi_status kivi_latent_expanded(kivi_latent_t c, const void *q, const void *q_rope, const void *K, const void *Kr,
                                 const void *V, int h, const int32_t *T, const int32_t *n, int n_stride, int s_stride,
                                 float scale, void *out, kivi_stream_t stream);

/* As kivi_cache_check, for the current device's calls that have no handle
 * (kivi_head_product, kivi_latent_prompt_attn, kivi_latent_expanded_attn): one word
 * for all streams and threads, cleared by the call that reads it. */
kivi_status kivi_device_check(uint32_t *flags, kivi_stream_t stream);

/* Append one token to every sequence: k and v fp16 [b][h_kv][d] (device).
 * First, per sequence, the maintenance of item 4 left over from the previous
 * step: the fp16 key block is quantized if it holds R keys, and the oldest
 * fp16 value is popped and quantized if the queue holds R + 1.  Then k and
 * v join the fp16 windows.  Returns KIVI_ERR_CAPACITY (and changes nothing)
 * if any sequence is full. */
kivi_status kivi_append(kivi_cache_t c, const void *k, const void *v, kivi_stream_t stream);

/* Decode attention (item 5) for every sequence and query head.  q fp16
 * [b][h_q][d] (device), out fp16 [b][h_q][d] (device, caller-owned);
 * query head i reads KV head i / (h_q / h_kv).  Scores are q.k / sqrt(d)
 * over the quantized keys followed by the fp16 keys, one softmax over both,
 * weights applied to the quantized then fp16 values; fp32 accumulation.
 * A sequence with no tokens gets an all-zero output.  Read-only on the
 * cache (the call can be repeated, with bitwise identical results).  Preconditions: inputs finite and
 * |q_c| * s < 65504 for every key scale s (the scaled query is staged in
 * fp16 for the tensor-core contraction).  The kernel is launched as a
 * programmatic dependent of the previous kernel on the stream: its blocks
 * may be placed and set up while that kernel finishes, but nothing in
 * global memory is read before it has completed, so stream order holds. */
kivi_status kivi_decode_attn(kivi_cache_t c, const void *q, int h_q, void *out,
                             kivi_stream_t stream);

/* kivi_decode_attn with a sliding window and sinks: the query is the newest
 * token's (position T_i - 1).  Blocks it does not see are not read.  With
 * window == 0 the call is kivi_decode_attn.  The cache's device must be
 * current (KIVI_ERR_INVALID_ARG). */
kivi_status kivi_decode_attn_window(kivi_cache_t c, const void *q, int h_q, int window, int sinks, void *out,
                                    kivi_stream_t stream);

/* Decode attention with each token's attention weight: out as
 * kivi_decode_attn computes it (bitwise the same), and, for sequence i,
 * query head h and token t < T_i, probs[(i h_q + h) ld + t] = the softmax
 * weight of token t in that head's attention (fp32, device; tokens in
 * sequence order, quantized and fp16 alike; a row's weights sum to 1).
 * Entries t >= T_i are left as they were.  mass (device, same layout, may
 * be NULL) accumulates the weights: mass[...] += probs[...] for t < T_i, so
 * that repeated steps sum each token's attention over decode steps.  That
 * sum is H2O's eviction score ("Literature audit -- Group 2 (KV-cache
 * compression primary sources)", section 4 "H2O (Heavy-Hitter Oracle)":
 * per head, each key's softmax weights added over the query rows seen so
 * far), and section 1 "KIVI" counts KIVI as orthogonal to, and combinable
 * with, such eviction.  Token positions are stable across appends, so mass
 * rows stay aligned.
 * ld >= 1 and ld >= every T_i; probs and mass 4-byte aligned and distinct
 * (KIVI_ERR_INVALID_ARG otherwise).  Two launches: the decode kernel writes
 * raw scores into probs, a second kernel turns them into weights. */
kivi_status kivi_decode_attn_probs(kivi_cache_t c, const void *q, int h_q, void *out, float *probs,
                                   float *mass, int64_t ld, kivi_stream_t stream);

/* One decode step in one call: kivi_append(k, v) then kivi_decode_attn(q,
 * h_q, out), once both sets of arguments have been validated (a failed call
 * changes nothing; KIVI_ERR_CAPACITY if a sequence is full).  The cache
 * afterwards is bitwise the one the two calls leave; out agrees with theirs
 * within the decode tolerance (the work may be split differently).
 *
 * With h_q / h_kv <= 4 and no more (sequence, kv head) pairs than twice
 * the GPU's SM count, the step is one kernel launch: the decode kernel
 * appends the token itself (item 4's one-token maintenance: the new key
 * and value, and the value token leaving the queue, quantized per token as
 * in kivi_append) for every sequence whose key window is not full.  On a
 * step where some sequence's key window is full (every R steps per
 * sequence) the append kernel first handles just those sequences (two
 * launches).  Otherwise the call launches the append kernel and then the
 * decode kernel (with many pairs the append kernel's parallel appends are
 * faster than appends spread over the persistent decode CTAs).  The
 * environment variable KIVI_FUSED_STEP=0 forces two launches, =1 the fused
 * kernel wherever h_q / h_kv <= 4.  kivi_decode_plan reports the call's
 * launches.  k and v must stay unchanged until the call's work on `stream`
 * completes (the fused kernel reads them). */
kivi_status kivi_append_decode(kivi_cache_t c, const void *k, const void *v, const void *q, int h_q,
                               void *out, kivi_stream_t stream);

/* Per-sequence token counts (HOST arrays of b int32; any may be NULL):
 * T total, Tqk quantized keys, Tqv quantized values.  The fp16 windows hold
 * T - Tqk keys and T - Tqv values.  Reads the host mirror; no sync. */
kivi_status kivi_cache_lengths(kivi_cache_t c, int32_t *T, int32_t *Tqk, int32_t *Tqv);

/* Byte sizes of the six arrays kivi_cache_export writes, in its order. */
kivi_status kivi_cache_export_sizes(kivi_cache_t c, size_t sizes[6]);

/* Copy the cache's contents into HOST buffers (sizes from
 * kivi_cache_export_sizes), in the packed format below, then synchronize
 * `stream`.  Any pointer may be NULL to skip that array.  (On the device
 * the first four arrays are stored interleaved as block records, see
 * kivi_cache_export_records; this call splits them apart on the host.)
 *   Kc  uint32 [b][h_kv][fcap/64][2 d k_bits]  key codes, 64-token blocks
 *   Ksz fp16   [b][h_kv][fcap/G][2][d]          key scale (row 0), zero (row 1)
 *   Vc  uint32 [b][h_kv][fcap/16][d v_bits / 2] value codes, 16-token blocks
 *   Vsz fp16   [b][h_kv][fcap/16][2][d/G][16]   value scale / zero per token
 *   Kf  fp16   [b][h_kv][R][d]                  fp16 keys, token tau at tau % R
 *   Vf  fp16   [b][h_kv][R+1][d]                fp16 values, tau at tau % (R+1)
 * fcap = max_tokens rounded up to a multiple of max(64, G).
 * Inside a key block kb, the word of lane L = 4g + t (g < 8, t < 4) and lane
 * word u = (2 j + hh) (k_bits/2) + wi (j < d/16, hh < 2, wi < k_bits/2) is
 * word (u/4) 128 + 4 L + u%4.  Its low 16 bits hold channel 16j + 8hh + 2t,
 * its high 16 bits that channel + 1, each packing along tokens: the field at
 * bits [r k_bits, (r+1) k_bits) of a half is token 64 kb + 8 (wi 16/k_bits
 * + r) + g (item 2's packing along the token axis, interleaved by 8).
 * Inside a value block vb, the word of lane L and lane word u = p nwv + w
 * (p < 2, w < nwv = d v_bits / 128) is word (u/cs) 32 cs + L cs + u%cs with
 * cs = min(4, d v_bits / 64).  Its low half holds token 16 vb + 2t + 8p,
 * its high half that token + 1, each packing along channels: the field at
 * bits [r v_bits, (r+1) v_bits) is channel 8 (w 16/v_bits + r) + g.
 * Fields of tokens not yet quantized are zero. */
kivi_status kivi_cache_export(kivi_cache_t c, void *Kc, void *Ksz, void *Vc, void *Vsz, void *Kf,
                              void *Vf, kivi_stream_t stream);

/* The packed arrays as the device stores them: one record per 64-token
 * block kb of each (sequence i, kv head j), records ordered [b][h_kv][fcap/64],
 * each record holding, back to back, in the element formats above:
 *   Kc block kb                      2 d k_bits words
 *   Ksz rows of the block's groups   [max(1, 64/G)][2][d] fp16 (G = 128: the
 *                                    rows of group kb/2, in both its records)
 *   Vc value blocks 4kb .. 4kb+3     4 (d v_bits / 2) words
 *   Vsz value blocks 4kb .. 4kb+3    4 [2][d/G][16] fp16
 * except that inside a record every scale or zero row is stored lane-major:
 * in a key row (d halves) channel c = 16 jj + 8 hh + 2 t + lo (t < 4,
 * lo < 2) sits at position t d/4 + 4 jj + 2 hh + lo, and in a value row (16
 * halves) token tau = 2 t + 8 p + lo sits at 4 t + 2 p + lo.
 * With records == NULL, writes the byte size of all records to *bytes.
 * Otherwise copies them into `records` (host or device memory, *bytes at
 * least that size; cudaMemcpyDefault), synchronizes `stream` and sets *bytes
 * to the size copied.  Errors: KIVI_ERR_INVALID_ARG (bytes NULL, buffer too
 * small). */
kivi_status kivi_cache_export_records(kivi_cache_t c, void *records, size_t *bytes,
                                      kivi_stream_t stream);

/* Synchronize `stream` and read the device status word into *flags (HOST).
 * 0 means no kernel recorded an anomaly; bit 0: a counter out of range,
 * bit 1: a bounded wait for a shared-memory copy ran out.  Clears it. */
kivi_status kivi_cache_check(kivi_cache_t c, uint32_t *flags, kivi_stream_t stream);

/* Kernel timing for measurement: when on, kivi_decode_attn records a pair
 * of CUDA events around its attention kernel(s) (up to 4096 pairs, then it
 * stops recording).  kivi_profile_read synchronizes them, returns the summed
 * milliseconds and the number of launches timed, and clears the record. */
kivi_status kivi_profile_enable(kivi_cache_t c, int on);
kivi_status kivi_profile_read(kivi_cache_t c, double *total_ms, int *launches);

/* How the last decode call (kivi_decode_attn, kivi_decode_attn_probs or
 * kivi_append_decode) was launched (HOST outputs, any may be NULL):
 * persistent CTAs of the decode kernel, and the call's launches of the
 * decode kernel (1) plus kivi_append_decode's append kernel when it
 * launched one (the weights' finalizing kernel is not counted). */
kivi_status kivi_decode_plan(kivi_cache_t c, int *splits, int *launches);

/* A packed cache held in caller-owned device memory: the block records
 * that kivi_cache_export_records documents, the fp16 windows Kf and Vf as
 * kivi_cache_export documents them (fcap as there), and the per-sequence
 * counters as DEVICE int32 arrays of b entries. */
typedef struct {
    int b, h_kv, d, k_bits, v_bits, G, R, max_tokens;
    const void *blocks, *Kf, *Vf;   /* device, 16-byte aligned */
    const int32_t *T, *Tqk, *Tqv;   /* device counters */
} kivi_packed_cache;

/* Decode attention that allocates nothing.  (The pages have no counterpart:
 * this is a library service for callers that cannot call cudaMalloc, e.g.
 * code running while a framework's memory pool owns the device memory, in
 * an allocator callback, or under a real-time budget that forbids device
 * allocation after start-up.)  Computes exactly what kivi_decode_attn
 * computes, over the cache described by *cache; q and out as there; the
 * shape rules are kivi_cache_create's.
 * Its scratch (split partials, merge tickets, status word) lives in one
 * fixed 16 MiB __device__ array inside the library; shapes whose scratch
 * b * h_q * P * (d + 4) * 4 bytes plus tickets exceed it (P: the most
 * persistent CTAs sharing one (sequence, kv head, head group)) are
 * rejected with KIVI_ERR_UNSUPPORTED and a kivi_last_error() message.  The
 * call launches on `stream` and clears the tickets itself; all calls share
 * the array, so calls whose kernels overlap on the GPU race and must not be
 * issued.  CUDA loads device code and __device__ arrays lazily: the first
 * call on a device loads the array (16 MiB of device memory, held until the
 * process exits) and looks up its device address (cudaGetSymbolAddress)
 * with that device current, and the first call of each shape (d, k_bits,
 * v_bits, G) loads that kernel's code.  So make one warm-up call per device
 * and shape before a memory pool takes the device memory, and before any
 * stream capture; later calls take no device memory.  After a
 * cudaDeviceReset the entry point must not be used (the looked-up address
 * is stale).  The kernel's status word is cleared by each call and not
 * reported: this path has no counterpart of kivi_cache_check.  No
 * cudaMalloc, cudaFree or other allocating routine is called. */
kivi_status kivi_decode_attn_noalloc(const kivi_packed_cache *cache, const void *q, int h_q,
                                     void *out, kivi_stream_t stream);

/* The launch plan kivi_decode_attn would use for a cache of this shape
 * (kivi_cache_create's rules; max_tokens sets the capacity) holding these
 * per-sequence counters (HOST arrays of b int32, 0 <= Tqk, Tqv <= T <=
 * max_tokens) for h_q query heads, on a GPU with num_sms SMs.  Host-only:
 * no CUDA call is made, so it runs without a GPU.  out (HOST, 6 int64):
 * persistent CTAs, warps per CTA, ring stages per warp, the most split
 * partials any (sequence, kv head, group of up to 4 query heads) receives,
 * the partial slots a cache of this shape holds for each, and the total
 * work units (a fully quantized 64-token block is one unit, any other
 * block a fixed larger weight).  The kernel requires partials <= slots. */
kivi_status kivi_plan_preview(int b, int h_kv, int d, int k_bits, int v_bits, int G, int R, int max_tokens,
                              int h_q, const int32_t *T, const int32_t *Tqk, const int32_t *Tqv, int num_sms,
                              int64_t out[6]);

const char *kivi_status_str(kivi_status s);
/* Text of the last error on the calling thread ("" if none). */
const char *kivi_last_error(void);
int kivi_abi_version(void);

#ifdef __cplusplus
}
#endif
#endif /* KIVI_H */
