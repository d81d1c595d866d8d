/*
 * lla.h — C ABI of the Looped Latent Attention (LLA) GPU library (liblla.so).
 *
 * LLA ("Looped Latent Attention: Cross-Loop KV Compression for Looped
 * Transformers", arXiv 2607.15456v2) replaces the per-loop K/V cache of a
 * weight-tied looped decoder (T loops, D layers, H heads of width d) by one K
 * latent and one V latent per token, layer and head, and rebuilds the loop-t
 * K/V only when attention reads them (§1, §3; §7 "latent-store path").  This
 * library is the data-parallel hot path of that latent-store decode:
 *
 *   lla_encode       Eq. (2)  c = (x - mu) W_down, written into cache slots
 *   lla_decode_attn  Eq. (3)  k_t = c_k W_up,k,t^T + mu_k,t (v likewise),
 *                    RoPE after reconstruction (§3 "RoPE and reconstruction"),
 *                    softmax(q.k/sqrt(d)) v over each sequence's history,
 *                    for one layer and one loop, all heads and sequences.
 *
 * Conventions shared by every call
 * --------------------------------
 * - Pointers marked "device" are CUDA device pointers owned by the caller;
 *   the library allocates nothing and keeps no per-call state.  "host"
 *   pointers are ordinary CPU memory.
 * - Arrays are dense and row-major, with the shapes given below.  Storage
 *   types follow lla_dims.dtype: LLA_BF16 stores latents, W, x and q as
 *   bfloat16 (mu always fp32); LLA_F32 stores everything as fp32.
 * - Every device pointer must be 16-byte aligned.
 * - Calls are asynchronous on `stream` (a cudaStream_t; NULL = legacy default
 *   stream).  Argument errors found on the host return before any launch.
 *   Values that live on the device (seq_lens, q_pos, seq_idx, pos) are
 *   checked by the kernels: an out-of-range value is clamped or its token
 *   skipped, and LLA_ERR_DEVICE_ARG is recorded in the workspace status word
 *   (read it with lla_device_status).  Every wait inside a kernel is bounded
 *   (about one second); on expiry the kernel records LLA_ERR_TIMEOUT and
 *   returns.
 * - The workspace is caller-allocated device memory of at least
 *   lla_workspace_size() bytes.  Its first 256 bytes hold the status word and
 *   must be zero before the first call; the rest is scratch.  Calls that
 *   share a workspace must be ordered on one stream.
 * - Test hook of the timeout path: while the 32-bit word at byte 4 of the
 *   workspace holds LLA_TEST_STALL, the per-head bf16 tile decode kernel
 *   ("tile" in lla_decode_kernel) waits on a barrier that one arrival short
 *   never completes; the wait expires after about one second and the call's
 *   status becomes LLA_ERR_TIMEOUT (outputs undefined).  Zero the word to
 *   resume normal calls.
 * - Constraints: d_head == 128; r_k and r_v multiples of 16 in [16, 256]
 *   (LLA_PER_HEAD) or [16, 512] (LLA_2D, one latent per token, "The LLA-2D
 *   variant"); T >= 1; H >= 1.  Other shapes return LLA_ERR_UNSUPPORTED.
 */
#ifndef LLA_H
#define LLA_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define LLA_ABI_VERSION 1

/* Value of workspace word 1 (byte offset 4) that makes the next tile decode
 * kernel's bounded wait expire (see the test hook above). */
#define LLA_TEST_STALL 0x4C415453u

typedef enum {
    LLA_OK = 0,
    LLA_ERR_INVALID_ARG = 1,   /* bad host-side argument: nothing launched       */
    LLA_ERR_UNSUPPORTED = 2,   /* valid but not implemented shape/variant/dtype  */
    LLA_ERR_CUDA = 3,          /* a CUDA runtime/driver call failed              */
    LLA_ERR_TIMEOUT = 4,       /* a kernel's bounded wait expired (device word)  */
    LLA_ERR_DEVICE_ARG = 5,    /* out-of-range seq_lens/q_pos/seq_idx/pos seen
                                  by a kernel (device word)                       */
    LLA_ERR_RANGE = 6          /* a folded query operand left the f16 range of
                                  the small-rank decode path, or is infinite in
                                  the 4-bit one (device word)                     */
} lla_status;

typedef enum { LLA_BF16 = 0, LLA_F32 = 1 } lla_dtype;

/* LLA_PER_HEAD: one latent per (token, layer, head) (§3 "Cross-loop codec").
 * LLA_2D: one latent per (token, layer) shared by all heads, reconstructing
 * every head (§3 "The LLA-2D variant"). */
typedef enum { LLA_PER_HEAD = 0, LLA_2D = 1 } lla_variant;

/* RoPE pairing: LLA_ROPE_HALF rotates (i, i + d/2); LLA_ROPE_INTERLEAVED
 * rotates (2i, 2i+1).  Frequencies theta_f = rope_base^(-2f/d). */
typedef enum { LLA_ROPE_HALF = 0, LLA_ROPE_INTERLEAVED = 1 } lla_rope_style;

typedef struct {
    int T;                      /* loops                                   */
    int H;                      /* heads                                   */
    int d_head;                 /* head width (must be 128)                */
    int r_k, r_v;               /* latent ranks                            */
    lla_variant variant;
    lla_dtype dtype;
    float rope_base;            /* e.g. 10000                              */
    lla_rope_style rope_style;
} lla_dims;

/* One layer's latent cache (device).  Per-head: k [B][H][L_max][r_k],
 * v [B][H][L_max][r_v]; element (b,h,j,i) of k at ((b*H+h)*L_max+j)*r_k+i.
 * LLA-2D: k [B][L_max][r_k], v [B][L_max][r_v]. */
typedef struct {
    void* k;
    void* v;
    int B;
    int64_t L_max;
} lla_cache;

/*
 * lla_encode — Eq. (2) of §3: for each of N tokens and each head,
 *     c_k = (x_k - mu_k) W_down,k ,  c_v = (x_v - mu_v) W_down,v
 * rounded to the cache dtype (round-to-nearest-even) and stored in cache slot
 * (seq_idx[n], pos[n]).  x is the loop stack of Eq. (1): index t*d+i.
 *   x_k, x_v        device  [N][H][T*d]      (LLA-2D: [N][T*H*d], index (t*H+h)*d+i)
 *   seq_idx, pos    device  int32 [N]        slot of token n; entries outside
 *                                            [0,B) x [0,L_max) are skipped and
 *                                            flagged LLA_ERR_DEVICE_ARG
 *   w_down_k/_v     device  [H][T*d][r]      (LLA-2D: [T*H*d][r])
 *   mu_k, mu_v      device  fp32 [H][T*d]    (LLA-2D: [T*H*d])
 * Used both for a decode step's new token and for prefill (N = all prompt
 * tokens of a layer).  Two tokens writing the same slot race.
 */
lla_status lla_encode(const lla_dims* dims, const void* x_k, const void* x_v, int N,
                      const int32_t* seq_idx, const int32_t* pos,
                      const void* w_down_k, const void* w_down_v,
                      const float* mu_k, const float* mu_v,
                      lla_cache cache, void* workspace, size_t ws_bytes, void* stream);

/*
 * lla_decode_attn — one layer, one loop t (0-based; the paper counts t=1..T),
 * all heads and all B sequences.  For sequence b with L = seq_lens[b] cached
 * tokens (positions 0..L-1) and a query at position q_pos[b]:
 *     k_j = c_k,j W_up,k,t^T + mu_k,t ,  v_j = c_v,j W_up,v,t^T + mu_v,t   (Eq. (3))
 *     s_j = RoPE(q, q_pos) . RoPE(k_j, j) / sqrt(d)   for j < L
 *     out = sum_j softmax(s)_j v_j ,  lse = ln sum_j exp(s_j)
 * mu_t is the t-th d-slice of the codec mean mu of Eq. (2).
 *   q              device  [B][H][d]               pre-RoPE query
 *   seq_lens       device  int32 [B]                0 <= L <= L_max (L=0: out=0, lse=-inf)
 *   q_pos          device  int32 [B]                0 <= q_pos < rope_len
 *   w_up_k, w_up_v device  [T][H][d][r]             all loops (LLA-2D: [T][H*d][r])
 *   mu_k, mu_v     device  fp32 [H][T*d]            (LLA-2D: [T*H*d])
 *   rope_cos/_sin  device  fp32 [rope_len][d/2]     cos/sin(p*theta_f) as made by
 *                                                   lla_rope_table; rope_len >=
 *                                                   max(L_max, 128)
 *   out            device  fp32 [B][H][d]
 *   lse            device  fp32 [B][H]              natural log
 * The new token's own K/V are attended only if the caller has encoded them
 * into slot q_pos (the paper's latent-store decoder reads every cached token
 * back through its latent); lse lets a caller merge further exact terms.
 * LLA_2D (§3 "The LLA-2D variant"): every head h reads the sequence's one latent
 * and reconstructs with rows h*d .. h*d+d-1 of W_up,t; mu_t is the loop-t slice
 * [H*d] of mu [T*H*d] (index (t*H + h)*d + e).  The bf16 kernel runs on pairs of
 * CTAs (thread-block clusters of two).
 */
lla_status lla_decode_attn(const lla_dims* dims, int loop_t, const void* q,
                           lla_cache cache, const int32_t* seq_lens, const int32_t* q_pos,
                           const void* w_up_k, const void* w_up_v,
                           const float* mu_k, const float* mu_v,
                           const float* rope_cos, const float* rope_sin, int64_t rope_len,
                           float* out, float* lse,
                           void* workspace, size_t ws_bytes, void* stream);

/* A paged per-head latent cache (device), as the page tables of "Enabling
 * dynamic computation in Looped LMs" (arXiv 2610.09013, §"Ragged KV" and
 * Appendix A.1 "Page-table aliases for compact K/V storage"): a pool of physical
 * pages and a logical-to-physical table per sequence.
 *   k, v         device  pools [num_pages][H][page_size][r_k / r_v]
 *   block_table  device  int32 [B][max_pages]: logical page p of sequence b
 *                        (tokens p*page_size .. (p+1)*page_size-1) is physical
 *                        page block_table[b*max_pages + p]; several entries may
 *                        name the same page (aliased reads)
 * The logical capacity per sequence is L_max = max_pages * page_size.  Only the
 * entries of pages that hold written or read tokens are looked at; an entry
 * outside [0, num_pages) records LLA_ERR_DEVICE_ARG (reads then use a page
 * inside the pool, writes are skipped), so no access leaves the pool.  Per-head variant only;
 * any page_size >= 1 in both storage types.  In bf16 the tile kernel copies a
 * 128-token tile whole when page_size is a multiple of 128, as 128/P page pieces when
 * P is 8, 16, 32 or 64 (with r_v a multiple of 32, one copy per page holds all of its
 * V columns), and other page sizes (one-token pages, as vLLM's) run a kernel that
 * gathers token rows one by one (correct, much slower); the small-rank kernel copies
 * one page for a whole set of heads when P is 8, 16, 32 or 64, else each tile's rows
 * page by page (any page size). */
typedef struct {
    void* k;
    void* v;
    const int32_t* block_table;
    int B;
    int max_pages;
    int page_size;
    int64_t num_pages;
} lla_paged_cache;

/*
 * lla_encode_paged / lla_decode_attn_paged — lla_encode and lla_decode_attn over
 * a paged cache: token j of (sequence b, head h) lives in row j mod page_size of
 * head h of page block_table[b][j / page_size].  Every other argument, result
 * and rule is that of the dense call with L_max = max_pages * page_size (the
 * workspace is lla_workspace_size(dims, B, max_pages * page_size, N)).
 * LLA_ERR_UNSUPPORTED: LLA-2D.
 */
lla_status lla_encode_paged(const lla_dims* dims, const void* x_k, const void* x_v, int N,
                            const int32_t* seq_idx, const int32_t* pos,
                            const void* w_down_k, const void* w_down_v,
                            const float* mu_k, const float* mu_v,
                            lla_paged_cache cache, void* workspace, size_t ws_bytes, void* stream);
lla_status lla_decode_attn_paged(const lla_dims* dims, int loop_t, const void* q,
                                 lla_paged_cache cache, const int32_t* seq_lens, const int32_t* q_pos,
                                 const void* w_up_k, const void* w_up_v,
                                 const float* mu_k, const float* mu_v,
                                 const float* rope_cos, const float* rope_sin, int64_t rope_len,
                                 float* out, float* lse,
                                 void* workspace, size_t ws_bytes, void* stream);

/*
 * lla_evict_window — token eviction composed with LLA (LLA paper, Appendix D
 * "Token-eviction composition table" and Appendix J "Eviction and long-context
 * prefill"): a StreamingLLM/H2O-style budget keeps each sequence's first `sink`
 * tokens and its `window` newest, and only their latents stay in the cache.
 * For every sequence with L = seq_lens[b] > sink + window, the latent rows of
 * tokens L-window .. L-1 move, in order, to slots sink .. sink+window-1 (every
 * head, K and V, in place) and seq_lens[b] becomes sink + window; sequences at
 * or below the budget are untouched.  A later lla_decode_attn rotates slot j at
 * position j, i.e. positions within the kept cache (StreamingLLM's re-indexing);
 * the query's position is then its slot in the kept cache.  Rows past the new
 * length keep stale latents.
 *   cache      dense cache, as for lla_decode_attn (any variant, dtype)
 *   seq_lens   device int32 [B], read and rewritten; a length outside
 *              [0, L_max] is left alone and records LLA_ERR_DEVICE_ARG
 *   sink, window  >= 0, sink + window >= 1
 *   workspace  device, >= 256 bytes: the status word
 * Asynchronous on `stream`; decode calls after it on the same stream see the new
 * lengths.
 */
lla_status lla_evict_window(const lla_dims* dims, lla_cache cache, int32_t* seq_lens, int sink,
                            int window, void* workspace, size_t ws_bytes, void* stream);

/*
 * lla_window_attn — exact attention over each sequence's window of recent
 * tokens, merged into a latent-store result ("Hybrid Latent Attention for Looped
 * Language Models", §3.4 "Exact sliding window", Eq. (4), and Appendix I
 * "Serving Implementation").  Eq. (4) takes one softmax over the latent tokens
 * before the window and the window's exact keys; with `out`/`lse` holding
 * lla_decode_attn's result for the latent tokens (seq_lens = their count) at
 * loop t, this call computes the window's own softmax and merges the two by
 * log-sum-exp, which equals that single softmax.  Any lla_dims variant; the
 * window is per head in both.
 *   q         device  [B][H][d]        the query lla_decode_attn took
 *   k_win     device  [B][H][W][d]     exact keys of loop t, BEFORE RoPE
 *   v_win     device  [B][H][W][d]     exact values of loop t
 *   win_len   device  int32 [B]        window tokens in use, 0..W
 *   win_pos   device  int32 [B]        position of window token 0; token w is
 *                                      rotated at win_pos[b] + w
 *   q_pos     device  int32 [B]        as for lla_decode_attn
 *   rope_cos/_sin, rope_len            as for lla_decode_attn (rope_len >= 128);
 *                                      every window position must be < rope_len
 *   out, lse  device  fp32 [B][H][d], [B][H]   in: latent part; out: merged
 *                                      (rows with win_len 0 are left as they are)
 *   workspace device  >= 256 bytes: the status word (lla_device_status)
 * q, k_win and v_win use the storage dtype (bf16 or fp32).  A win_len outside
 * [0, W] or a window reaching past rope_len skips that sequence's window, a
 * q_pos outside [0, rope_len) is clamped; both record LLA_ERR_DEVICE_ARG.
 * W == 0 or B == 0 launches nothing.
 */
lla_status lla_window_attn(const lla_dims* dims, int B, int W, const void* q,
                           const void* k_win, const void* v_win, const int32_t* win_len,
                           const int32_t* win_pos, const int32_t* q_pos,
                           const float* rope_cos, const float* rope_sin, int64_t rope_len,
                           float* out, float* lse, void* workspace, size_t ws_bytes, void* stream);

/*
 * lla_decode_attn_decoupled — absorbed decoupled-RoPE decode (LLA paper,
 * Appendix J "Absorbed attention"; the path its Table 13 times).  The K
 * up-projection moves to the query side (an MLA-style content path on the
 * latents without RoPE) and position enters through a small explicit rotary
 * branch of d_rope = 64 dimensions per token and head, stored once for all loops:
 *   s_j = (q_c . (c_k,j W_up,k,t^T + mu_k,t) + RoPE(q_r, q_pos) . RoPE(r_j, j))
 *         / sqrt(d + d_rope),
 *   out = sum_j softmax(s)_j (c_v,j W_up,v,t^T + mu_v,t),  lse = ln sum_j exp(s_j).
 * This is a different function from lla_decode_attn (no RoPE on the content
 * keys); a model must have been trained or adapted for it (Appendix J, Table 14).
 * LLA_PER_HEAD only; d_rope must be 64; r_k <= 128 on the bf16 kernel.
 *   q          device  [B][H][d + d_rope]   content part then rotary part
 *   k_rope     device  [B][H][L_max][d_rope] rotary keys before RoPE (storage dtype)
 *   rope_cos/_sin      [rope_len][d_rope/2] for the rotary branch: lla_rope_table
 *                      with lla_dims.d_head = d_rope (theta_f = base^(-2f/d_rope));
 *                      rope_len >= max(L_max, 128)
 *   workspace          >= lla_decoupled_workspace_size() bytes, first 256 zero
 * Everything else as lla_decode_attn (cache, seq_lens, q_pos, W_up, mu, out, lse).
 */
size_t lla_decoupled_workspace_size(const lla_dims* dims, int d_rope, int B, int64_t L_max);
lla_status lla_decode_attn_decoupled(const lla_dims* dims, int loop_t, int d_rope, const void* q,
                                     lla_cache cache, const void* k_rope,
                                     const int32_t* seq_lens, const int32_t* q_pos,
                                     const void* w_up_k, const void* w_up_v,
                                     const float* mu_k, const float* mu_v,
                                     const float* rope_cos, const float* rope_sin, int64_t rope_len,
                                     float* out, float* lse,
                                     void* workspace, size_t ws_bytes, void* stream);

/*
 * RoPE as operators of its own, beside the rotation that the decode calls fuse.
 *
 * lla_rope_scaling — frequencies for contexts beyond the trained one; with
 * theta_f = rope_base^(-2f/d_head), f < d_head/2:
 *   LLA_ROPE_PLAIN     theta_f
 *   LLA_ROPE_LINEAR    theta_f / factor                      (positions interpolated)
 *   LLA_ROPE_BASE      rope_base scaled by factor^(d/(d-2))  (d_head >= 4)
 *   LLA_ROPE_BY_PARTS  with r = original_len theta_f / 2 pi turns over the original
 *                      context and g = clamp((r - slow) / (fast - slow), 0, 1):
 *                      (1 - g) theta_f / factor + g theta_f; fast > slow >= 0,
 *                      original_len >= 1
 * factor > 0.  A field that the kind does not use is ignored.
 */
typedef enum {
    LLA_ROPE_PLAIN = 0,
    LLA_ROPE_LINEAR = 1,
    LLA_ROPE_BASE = 2,
    LLA_ROPE_BY_PARTS = 3
} lla_rope_scaling_kind;

typedef struct {
    int kind;                   /* lla_rope_scaling_kind                   */
    double factor;
    int64_t original_len;
    double fast, slow;
} lla_rope_scaling;

/*
 * lla_rope_table_scaled — a RoPE table built on the GPU: row i gets cos and sin of
 * (pos0 + i) theta_f for f < d_head/2.  Rows have the layout of lla_rope_table (whose
 * values it equals to about 1 ulp with scaling NULL or LLA_ROPE_PLAIN), so with pos0 = 0
 * the result serves every call that takes a RoPE table.  Angles are exact products, in
 * 64-bit fixed point, of the position and a frequency held in fp64, so what a far position
 * loses is the frequency's own rounding: 2^-52 of the angle at most (an fp32 half step
 * from 2^28 radians on, 5e-7 at 2^31).
 *   scaling              host; NULL: plain
 *   rope_cos, rope_sin   device fp32 [n_pos][d_head/2], 16-byte aligned
 * Of lla_dims only rope_base and d_head (even, 2..256) are used.  pos0 and n_pos are
 * at most 2^31.  Asynchronous on `stream`.
 */
lla_status lla_rope_table_scaled(const lla_dims* dims, const lla_rope_scaling* scaling, int64_t pos0,
                                 int64_t n_pos, float* rope_cos, float* rope_sin, void* stream);

/*
 * lla_rope_apply — rotate elements offset .. offset+d_rope-1 of every head's vector by
 * its token's position and scale them; the other elements pass through:
 *     out = scale * RoPE(x, pos)            (inverse == 0)
 *     out = scale * RoPE(x, -pos)           (inverse != 0: the gradient of the former
 *                                            with respect to x, given out's gradient as x)
 * Pairs are those of lla_dims.rope_style within the d_rope elements.  `scale` is for the
 * attention factor that some scalings put on the rotated part; 1 for a plain rotation.
 *   x, out     device  element (n, h, e) at n*tok_stride + h*head_stride + e, e < d_x
 *                      (strides in elements, so a slice of a fused projection is taken as it
 *                      is); storage dtype; aligned to an element (16-byte alignment of
 *                      bases, strides, offset, d_rope/2 and d_x is faster)
 *   pos        device  int32 [N]; outside [0, rope_len) is clamped and records
 *                      LLA_ERR_DEVICE_ARG
 *   rope_cos/_sin      device fp32 [rope_len][d_rope/2]
 *   workspace          device, >= 256 bytes: the status word
 * out == x with the same strides rotates in place (only the rotated part is written);
 * other overlaps return LLA_ERR_INVALID_ARG, but two slices of one buffer with equal strides
 * whose rows lie apart (q and k next to each other per token, per head or head-major) are no
 * overlap.  Rows of `out` must not overlap each other.  Arithmetic in fp32, rounded once.
 * Of lla_dims only dtype and rope_style are used.
 */
lla_status lla_rope_apply(const lla_dims* dims, const void* x, int64_t x_tok_stride, int64_t x_head_stride,
                          void* out, int64_t out_tok_stride, int64_t out_head_stride, int N, int heads,
                          int d_x, int offset, int d_rope, const int32_t* pos, const float* rope_cos,
                          const float* rope_sin, int64_t rope_len, float scale, int inverse,
                          void* workspace, size_t ws_bytes, void* stream);

/*
 * lla_page_plan — the block tables and slot maps of one step, built on the GPU from the
 * requests' lengths and a list of free pages ("Enabling dynamic computation in Looped
 * LMs", Appendix A.1).  Request b holds ctx_lens[b] cached tokens, in pages that its
 * table row names already, and brings new_lens[b] more.  Its new tokens are numbered from
 * tok_start[b] = sum of new_lens before b, the order in which the step's activations are
 * packed.  A request is granted if its table row can hold all of its tokens
 * (ctx + new <= max_pages * page_size), its tokens lie below n_tok, and the free pages
 * reach it: pages are handed out in request order, and the first request that they do
 * not suffice for ends the hand-out for every later one that needs a page (requests whose
 * last page has room are still granted).
 *   ctx_lens, new_lens  device int32 [B]       a negative value counts as 0 and records
 *                                              LLA_ERR_DEVICE_ARG
 *   free_pages          device int32 [n_free]  physical pages, taken from free_head on
 *   free_head           device int32 [1] or NULL (0): entries already taken; outside
 *                                              [0, n_free] counts as n_free, flagged
 *   block_table         device int32 [B][max_pages], updated: the entries of the pages
 *                                              that granted requests take; no other
 *   seq_lens            device int32 [B]       out: ctx + new where granted, else ctx
 *   tok_start           device int32 [B+1]     out; entry B is the sum (saturating)
 *   granted             device int32 [B]       out: 1 or 0
 *   seq_idx, pos        device int32 [n_tok]   out: request and position of token n, as
 *                                              lla_encode_paged takes them
 *   slots               device int64 [n_tok]   out: physical page * page_size + row, as
 *                                              lla_q4_store takes them
 *                                              (entries of no granted token: -1 in all three)
 *   counts              device int32 [2]       out: the next call's free_head; tokens granted
 *   workspace           device, >= 256 bytes: the status word
 * A table or free-list entry outside [0, num_pages) that a token falls on records
 * LLA_ERR_DEVICE_ARG and its slot is -1.  No output may overlap an input (a step's
 * seq_lens become the next step's ctx_lens by alternating two arrays).  B <= 8192,
 * max_pages * page_size <= 2^30; else LLA_ERR_UNSUPPORTED.
 */
lla_status lla_page_plan(int B, int page_size, int max_pages, int64_t num_pages, const int32_t* ctx_lens,
                         const int32_t* new_lens, const int32_t* free_pages, int n_free,
                         const int32_t* free_head, int32_t* block_table, int32_t* seq_lens,
                         int32_t* tok_start, int32_t* granted, int n_tok, int32_t* seq_idx, int32_t* pos,
                         int64_t* slots, int32_t* counts, void* workspace, size_t ws_bytes, void* stream);

/*
 * A paged per-head latent cache held in 4 bits (device): rows [num_pages][H][page_size]
 * of lla_q4_row_bytes() bytes, one per token and head with its K and its V latent:
 * K codes, V codes, one bf16 scale per 32 columns (the last group of a rank may have
 * 16) of K, then of V, zero padding to 16 bytes.  Eight columns make a 32-bit word;
 * column c of a word is bits 4(c/2) + 16(c mod 2) .. +3, holding code + 8 with code in
 * [-7, 7]; the latent is code * scale.  At (r_k, r_v) = (96, 160) a row is 144 bytes
 * against 512 in bf16, at (16, 32) 32 against 96.  block_table as in lla_paged_cache;
 * lla_q4_store and lla_q4_load use only rows, page_size and num_pages.
 */
typedef struct {
    void* rows;
    const int32_t* block_table;
    int B;
    int max_pages;
    int page_size;
    int64_t num_pages;
} lla_q4_cache;

/* Bytes of a row (a multiple of 16); 0 for invalid dims and LLA_2D. */
size_t lla_q4_row_bytes(const lla_dims* dims);

/*
 * lla_q4_store / lla_q4_load — round N tokens' latents into 4-bit rows, and read rows
 * back as latents.  Per group of 32 columns scale = bf16(max|c| / 7) and
 * code = round(c / scale), half to even, both divisions in fp32; a group of zeros has
 * scale 0, a group with a value that is not finite reads back as NaN.
 *   c_k, c_v   device  [N][H][r_k], [N][H][r_v] in the storage dtype: what lla_encode
 *                      writes into a cache of B = N sequences and L_max = 1
 *   slots      device  int64 [N]: physical page * page_size + row within it, as made by
 *                      lla_page_plan; a negative slot is skipped (a load leaves that
 *                      token's output as it is), one beyond the pool is skipped and
 *                      records LLA_ERR_DEVICE_ARG; two tokens storing to one slot race
 *   workspace  device, >= 256 bytes: the status word
 * A load rounds code * scale to the storage dtype.  LLA_PER_HEAD only.
 */
lla_status lla_q4_store(const lla_dims* dims, const void* c_k, const void* c_v, int N, const int64_t* slots,
                        const lla_q4_cache* cache, void* workspace, size_t ws_bytes, void* stream);
lla_status lla_q4_load(const lla_dims* dims, const int64_t* slots, int N, const lla_q4_cache* cache,
                       void* c_k, void* c_v, void* workspace, size_t ws_bytes, void* stream);

/*
 * lla_decode_attn_q4 — lla_decode_attn_paged over a 4-bit cache: the same attention of the
 * latents that the rows stand for.  `out` is [B][H][d] in the storage dtype (rounded
 * once); `lse` may be NULL.  Everything else as lla_decode_attn_paged, with a workspace of
 * lla_q4_workspace_size() bytes (L_max = max_pages * page_size), the first 256 zero.  A row
 * with a NaN scale makes its sequence-head's result NaN.  bf16 storage: scores carry one f16
 * rounding of the folded query and one of the table's rows (|cos|, |sin| below 65504), weights one of
 * p * scale (11 bits down to 2^-21 of the largest p * scale among 32 tokens, one bit fewer per power of
 * two below); sums are fp32 and leave out what lies 2^64 below the largest.  fp32 storage: fp32 throughout.
 * An attention factor f that a scaling puts on rotated queries and keys: rows of a table multiplied by
 * f, which the query and the keys both take (scores times f^2).
 * lla_encode writes latents in the storage dtype only (lla_q4_store rounds them).  The decoupled and
 * eviction calls do not take a 4-bit cache; lla_window_attn merges into an fp32 `out`, which this call
 * writes in fp32 storage.
 */
size_t lla_q4_workspace_size(const lla_dims* dims, int B, int64_t L_max);
lla_status lla_decode_attn_q4(const lla_dims* dims, int loop_t, const void* q, const lla_q4_cache* cache,
                              const int32_t* seq_lens, const int32_t* q_pos,
                              const void* w_up_k, const void* w_up_v,
                              const float* mu_k, const float* mu_v,
                              const float* rope_cos, const float* rope_sin, int64_t rope_len,
                              void* out, float* lse, void* workspace, size_t ws_bytes, void* stream);

/*
 * A step that verifies drafted tokens (speculative decoding).  Every sequence brings a
 * tree of drafted tokens, its nodes; all of them go through the model in one step, each
 * attending to the cached tokens and to the nodes on its own path (itself and its
 * ancestors).  lla_tree_attn is that attention, lla_logits_adjust prepares each node's
 * logits and names its best token, lla_tree_accept walks down the tree along the chosen
 * tokens and says which nodes stay and where lla_encode writes them.
 *
 * lla_tree — the nodes of B sequences, packed in sequence order: those of sequence b are
 * the token entries tok_start[b] .. tok_start[b+1]-1.  A sequence may have none; entries
 * from tok_start[B] on are padding, and no output of theirs is written.
 *   n_tok       entries of the arrays that have one per token
 *   max_nodes   most nodes of a sequence, 1..LLA_TREE_MAX_NODES
 *   tok_start   device int32 [B+1]   as made by lla_page_plan; a sequence whose entries are
 *                                    not 0 <= start <= end <= n_tok with at most max_nodes
 *                                    between counts as one without nodes
 *   parent      device int32 [n_tok] the parent's index among the sequence's nodes, below
 *                                    the node's own; -1 for a root (anything else counts
 *                                    as -1).  A chain has parent i-1.
 *   pos         device int32 [n_tok] positions of the nodes, as a rule cached tokens + depth
 *                                    (lla_tree_attn only; else it may be NULL); outside
 *                                    [0, rope_len) is clamped
 * Everything that "counts as" something else or is clamped records LLA_ERR_DEVICE_ARG.
 */
#define LLA_TREE_MAX_NODES 128

typedef struct {
    int B;
    int n_tok;
    int max_nodes;
    const int32_t* tok_start;
    const int32_t* parent;
    const int32_t* pos;
} lla_tree;

/*
 * lla_tree_attn / lla_tree_attn_paged — one layer, one loop t, all heads: attention of every
 * node i over its sequence's L = seq_lens[b] cached tokens, whose keys and values are
 * reconstructed from their latents as in lla_decode_attn, and over the exact keys and values
 * of the nodes on its path:
 *     s_j = RoPE(q_i, pos_i) . RoPE(k_j, j) / sqrt(d)       k_j of Eq. (3), j < L
 *     s_a = RoPE(q_i, pos_i) . RoPE(k_a, pos_a) / sqrt(d)   a on the path of i
 *     out = softmax over both, times v_j and v_a;  lse = ln of the sum of exponentials
 * A node sees itself, so L = 0 is an ordinary case.  Drafted tokens are not in the cache:
 * once they are accepted, lla_encode writes their latents.
 *   q, k, v   device  [n_tok][H][d] of loop t, before RoPE, storage dtype: element (n, h, e)
 *                     at n*stride + h*d + e (strides in elements, multiples of 16 bytes of
 *                     at least H*d: slices of one fused projection are taken as they are)
 *   out       device  [n_tok][H][d] in the storage dtype, rounded once
 *   lse       device  fp32 [n_tok][H] or NULL; no output, the workspace among them, may overlap an
 *                     input or another output (LLA_ERR_INVALID_ARG)
 *   workspace device  >= lla_tree_workspace_size() bytes (L_max: that of the cache, or
 *                     max_pages * page_size), the first 256 zero
 * cache.B is the tree's B.  seq_lens, w_up, mu, rope tables and the paged cache as for
 * lla_decode_attn and lla_decode_attn_paged; rope_len >= max(L_max, 128) and past every pos.
 * fp32 arithmetic, or ("tensor" of lla_tree_kernel) matrix instructions on operands that keep 22
 * bits of keys and queries, 16 of the cached tokens' weights and 24 of the drafted ones' and of the
 * latent sums, with fp32 sums: lse is off by some 2^-20 of |q| |k| / sqrt(d) (2e-5 at most for scores
 * of ordinary size, at any length), out by its own rounding and 2^-13 of a sum of its terms' sizes.
 * There the table's rows have to be cos and sin of j theta_f (those of any scaling), in both paths
 * times an attention factor if there is one, the same in every row, which then multiplies queries
 * and keys.  A sequence with keys 2^11 times above most of its others' may take a slower way to the
 * same result (0.9 us for each of its cached tokens).  A NaN or an infinity reaches the nodes that
 * see it and no others: a cached latent's its sequence's nodes, a node's key and value the nodes
 * below it, a query its own node.  LLA_ERR_UNSUPPORTED: LLA-2D.
 */
size_t lla_tree_workspace_size(const lla_dims* dims, int B, int max_nodes, int64_t L_max);
lla_status lla_tree_attn(const lla_dims* dims, int loop_t, const lla_tree* tree, const void* q, int64_t q_stride,
                         const void* k, int64_t k_stride, const void* v, int64_t v_stride, lla_cache cache,
                         const int32_t* seq_lens, const void* w_up_k, const void* w_up_v, const float* mu_k,
                         const float* mu_v, const float* rope_cos, const float* rope_sin, int64_t rope_len,
                         void* out, float* lse, void* workspace, size_t ws_bytes, void* stream);
lla_status lla_tree_attn_paged(const lla_dims* dims, int loop_t, const lla_tree* tree, const void* q,
                               int64_t q_stride, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                               lla_paged_cache cache, const int32_t* seq_lens, const void* w_up_k,
                               const void* w_up_v, const float* mu_k, const float* mu_v, const float* rope_cos,
                               const float* rope_sin, int64_t rope_len, void* out, float* lse, void* workspace,
                               size_t ws_bytes, void* stream);

/*
 * lla_logits_adjust — penalties, biases and grammar masks on the logits of every node, and
 * each row's best token and log-sum-exp.  Row n holds what the model predicts after node n of
 * request b; its context is the request's history and the tokens of the nodes on n's path
 * (itself among them; a step without drafting has one node a request, its newest token).  With
 * c = occurrences of the token in the output part of the history (from prompt_len on) and on
 * the path, and seen = c > 0 or it occurs in the prompt part, in fp32, each step rounded:
 *     x = seen ? (x > 0 ? x / repetition : x * repetition) : x
 *     x = x - frequency * c;  x = x - presence if c > 0;  x = x + bias
 *     x = -inf unless the row's mask allows the token
 *     best = the lowest index of the largest x (a NaN is never the largest; -1 if no x is above
 *     -inf),  lse = ln sum exp(x) (-inf if nothing is allowed)
 *   token       device int32 [n_tok]   token of each node
 *   logits      device [n_tok] rows of `vocab` elements, row n at n*row_stride elements; dtype
 *                                      LLA_BF16 or LLA_F32, aligned to an element
 *   out         the same layout with out_stride, rounded once; out == logits with equal strides
 *               is in place, any other overlap of an output or the workspace with an input or
 *               another output LLA_ERR_INVALID_ARG; NULL: not written
 *   best        device int32 [n_tok] or NULL: from x before `out` rounds it
 *   lse         device fp32 [n_tok] or NULL; at least one of out, best, lse
 *   workspace   device, >= lla_logits_workspace_size() bytes, the first 256 zero
 * Tokens outside [0, vocab) count nowhere and record LLA_ERR_DEVICE_ARG.
 */
typedef struct {
    const int32_t* history;     /* device [B][max_history]: tokens, prompt then output           */
    const int32_t* hist_len;    /* device [B], 0..max_history (clamped, flagged)                  */
    const int32_t* prompt_len;  /* device [B], 0..hist_len (clamped, flagged); NULL: 0            */
    int max_history;            /* 0: no history (the three above may be NULL)                    */
    const float* repetition;    /* device [B]; NULL: 1                                            */
    const float* presence;      /* device [B]; NULL: 0                                            */
    const float* frequency;     /* device [B]; NULL: 0                                            */
    const int32_t* bias_token;  /* device [B][max_bias]: a negative entry is unused; a token      */
    const float* bias;          /*        listed more than once gets the sum, in list order       */
    int max_bias;               /* 0: no biases                                                   */
    const uint32_t* allowed;    /* device [n_masks][ceil(vocab/32)]: bit v%32 of word v/32        */
    const int32_t* allowed_row; /* device [n_tok]: the row's mask, negative: none (beyond         */
    int n_masks;                /* n_masks: none, flagged).  n_masks 0: no masks                  */
} lla_logit_rules;

size_t lla_logits_workspace_size(int n_tok, int vocab);
lla_status lla_logits_adjust(const lla_tree* tree, const int32_t* token, int dtype, const void* logits,
                             int64_t row_stride, int vocab, const lla_logit_rules* rules, void* out,
                             int64_t out_stride, int32_t* best, float* lse, void* workspace, size_t ws_bytes,
                             void* stream);

/*
 * lla_tree_accept — which drafted tokens stay.  Node 0 of a sequence is accepted (it is the
 * token that the step before chose); from an accepted node the walk goes on to its lowest child
 * whose token is the one chosen after that node, until there is none.
 *   token, chosen  device int32 [n_tok]  token of each node; token that the model chose after it
 *                                        (lla_logits_adjust's best, or a sample)
 *   ctx_lens       device int32 [B]      cached tokens of each sequence
 *   count          device int32 [B]      out: accepted nodes (0 for a sequence without nodes)
 *   next_token     device int32 [B]      out: the token chosen after the last of them (-1 likewise)
 *   seq_lens       device int32 [B]      out: ctx_lens + count
 *   path           device int32 [n_tok]  out: entries of the accepted nodes in path order, from
 *                                        each sequence's first entry on, then -1
 *   seq_idx, pos   device int32 [n_tok]  out: as lla_encode takes them: accepted nodes go to slots
 *                                        ctx_lens .. seq_lens-1 in path order, the others behind
 *                                        them in node order (every entry has a slot of its own; what
 *                                        lies behind seq_lens is overwritten by the next step).
 *                                        Entries of no sequence keep what they held, a call before
 *                                        perhaps: where all n_tok go to lla_encode, set seq_idx to -1
 *                                        first (it skips and flags those, as lla_page_plan's)
 *   workspace      device, >= 256 bytes: the status word
 * A negative ctx_lens counts as 0 and records LLA_ERR_DEVICE_ARG.  No output may overlap an input or
 * another output (LLA_ERR_INVALID_ARG).
 */
lla_status lla_tree_accept(const lla_tree* tree, const int32_t* token, const int32_t* chosen,
                           const int32_t* ctx_lens, int32_t* count, int32_t* next_token, int32_t* seq_lens,
                           int32_t* path, int32_t* seq_idx, int32_t* pos, void* workspace, size_t ws_bytes,
                           void* stream);

/* Size of the fixed scratch array behind lla_decode_attn_noalloc (64 MiB). */
#define LLA_NOALLOC_SCRATCH_BYTES (64u << 20)

/*
 * lla_decode_attn_noalloc — lla_decode_attn without a caller workspace, for
 * callers that cannot allocate device memory (for example a plugin inside a
 * host framework whose memory pool owns the GPU, or a serving path that must
 * never call cudaMalloc).  The paper has no counterpart: this is a deployment
 * convenience.  Arguments and results are those of lla_decode_attn, minus
 * `workspace` and `ws_bytes`.
 *   - Scratch lives in a fixed __device__ array of LLA_NOALLOC_SCRATCH_BYTES
 *     inside this library; every GPU that loads the library keeps it until
 *     the process exits.  The call allocates nothing.
 *   - Shapes whose workspace (lla_workspace_size) exceeds that size return
 *     LLA_ERR_UNSUPPORTED before any launch (e.g. beyond about 2,000 sequence-heads
 *     at r_k = 96, r_v = 160).
 *   - The first call on each device looks up the array's device address with
 *     the device current; make that first call before any stream capture.
 *   - The array is shared by every call and keeps the last call's contents;
 *     once the host checks have passed, the status word is cleared on `stream`
 *     before the first launch (a call rejected on the host enqueues nothing).
 *     Calls that overlap on the GPU race and must be serialised by the caller.
 *   - The kernels' device status (LLA_ERR_DEVICE_ARG, LLA_ERR_TIMEOUT,
 *     LLA_ERR_RANGE) is read with lla_device_status(NULL, stream, clear) on
 *     the same device.
 */
lla_status lla_decode_attn_noalloc(const lla_dims* dims, int loop_t, const void* q,
                                   lla_cache cache, const int32_t* seq_lens, const int32_t* q_pos,
                                   const void* w_up_k, const void* w_up_v,
                                   const float* mu_k, const float* mu_v,
                                   const float* rope_cos, const float* rope_sin, int64_t rope_len,
                                   float* out, float* lse, void* stream);

/* Name of the kernel family lla_decode_attn runs for `dims` (host-only, no
 * launch): "fp32" (LLA_F32), "pair-2d" (LLA_2D bf16 with an even H <= 16,
 * r_k <= 128 and r_v <= 256: CTA-pair score kernel on the tensor cores, then a
 * tensor-core value kernel), "plain-2d" (every other LLA_2D bf16 shape: the
 * plain per-(sequence, head) kernels in fp32 arithmetic over the bf16 storage;
 * correct, not tuned), "small-rank"
 * (LLA_PER_HEAD bf16 with r_k in {16, 32}, r_v in {32, 64} and an even H <= 16
 * whose H query images and a 4-slot latent ring fit in shared memory:
 * positions split over CTAs, RoPE applied by the tensor cores), "tile"
 * (every other LLA_PER_HEAD bf16 shape: 128-token tiles over (sequence, head)
 * split over CTAs), or NULL for invalid or unsupported dims. */
const char* lla_decode_kernel(const lla_dims* dims);

/* Name of the kernel family lla_decode_attn_decoupled runs for `dims` and
 * d_rope (host-only, no launch): "fp32" (LLA_F32), "small-rank" (bf16 with r_k in
 * {16, 32}, r_v in {32, 64} and an even H <= 16: positions split over CTAs,
 * rotary branch and content score on the tensor cores, fp32 cos/sin per token),
 * "tile" (every other bf16 shape with r_k <= 128 and r_v <= 256: 128-token
 * tiles over (sequence, head), the same tensor-core score, V read from L2), or
 * NULL for invalid or unsupported dims (LLA_2D, d_rope != 64, larger ranks). */
const char* lla_decoupled_kernel(const lla_dims* dims, int d_rope);

/* Name of the kernel family lla_tree_attn (page_size 0) or lla_tree_attn_paged runs for
 * `dims` (host-only, no launch), the same for every page size and number of nodes: "tensor" (LLA_BF16
 * whose operands fit in shared memory beside the largest block of nodes, 64 for r_v up to 176 and 32
 * above: r_k up to 208 with any r_v; r_k 224 but for r_v 176, 240 and 256; r_k 240 with r_v up to 128
 * or 192; r_k 256 with r_v up to 96), "plain" (others: fp32 arithmetic, not tuned for bf16), or NULL for invalid or unsupported dims (LLA_2D). */
const char* lla_tree_kernel(const lla_dims* dims, int page_size);

/* Workspace bytes for calls with at most B sequences of L_max slots and
 * encode batches of at most max_N tokens, on the current CUDA device.
 * Returns 0 for invalid dims. */
size_t lla_workspace_size(const lla_dims* dims, int B, int64_t L_max, int max_N);

/* Host-side RoPE table: cos_out/sin_out (host, fp32 [n_pos][d/2]) get
 * cos(p*theta_f), sin(p*theta_f) for p < n_pos, computed in fp64 and rounded
 * once to fp32. */
lla_status lla_rope_table(const lla_dims* dims, int64_t n_pos, float* cos_out, float* sin_out);

/* Synchronise `stream`, then return the status word the kernels recorded in
 * `workspace` (LLA_OK if none); clear it when `clear` is non-zero.  With
 * workspace == NULL the word read is that of lla_decode_attn_noalloc's fixed
 * scratch on the current device. */
lla_status lla_device_status(void* workspace, void* stream, int clear);

/* Static description of a status code. */
const char* lla_status_string(lla_status status);

/* LLA_ABI_VERSION of the loaded library. */
int lla_abi_version(void);

#ifdef __cplusplus
}
#endif
#endif /* LLA_H */
