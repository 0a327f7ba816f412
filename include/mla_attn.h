/*
 * mla_attn.h -- C ABI of the GB300 (sm_103a) MLA causal-attention library.
 *
 * The operation is the causal-attention core of Kimi K2's Multi-head Latent Attention,
 * as quoted on the page "Kimi K2 · Similarities" (section "Contextual evidence from
 * Query-key similarity", the MLA forward of modeling_deepseek.py) and on the page
 * "Weighted sum of values" (tensor card: weights [B,64,T,T] times values [B,64,T,128]
 * give [B,64,T,128]).  Per sequence b, head h and query i:
 *
 *   Q   = [q_nope[b,h,i,0:128] | q_pe[b,h,i,0:64]]           (query concat)
 *   K_j = [k_nope[b,h,j,0:128] | k_pe_shared[b,j,0:64]]      (key concat; one rotary
 *                                                             key row shared by all heads)
 *   s_j = softmax_scale * (Q . K_j)                          (scores, then scale)
 *   key j is visible iff j <= i + past_len and j < kv_len[b] (4D causal mask offset by
 *                                                             the cached length, plus
 *                                                             right padding)
 *   w   = softmax over visible j of s_j, in fp32             (hidden keys get weight 0)
 *   out[b,h,i,:] = sum_j bf16(w_j) * v[b,h,j,:]              (weights cast to bf16, then
 *                                                             the weighted sum of values)
 *
 * Dropout (attention_dropout = 0.0 in the config.json excerpt on "Kimi K2 · Logits") is
 * the identity and is not applied.  The cache layout follows the cache update in the
 * same excerpt: the Tk = past_len + Tq key/value rows hold the cached prefix first and
 * the Tq new rows last, and query i sits at position past_len + i (positions are
 * numbered from the cached length, page "Kimi K2 · Causal mask", section "Construct
 * causal mask").
 *
 * Head widths are fixed by the config.json excerpt: qk_nope_head_dim 128,
 * qk_rope_head_dim 64, v_head_dim 128.  The head count H is a runtime argument (64 in
 * Kimi K2).
 *
 * Data types and layout.  bf16 tensors are passed as uint16_t bit patterns; every tensor
 * is row-major and contiguous in the shape given, in DEVICE memory of the current CUDA
 * device:
 *   q_nope      [B, H, Tq, 128]      q_pe        [B, H, Tq, 64]
 *   k_nope      [B, H, Tk, 128]      k_pe_shared [B, Tk, 64]
 *   v           [B, H, Tk, 128]      out         [B, H, Tq, 128]
 *   kv_len      [B] int32, or NULL meaning kv_len[b] = Tk for every b
 * Every pointer must be 16-byte aligned (bulk/tensor copies move 16-byte units).
 *
 * Ownership.  The caller owns every buffer: inputs, out, kv_len and the workspace.  The
 * library never allocates or frees device memory on the call path.  Inputs are only
 * read; out is fully overwritten.  Work is enqueued asynchronously on cuda_stream (a
 * cudaStream_t, NULL for the legacy default stream); the call returns before it runs.
 *
 * Errors.  Host-side checks run before anything is enqueued and are returned directly
 * (nothing is launched when a check fails).  Problems only the device can see
 * (kv_len[b] outside [1, Tk]; a bounded wait that gave up) are recorded in a status word
 * inside the workspace; mla_attn_get_status reads it.  Such a call still completes: an
 * out-of-range kv_len is clamped to [1, Tk] for memory safety and the output for that
 * sequence is not meaningful.
 */
#ifndef MLA_ATTN_H_
#define MLA_ATTN_H_

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define MLA_API __attribute__((visibility("default")))
#else
#define MLA_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  MLA_OK = 0,
  MLA_ERR_NULL = 1,      /* a required pointer is NULL */
  MLA_ERR_SHAPE = 2,     /* B, H, Tq < 1, past_len < 0, Tk != past_len + Tq, or too large:
                            the score-shape check of the attention excerpt (scores must be
                            [B, H, Tq, Tk]) */
  MLA_ERR_ALIGN = 3,     /* a pointer is not 16-byte aligned */
  MLA_ERR_WORKSPACE = 4, /* workspace NULL or smaller than mla_attn_workspace_bytes() */
  MLA_ERR_DEVICE = 5,    /* the current device is not an sm_103 (GB300-class) GPU */
  MLA_ERR_CUDA = 6,      /* a CUDA runtime call or kernel launch failed */
  MLA_ERR_KVLEN = 7,     /* (device) some kv_len[b] outside [1, Tk] */
  MLA_ERR_TIMEOUT = 8,   /* (device) a bounded wait inside a kernel gave up */
  MLA_ERR_ARG = 9,       /* an option value is out of range */
  MLA_ERR_PAGE = 10,     /* (device) a page or slot outside the pool, or no free page left */
  MLA_ERR_TREE = 11      /* (device) a parent that does not come before its token, or more
                            drafted tokens in a sequence than a 64-bit mask holds */
} mla_status;

/*
 * Bytes of device workspace mla_attn_fwd needs for these sizes (a status word plus the
 * split-KV partial results of the decode path).  The workspace must be zero-filled once
 * before its first use (cudaMemset); afterwards the library keeps the status word
 * consistent itself.  Returns 0 for invalid sizes.
 */
MLA_API size_t mla_attn_workspace_bytes(int B, int H, int Tq, int Tk);

/*
 * The attention core described at the top of this file.  past_len is the cached length
 * (Tk must equal past_len + Tq); softmax_scale (finite, > 0, else MLA_ERR_ARG) multiplies
 * the raw scores (192^-0.5 for Kimi K2 before any YaRN adjustment, which the caller folds
 * in).  Tq == 1 takes the
 * split-KV decode path; Tq > 1 the tensor-core prefill path.  Returns MLA_OK once the
 * work is enqueued, or a host-side error code.
 */
MLA_API mla_status mla_attn_fwd(const uint16_t* q_nope, const uint16_t* q_pe, const uint16_t* k_nope,
                        const uint16_t* k_pe_shared, const uint16_t* v, const int32_t* kv_len,
                        int B, int H, int Tq, int Tk, int past_len, float softmax_scale,
                        uint16_t* out, void* workspace, size_t workspace_bytes,
                        void* cuda_stream);

/* Path selection for mla_attn_fwd_ex. */
typedef enum { MLA_PATH_AUTO = 0, MLA_PATH_PREFILL = 1, MLA_PATH_DECODE = 2 } mla_path;

/*
 * Options for mla_attn_fwd_ex.  Zero-initialised options mean "choose automatically",
 * which is what mla_attn_fwd does.
 *   path:         force the prefill (any Tq >= 1) or decode (Tq == 1 only) path.
 *   decode_chunk: keys per split of the decode path (a multiple of 64, at most 65536);
 *                 0 lets the scheduler pick it from B, H and Tk.
 */
typedef struct {
  int path;
  int decode_chunk;
  int reserved[6];
} mla_attn_options;

/* mla_attn_fwd with explicit options (same arguments and semantics otherwise). */
MLA_API mla_status mla_attn_fwd_ex(const uint16_t* q_nope, const uint16_t* q_pe,
                           const uint16_t* k_nope, const uint16_t* k_pe_shared,
                           const uint16_t* v, const int32_t* kv_len, int B, int H, int Tq,
                           int Tk, int past_len, float softmax_scale, uint16_t* out,
                           void* workspace, size_t workspace_bytes, void* cuda_stream,
                           const mla_attn_options* options);

/*
 * Cache append + attention.  The cache update of the attention excerpt on "Kimi K2 ·
 * Similarities" (past_key_value.update: the new key/value rows follow the cached prefix)
 * fused with the core described at the top of this file:
 *
 *   k_nope_cache[b,h,past_len+t,:] = k_nope_new[b,h,t,:]    (t < Tq)
 *   k_pe_cache  [b,  past_len+t,:] = k_pe_new  [b,  t,:]
 *   v_cache     [b,h,past_len+t,:] = v_new     [b,h,t,:]
 *   out = attention over rows [0, Tk) of the caches, Tk = past_len + Tq
 *
 * Caches: k_nope_cache / v_cache [B, H, T_cap, 128], k_pe_cache [B, T_cap, 64], device,
 * T_cap >= past_len + Tq rows per (b, h) (per b for k_pe); rows outside [past_len, Tk) are
 * not written.  New rows: k_nope_new / v_new [B, H, Tq, 128], k_pe_new [B, Tq, 64].  The
 * other arguments are those of mla_attn_fwd (kv_len, when given, still hides keys >=
 * kv_len[b]; the new rows are written at past_len regardless).  With Tq == 1 the append
 * is fused into the decode kernel (the stage holding the new row reads it from the new
 * buffers; one CTA per head group writes it to the cache).  With Tq > 1, past_len a
 * multiple of 128 and kv_len NULL it is fused into the prefill kernel: key tiles past the
 * cached prefix are read from the new buffers, and the work unit holding each such tile on
 * its causal diagonal writes it into the caches (every new row is then read by its owner).
 * Other prefills run a copy kernel that appends the rows before the attention kernel.  The
 * output is the same either way.  Errors as for mla_attn_fwd; MLA_ERR_SHAPE also when
 * past_len + Tq > T_cap.
 */
MLA_API mla_status mla_attn_append_fwd(const uint16_t* q_nope, const uint16_t* q_pe,
                                       const uint16_t* k_nope_new, const uint16_t* k_pe_new,
                                       const uint16_t* v_new, uint16_t* k_nope_cache,
                                       uint16_t* k_pe_cache, uint16_t* v_cache,
                                       const int32_t* kv_len, int B, int H, int Tq, int T_cap,
                                       int past_len, float softmax_scale, uint16_t* out,
                                       void* workspace, size_t workspace_bytes,
                                       void* cuda_stream);

/*
 * Attention with a 2D padding mask on the keys.  The model's attention_mask ("Kimi K2 ·
 * Causal mask", section "Construct causal mask") is expanded to 4D and merged with the
 * causal mask, so a hidden key gets the same additive minimum as a causally hidden one:
 *
 *   key j is visible to query i of sequence b iff j <= i + past_len, j < kv_len[b] and
 *   key_mask[b * Tk + j] != 0
 *
 * key_mask: [B, Tk] bytes in device memory (any alignment), nonzero = attend.  Left
 * padding (a run of zeros first) and arbitrary holes are both expressible.  A query row
 * that sees no visible key at all has every score equal to the minimum, so its weights
 * are uniform over all Tk keys: its output is the mean of the Tk value rows (the eager
 * result; such rows are usually padding queries).  The other arguments are those of
 * mla_attn_fwd; the workspace must hold mla_attn_masked_workspace_bytes(B, H, Tq, Tk)
 * bytes (for Tq > 1 it also holds the mask packed to bits).  MLA_ERR_NULL without key_mask.
 */
MLA_API size_t mla_attn_masked_workspace_bytes(int B, int H, int Tq, int Tk);
MLA_API mla_status mla_attn_masked_fwd(const uint16_t* q_nope, const uint16_t* q_pe,
                                       const uint16_t* k_nope, const uint16_t* k_pe_shared,
                                       const uint16_t* v, const int32_t* kv_len,
                                       const uint8_t* key_mask, int B, int H, int Tq, int Tk,
                                       int past_len, float softmax_scale, uint16_t* out,
                                       void* workspace, size_t workspace_bytes,
                                       void* cuda_stream);

/*
 * Decode over the latent cache.  The MLA init excerpt on "Kimi K2 · Similarities" (section
 * "Scale scores") has kv_a_proj_with_mqa produce a 512-wide latent row plus the shared
 * 64-wide rotary key per token, and kv_b_proj map the latent to 64 heads x (128 no-rope
 * key + 128 value).  A cache of latent rows holds 1152 bytes per token instead of the
 * 32,896 of per-head keys and values.  This call computes, for Tq = 1 (query at the last
 * position, causality vacuous) and every head h,
 *
 *   k_nope[b,h,j] = W[256h : 256h+128] . c_kv[b,j]      (no-rope key of key j)
 *   v[b,h,j]      = W[256h+128 : 256h+256] . c_kv[b,j]  (value of key j)
 *   out[b,h]      = the attention core of mla_attn_fwd on [q_nope | q_pe] and
 *                   [k_nope | k_pe], keys j < kv_len[b]
 *
 * without materialising k_nope or v: the no-rope key rows of W are folded into the query
 * (q_lat = W_K^T q_nope), the value rows applied once to the weighted latent sum.  Reading
 * of the weight layout: per head, the first 128 of its 256 kv_b_proj output rows are the
 * no-rope key, the next 128 the value.
 *
 *   q_nope [B, H, 128], q_pe [B, H, 64]           (bf16, device)
 *   c_kv   [B, Tk, 512], k_pe [B, Tk, 64]         (bf16, device: the latent cache)
 *   w_kvb  [H * 256, 512]                         (bf16, device: the kv_b_proj weight)
 *   kv_len [B] int32 or NULL, out [B, H, 128]
 * H must be at most 64.  Workspace: mla_latent_workspace_bytes(B, H, Tk), zeroed once.
 * Errors as for mla_attn_fwd.
 */
MLA_API size_t mla_latent_workspace_bytes(int B, int H, int Tk);
MLA_API mla_status mla_latent_decode_fwd(const uint16_t* q_nope, const uint16_t* q_pe,
                                         const uint16_t* c_kv, const uint16_t* k_pe,
                                         const uint16_t* w_kvb, const int32_t* kv_len, int B,
                                         int H, int Tk, float softmax_scale, uint16_t* out,
                                         void* workspace, size_t workspace_bytes,
                                         void* cuda_stream);

/*
 * Output projection (o_proj) of the attention output.  The MLA init excerpt on "Kimi K2 ·
 * Similarities" (section "Scale scores") ends the attention block with
 * o_proj = nn.Linear(num_heads * v_head_dim, hidden_size, bias = attention_bias); the
 * config.json excerpt on "Kimi K2 · Logits" has hidden_size 7168 and attention_bias false.
 * Reading of its input (the forward's reshape is not shown): the row for (b, i) is the
 * heads' outputs concatenated in head order, feature k = 128 h + d of attn, which is read in
 * place in the layout mla_attn_fwd writes.
 *
 *   attn [B, H, T, 128]   bf16, device
 *   w_o  [N, H * 128]     bf16, device (nn.Linear's weight: out_features x in_features)
 *   y    [B, T, N]        bf16, device, fully overwritten:
 *   y[b, i, n] = sum over h, d of w_o[n, 128 h + d] * attn[b, h, i, d]  (fp32 accumulation)
 * N must be a multiple of 32 and every pointer 16-byte aligned.  Workspace:
 * mla_oproj_workspace_bytes() (the status word), zeroed once.  Errors: MLA_ERR_NULL,
 * MLA_ERR_SHAPE (a size < 1, N not a multiple of 32, a tensor too large), MLA_ERR_ALIGN,
 * MLA_ERR_WORKSPACE, MLA_ERR_DEVICE, MLA_ERR_CUDA; a bounded wait that gives up sets
 * MLA_ERR_TIMEOUT in the status word (mla_attn_get_status).
 */
MLA_API size_t mla_oproj_workspace_bytes(void);
MLA_API mla_status mla_oproj_fwd(const uint16_t* attn, const uint16_t* w_o, int B, int H, int T,
                                 int N, uint16_t* y, void* workspace, size_t workspace_bytes,
                                 void* cuda_stream);

/*
 * Rotary embedding.  The attention excerpt on "Kimi K2 · Similarities" rotates the query's
 * and the new keys' rotary parts before the cache update (rotary_emb gives cos and sin for
 * the positions, apply_rotary_pos_emb rotates q_pe and k_pe), and the rope_scaling block of
 * the config.json excerpt on "Kimi K2 · Logits" selects YaRN scaling (Peng et al., "YaRN:
 * Efficient Context Window Extension of Large Language Models", 2023).  The pages give the
 * calls and the configuration, not the function bodies; the library takes the published
 * YaRN method:
 *   extrapolated f_d = theta^(-2d/64), interpolated f_d / factor   (d = 0..31)
 *   dim(n) = 64 ln(L / (2 pi n)) / (2 ln theta)   (L = original_max_position)
 *   low = floor(dim(beta_fast)), high = ceil(dim(beta_slow)), clamped to [0, 31]
 *   ramp_d = clamp((d - low) / (high - low), 0, 1)   (high == low: high + 0.001)
 *   f_d = interpolated * ramp_d + extrapolated * (1 - ramp_d)
 *   mscale ratio = m(factor, mscale) / m(factor, mscale_all_dim),
 *                  m(s, k) = 0.1 k ln s + 1 for s > 1, else 1
 * and the rotate-half rotation of the 64 rotary columns of a row at position p:
 *   y[d]    = x[d]    * c - x[d+32] * s
 *   y[d+32] = x[d+32] * c + x[d]    * s,     c = cos(p f_d) * ratio, s = sin(p f_d) * ratio
 * Kimi K2's values: theta 50000, factor 32, original_max_position 4096, beta_fast 1,
 * beta_slow 1, mscale 1, mscale_all_dim 1.
 */
typedef struct {
  double rope_theta;            /* > 1 */
  double factor;                /* >= 1 */
  double original_max_position; /* > 0 */
  double beta_fast;             /* >= beta_slow */
  double beta_slow;             /* > 0 */
  double mscale;
  double mscale_all_dim;
} mla_rope_config;

/*
 * Host only: the 32 frequencies f_d and the mscale ratio of a configuration (written
 * through the non-NULL pointers).  MLA_ERR_NULL without cfg; MLA_ERR_ARG for values out of
 * the ranges above or not finite.
 */
MLA_API mla_status mla_rope_frequencies(const mla_rope_config* cfg, double* inv_freq,
                                        double* mscale_ratio);

/*
 * Fills table (device, float, [max_pos][64], 16-byte aligned) with cos(p f_d) * ratio in
 * columns 0..31 and sin(p f_d) * ratio in columns 32..63 for positions p < max_pos; the
 * angles are formed and evaluated in double, then rounded to float.  Build it once per
 * configuration and pass it to mla_attn_rope_append_fwd.  Enqueued on cuda_stream.
 */
MLA_API mla_status mla_rope_table(const mla_rope_config* cfg, int max_pos, float* table,
                                  void* cuda_stream);

/*
 * The same for rotary parts of another width: dim columns (even, 2 .. 256) in place of the 64,
 * dim / 2 frequencies, a table of dim columns (cosines in the first dim / 2).  With factor 1 the
 * angles are the plain p theta^(-2d/dim).  MLA_ERR_SHAPE for other dims.
 */
MLA_API mla_status mla_rope_frequencies_dim(const mla_rope_config* cfg, int dim, double* inv_freq,
                                            double* mscale_ratio);
MLA_API mla_status mla_rope_table_dim(const mla_rope_config* cfg, int dim, int max_pos,
                                      float* table, void* cuda_stream);

/*
 * The rotary step by itself, on rows of any tensor: queries before their attention, keys of a
 * checkpoint whose rotary columns come in neighbouring pairs, cached keys that are turned back,
 * gradients.  Row (t, h) of x is the R elements from x + t * x_row + h * x_head on (strides in
 * elements, the R elements contiguous: a part of a wider head is a slice), and with c, s the
 * columns d and R/2 + d of the table's row positions[t], for d < R/2
 *
 *   (u, v) = elements (d, d + R/2)   (MLA_ROPE_HALF) or (2d, 2d + 1)   (MLA_ROPE_INTERLEAVED)
 *   (u, v) -> (u c - v s, v c + u s),    with inverse (u c + v s, v c - u s)
 *
 * is written to row (t, h) of y in out_layout, rounded once to the tensors' type.  For a table of
 * ratio 1 the inverse undoes the step; for any table the gradient of a step from `layout` to
 * `out_layout` is the inverse step of y's gradient from `out_layout` to `layout`.
 *   x [T, H, R], y [T, H, R]   bf16, fp16 or fp32, both alike; x's strides may be 0, y's rows
 *                              do not overlap; y is x (with its strides), or shares no element
 *                              with it (other memory, or other columns of the same rows)
 *   positions [T] int32        rope_table [table_rows, R] float (mla_rope_table_dim)
 * R even, 2 .. 256.  MLA_ERR_SHAPE, MLA_ERR_ALIGN (a pointer that is no multiple of its element,
 * table and workspace 16 bytes), MLA_ERR_ARG (an option, or a y that overlaps what is read).  A
 * position outside the table is clamped to it (MLA_ERR_KVLEN in the status word).
 * workspace: 256 bytes (the status word), zeroed once.
 */
typedef enum { MLA_TYPE_BF16 = 0, MLA_TYPE_FP16 = 1, MLA_TYPE_FP32 = 2 } mla_type;
typedef enum { MLA_ROPE_HALF = 0, MLA_ROPE_INTERLEAVED = 1 } mla_rope_layout;
MLA_API mla_status mla_rope_apply(const void* x, int64_t x_row, int64_t x_head, void* y,
                                  int64_t y_row, int64_t y_head, int type, int T, int H, int R,
                                  const int32_t* positions, const float* rope_table,
                                  int table_rows, int layout, int out_layout, int inverse,
                                  void* workspace, size_t workspace_bytes, void* cuda_stream);

/* Bytes of workspace mla_attn_rope_append_fwd needs (0 for invalid sizes). */
MLA_API size_t mla_attn_rope_workspace_bytes(int B, int H, int Tq, int Tk);

/*
 * Rotary step + cache append + attention.  As mla_attn_append_fwd, except that q_pe_raw
 * and k_pe_new_raw arrive unrotated: query t and new key t are rotated at position
 * past_len + t with the table from mla_rope_table (table_rows >= past_len + Tq rows, else
 * MLA_ERR_SHAPE); the rotated new keys are what the k_pe cache receives (cached rows are
 * stored rotated and are not rotated again); the rotated queries are kept in the
 * workspace (at least mla_attn_rope_workspace_bytes(B, H, Tq, past_len + Tq) bytes, zeroed
 * once like mla_attn_fwd's).  Rotated values are rounded to bf16, the type of the cache.
 * With Tq == 1 the decode kernel itself rotates the query and the new rotary key (one
 * launch besides the split merge) and appends the new rows.  With Tq > 1 a rotation kernel
 * runs first: for a prefill that fuses the append (past_len a multiple of 128, kv_len
 * NULL; see mla_attn_append_fwd) it only rotates the queries and the new rotary keys into
 * the workspace and the prefill kernel appends all three new rows; otherwise it also writes
 * the rotated keys and the no-rope key and value rows into the caches before the prefill
 * kernel runs.  All host checks run before anything is enqueued.
 */
MLA_API mla_status mla_attn_rope_append_fwd(const uint16_t* q_nope, const uint16_t* q_pe_raw,
                                            const uint16_t* k_nope_new,
                                            const uint16_t* k_pe_new_raw, const uint16_t* v_new,
                                            uint16_t* k_nope_cache, uint16_t* k_pe_cache,
                                            uint16_t* v_cache, const int32_t* kv_len, int B,
                                            int H, int Tq, int T_cap, int past_len,
                                            float softmax_scale, const float* rope_table,
                                            int table_rows, uint16_t* out, void* workspace,
                                            size_t workspace_bytes, void* cuda_stream);

/*
 * Causal attention over whole prompts of different lengths, packed one behind the other: rows
 * cu_seqlens[b] .. cu_seqlens[b+1] - 1 of every tensor are sequence b, and row i of it attends
 * to its rows j <= i.  Per head the core described at the top of this file; the H query heads
 * come in groups of H / Hkv that share one key/value head (Hkv = H: a key/value head each), and
 * all share the rotary key.
 *
 *   q_nope [T, H, 128]    q_pe [T, H, 64]    k_nope, v [T, Hkv, 128]    k_pe [T, 64]
 *   cu_seqlens [B + 1] int32    out [T, H, 128], contiguous
 *
 * strides (elements; NULL: contiguous) lets the inputs be slices of larger tensors, such as the
 * query projection's [T, H, 192] and the key/value projection's [T, Hkv, 256]: the last
 * dimension is contiguous, the others' strides are positive multiples of 8.  Sequences may be
 * empty; rows in front of cu_seqlens[0] and from cu_seqlens[B] on are nobody's, and out is left
 * as it was there.  Another sequence's rows never reach a result, whatever they hold; a later row
 * of the same one takes part with weight zero, so its v has to be finite.
 * Offsets that are not rising within [0, T] are clamped (MLA_ERR_KVLEN in the status word; what
 * their sequences get is not meaningful, and where falling offsets make sequences overlap beyond
 * T / 256 + min(B, T) pairs of 128-row tiles, the sequences behind get nothing).  Workspace:
 * mla_attn_varlen_workspace_bytes(T, B), zeroed once.
 */
typedef struct {
  int64_t q_nope_row, q_nope_head, q_pe_row, q_pe_head;
  int64_t k_nope_row, k_nope_head, k_pe_row, v_row, v_head;
} mla_varlen_strides;
MLA_API size_t mla_attn_varlen_workspace_bytes(int T, int B);
MLA_API mla_status mla_attn_varlen_fwd(const uint16_t* q_nope, const uint16_t* q_pe,
                                       const uint16_t* k_nope, const uint16_t* k_pe,
                                       const uint16_t* v, const mla_varlen_strides* strides,
                                       const int32_t* cu_seqlens, int B, int T, int H, int Hkv,
                                       float softmax_scale, uint16_t* out, void* workspace,
                                       size_t workspace_bytes, void* cuda_stream);

/*
 * ---- Serving over a paged latent cache ---------------------------------------------------
 *
 * The latent cache (512-wide latent row + 64-wide rotary key per token, see
 * mla_latent_decode_fwd) can be held in pages that the sequences of a batch share out
 * between them:
 *
 *   c_pages  [num_pages, page_size, 512]   bf16      page_size a power of two, 16 .. 1024;
 *   pe_pages [num_pages, page_size, 64]    bf16      num_pages * page_size < 2^31
 *   block_table [B, max_pages]             int32     position p of sequence b is row
 *                                                    p % page_size of page
 *                                                    block_table[b, p / page_size]
 *   slot = page * page_size + row                    the same place as one number
 *
 * A step's new tokens are packed: sequence b holds rows cu_q[b] .. cu_q[b+1] - 1 of every
 * per-token tensor.  The per-token tensors may be longer than cu_q[B] (a captured graph has
 * one size for many batches): rows from cu_q[B] on are padding, and outputs are left as they
 * were there unless stated otherwise.
 */

/*
 * Bookkeeping of one step: takes pages for the new tokens from a free list and lists where
 * every token goes.  For sequence b with ctx = ctx_len[b] cached tokens and n = new_len[b]
 * new ones (n may be 0):
 *
 *   cu_q[b]   = new_len[0] + .. + new_len[b-1]      (cu_q[B] = all new tokens)
 *   kv_len[b] = ctx + n
 *   block_table[b, k] for ceil(ctx / page_size) <= k < ceil(kv_len / page_size) receives the
 *               next pages of free_pages, in order of b, then k, starting at free_pages[
 *               free_head[0]]; free_next[0] = the first entry not taken.  No other entry of
 *               the table is written.
 *   slots[t]     = the slot of position ctx + i     (t = cu_q[b] + i)
 *   positions[t] = ctx + depth, where depth is i without `parent`, and with it the number of
 *               ancestors of the token: parent[t] is the index within the sequence's new
 *               tokens of the token's parent (0 <= parent < i), or -1 for a root.
 *   draft_mask[t] (with parent only): bit j set where j is i or an ancestor of i: the form
 *               mla_latent_tree_fwd takes.  At most 64 new tokens per sequence then.
 * Rows t from cu_q[B] to T - 1: slots -1, positions 0, draft_mask 0.
 *
 * No output may overlap an input or another output (blocks read the ones while others write the
 * other; MLA_ERR_ARG); the block table is read and written.  Its entries at or past
 * ceil(ctx / page_size) are taken to be free: a server that drops drafted tokens puts their pages
 * back on its list first.
 * Problems only the device sees go to the status word, and the call completes: lengths below
 * zero or past max_pages * page_size, or more than T new tokens in all (MLA_ERR_KVLEN:
 * lengths are clamped, tokens past the table get slot -1); a free list that runs out, or an
 * entry outside [0, num_pages) (MLA_ERR_PAGE: table entry and slots become -1); a bad parent
 * or a sequence of more than 64 drafted tokens (MLA_ERR_TREE: the token becomes a root; the
 * tokens past 64 see nothing).
 * workspace: 256 bytes (the status word), zeroed once.
 */
MLA_API mla_status mla_paged_plan(const int32_t* ctx_len, const int32_t* new_len, int B,
                                  int32_t* block_table, int max_pages, const int32_t* free_pages,
                                  int n_free, const int32_t* free_head, int page_size,
                                  int num_pages, const int32_t* parent, int T, int32_t* cu_q,
                                  int32_t* kv_len, int32_t* slots, int32_t* positions,
                                  int64_t* draft_mask, int32_t* free_next, void* workspace,
                                  size_t workspace_bytes, void* cuda_stream);

/*
 * Append to the paged latent cache: row t of c_kv_new [T, 512] and k_pe_new [T, 64] goes to
 * slot slots[t] of c_pages / pe_pages; a negative slot marks a row that is skipped.  With
 * rope_table (from mla_rope_table, table_rows rows; positions [T] then required) k_pe_new is
 * unrotated and is rotated at positions[t] on its way, and so is q_pe [T, H, 64], if given,
 * into q_pe_out [T, H, 64] (which may be q_pe itself); rotated values are rounded to bf16.
 * Without rope_table the rows are copied and q_pe must be NULL.
 *
 * Slots must be distinct: of two rows with one slot, the cache keeps some mixture.  A slot
 * past the pool is not written (MLA_ERR_PAGE in the status word), a position outside the table
 * is clamped to it (MLA_ERR_KVLEN).  workspace: 256 bytes (the status word), zeroed once.
 */
MLA_API mla_status mla_latent_append(const uint16_t* c_kv_new, const uint16_t* k_pe_new,
                                     const int32_t* slots, int T, uint16_t* c_pages,
                                     uint16_t* pe_pages, int num_pages, int page_size,
                                     const int32_t* positions, const float* rope_table,
                                     int table_rows, const uint16_t* q_pe, int H,
                                     uint16_t* q_pe_out, void* workspace,
                                     size_t workspace_bytes, void* cuda_stream);

/*
 * Attention of a step's new tokens over the paged latent cache: drafted token trees
 * (speculative decoding), runs of tokens in order, or one token per sequence.
 *
 * The new tokens' own rows are already in the cache (mla_latent_append), as its last rows:
 * with n = cu_q[b+1] - cu_q[b] and ctx = kv_len[b] - n, cached token j < ctx of sequence b is
 * position j and new token i is position ctx + i of the block table's row b.  New token i
 * attends, per head h, to
 *   every key j < ctx, and the keys ctx + k (k < n) with
 *     k <= i                          without draft_mask (tokens in order), or
 *     bit k of draft_mask[t] set      with it (t = cu_q[b] + i; any bits, so a row may see
 *                                     nothing: its output is zero; n <= 64)
 * and the result is that of mla_latent_decode_fwd over those keys:
 *   s_j = softmax_scale * (W_K[h] c_j . q_nope[t,h] + k_pe_j . q_pe[t,h])
 *   out[t,h] = W_V[h] sum_j softmax(s)_j c_j,  fp32 softmax
 * with W_K[h], W_V[h] rows 256 h .. and 256 h + 128 .. of w_kvb.  Cache rows behind kv_len[b]
 * and other sequences' rows never reach a result, whatever they hold; a new key that the mask
 * hides from a row takes part with weight zero, so it has to be finite.
 *
 *   q_nope [T, H, 128], q_pe [T, H, 64], out [T, H, 128]    bf16; rows of out in front of
 *                                       cu_q[0] and from cu_q[B] on are left as they were (a
 *                                       call may take some of a batch's sequences: their
 *                                       entries of cu_q, kv_len and block_table)
 *   c_pages, pe_pages, block_table [B, max_pages], cu_q [B + 1], kv_len [B]    as above
 *   draft_mask [T] int64 or NULL        w_kvb [H * 256, 512] bf16
 * Only the entries of the block table below ceil(kv_len[b] / page_size) are read.
 * H up to 1024, T * H up to 2^26, max_pages * page_size up to 2^30; workspace
 * mla_latent_tree_workspace_bytes(T, H, B) bytes, zeroed once.
 * Device-side problems (the call completes): cu_q not rising within [0, T], kv_len[b] below n
 * or past max_pages * page_size (MLA_ERR_KVLEN, clamped); a page outside the pool
 * (MLA_ERR_PAGE, read as zeros); n > 64 with draft_mask (MLA_ERR_TREE: the keys past 64 are
 * hidden).  The output of such a sequence is not meaningful, but zero if no key is left.
 */
MLA_API size_t mla_latent_tree_workspace_bytes(int T, int H, int B);
MLA_API mla_status mla_latent_tree_fwd(const uint16_t* q_nope, const uint16_t* q_pe,
                                       const uint16_t* c_pages, const uint16_t* pe_pages,
                                       int num_pages, int page_size, const int32_t* block_table,
                                       int max_pages, const int32_t* kv_len, const int32_t* cu_q,
                                       const int64_t* draft_mask, const uint16_t* w_kvb, int B,
                                       int T, int H, float softmax_scale, uint16_t* out,
                                       void* workspace, size_t workspace_bytes,
                                       void* cuda_stream);

/*
 * The attention weight that each cached key receives from a step's new tokens, added to what its
 * slot holds: what mla_paged_evict goes by.  Over the tokens i of sequence b, all heads h and the
 * keys that token i sees (all as in mla_latent_tree_fwd, whose arguments these are), with
 *   s_ihj = softmax_scale * (W_K[h] c_j . q_nope[i,h] + k_pe_j . q_pe[i,h])
 *
 *   weights[slot of j] = decay * weights[slot of j] + sum_{i,h} softmax_j(s_ih)_j   j < ctx, cached
 *                      =                              sum_{i,h} softmax_j(s_ih)_j   a new token's key
 *
 * in fp32.  A score is off by about 2^-16 of |q_lat| . |c_j| and 2^-17 of |W_K[h]|^T |q_nope| . |c_j|
 * + |q_pe| . |k_pe_j| at most, times softmax_scale, with q_lat = W_K[h]^T q_nope: relative to the products
 * that make it up, and not to a score that is a small difference of large ones.  With decay 0 nothing is read
 * from weights, whatever it holds.  A hidden key gets nothing from a row, whatever it holds, and a
 * row that sees nothing gives nothing.  Sequences without new tokens are left as they are, and so
 * are all slots behind kv_len[b].  The weights of one token sum to H.  To let the last tokens of a prompt
 * observe the whole of it, call with those tokens' queries alone and decay 0.
 *
 *   weights [num_pages, page_size] float.  The sequences of a call have pages of their own: a slot
 *   of two of them gets the sum of one.
 * Results do not depend on how the work is shared out but through the order of fp32 sums, which
 * the sizes and lengths fix: the same call gives the same bits.  workspace:
 * mla_latent_key_weights_workspace_bytes(T, H, B, max_pages * page_size) bytes, zeroed once (up to
 * 256 MB of it for scores).  Limits and device-side problems as for mla_latent_tree_fwd; a key on
 * a page outside the pool counts as zeros.  MLA_ERR_ARG for a decay that is not finite.
 */
MLA_API size_t mla_latent_key_weights_workspace_bytes(int T, int H, int B, int max_keys);
MLA_API mla_status mla_latent_key_weights(const uint16_t* q_nope, const uint16_t* q_pe,
                                          const uint16_t* c_pages, const uint16_t* pe_pages,
                                          int num_pages, int page_size,
                                          const int32_t* block_table, int max_pages,
                                          const int32_t* kv_len, const int32_t* cu_q,
                                          const int64_t* draft_mask, const uint16_t* w_kvb, int B,
                                          int T, int H, float softmax_scale, float decay,
                                          float* weights, void* workspace, size_t workspace_bytes,
                                          void* cuda_stream);

/*
 * The rows that a sequence's cache keeps within its budget.  weights [num_pages, page_size] float
 * holds a weight per slot (mla_latent_key_weights accumulates the attention that each cached key
 * receives).  Of sequence b's n = kv_len[b] rows, k = min(n, budget[b]) are kept: all of them if
 * n <= budget[b]; otherwise the first s = min(sinks, k), the last r = min(recent, k - s), and of
 * those between the k - s - r with the largest weights.  Of equal weights the lower rows are kept;
 * NaN counts as lower than any number.
 *
 *   kept[b, i], i < k    the kept rows, rising; -1 for k <= i < K        kept [B, K]
 *   kept_len[b] = k
 *   freed, n_freed       (both or neither) the pages block_table[b, p] with ceil(k / page_size)
 *                        <= p < ceil(n / page_size), in order of b, then p, and their number;
 *                        freed [B * max_pages], entries from n_freed[0] on are left as they were
 *
 * Freed pages are listed as the table has them.  A page that several sequences name (a shared prefix), or
 * one sequence twice, comes up each time that it is past the kept rows, whoever still needs it: a server that
 * shares pages counts their holders.  An entry outside the pool is listed too (and reported,
 * MLA_ERR_PAGE): read the status before the list goes to those that are free.
 *
 * Nothing is moved and the table is not changed: mla_latent_compact moves the rows, in every layer
 * whose pages the table names (a layer may keep other rows than the next, as long as it keeps as
 * many), and only then may the freed pages go to another sequence.  kept_len is then the
 * sequence's cached length.  Positions of later tokens go on from where they were, which is then
 * more than the cached length: mla_paged_plan's positions count from the cached length, so a
 * server adds what it has dropped.
 *
 * K at least every min(kv_len[b], budget[b]); K and max_pages * page_size up to 2^30, B up to 65535,
 * B * max_pages below 2^31; no output may overlap an input or another output (MLA_ERR_ARG, as for
 * negative sinks or recent).
 * Device-side problems (the call completes): a length outside the table, a budget below zero or more
 * rows to keep than K (MLA_ERR_KVLEN, clamped); a page outside the pool (MLA_ERR_PAGE: its rows
 * count as lowest).  workspace: 256 bytes (the status word), zeroed once.
 */
MLA_API mla_status mla_paged_evict(const float* weights, int num_pages, int page_size,
                                   const int32_t* block_table, int max_pages,
                                   const int32_t* kv_len, const int32_t* budget, int B, int sinks,
                                   int recent, int32_t* kept, int K, int32_t* kept_len,
                                   int32_t* freed, int32_t* n_freed, void* workspace,
                                   size_t workspace_bytes, void* cuda_stream);

/*
 * Moves the kept rows of every sequence to the front of its pages: for i < kept_len[b], row
 * kept[b, i] of sequence b becomes its row i, in c_pages [num_pages, page_size, 512], pe_pages
 * [num_pages, page_size, 64] and, if given, weights [num_pages, page_size] (float).  Other rows
 * keep what they held, or hold what a moved row left behind.  The cached keys keep the rotary
 * angles that they have.
 *
 * kept [B, K] int32, each row rising, as mla_paged_evict lists it (any rising list of rows will
 * do); kept_len [B].  The sequences of a call have pages of their own: a page that two of them
 * name is moved by both at once, and holds some mixture.  K and max_pages * page_size up to 2^30, B
 * up to 65535, B * K up to 2^35.
 * Device-side problems (the call completes): kept_len outside [0, K] (MLA_ERR_KVLEN, clamped); an
 * entry below its own index or past the table (MLA_ERR_KVLEN), or a page outside the pool
 * (MLA_ERR_PAGE): that row is not moved.  A list that does not rise moves rows that others have
 * overwritten.  workspace: mla_latent_compact_workspace_bytes(B, K) bytes, zeroed once.
 */
MLA_API size_t mla_latent_compact_workspace_bytes(int B, int K);
MLA_API mla_status mla_latent_compact(uint16_t* c_pages, uint16_t* pe_pages, float* weights,
                                      int num_pages, int page_size, const int32_t* block_table,
                                      int max_pages, const int32_t* kept, int K,
                                      const int32_t* kept_len, int B, void* workspace,
                                      size_t workspace_bytes, void* cuda_stream);

/*
 * Synchronises cuda_stream, reads the device status word in the workspace, clears it,
 * and returns it (MLA_OK if no kernel recorded a problem since the last read).
 */
MLA_API mla_status mla_attn_get_status(void* workspace, void* cuda_stream);

/* Static, human-readable name of a status code. */
MLA_API const char* mla_status_string(mla_status status);

/*
 * The decode scheduler's choice for these sizes: keys per split and number of splits
 * (written through the non-NULL pointers).  Pure host arithmetic; returns MLA_ERR_SHAPE
 * for invalid sizes.
 */
MLA_API mla_status mla_attn_decode_plan(int B, int H, int Tk, int* chunk, int* splits);

/*
 * Decode (Tq == 1, past_len = Tk - 1) without a caller-provided workspace.  The pages
 * have no counterpart to this call: it exists for callers that cannot allocate device
 * memory for the library (a server whose KV-cache pool owns all free HBM, a plugin inside
 * a framework whose allocator owns the device, a loop that cannot afford cudaMalloc's
 * implicit synchronisation).  The split-KV partials live in a 32 MiB array inside the
 * library image, which every GPU that loads the library holds until the process exits.
 *
 * Arguments and result are those of mla_attn_fwd with Tq = 1 and the same split plan, so
 * the output matches mla_attn_fwd's.  device_status (device int, may be NULL) receives
 * device-detected errors (MLA_ERR_KVLEN, MLA_ERR_TIMEOUT) the way the workspace status
 * word does; the caller zeroes and reads it.  Pass it: with device_status NULL those
 * errors go unreported, and after a bounded wait gives up (a split that never wrote its
 * partial) the merge may read partials a previous call left in the array, so the output
 * is undefined without any sign of it.  Returns MLA_ERR_WORKSPACE when the plan for these
 * sizes needs more than the 32 MiB array (B * H * splits partials of 520 bytes each).
 *
 * The call allocates nothing.  Its first call on a device looks up the array's device
 * address (cudaGetSymbolAddress) with that device current and keeps it for the rest of
 * the process; make that first call before any stream capture.  The kept address belongs
 * to the device's context of that time: after cudaDeviceReset on that device it is stale,
 * so do not call this function on a device that has been reset since its first call.  All
 * calls share the array: calls that overlap on the GPU (other streams, other host
 * threads) race on it and must be serialised by the caller.
 */
MLA_API mla_status mla_attn_decode_noalloc(const uint16_t* q_nope, const uint16_t* q_pe,
                                           const uint16_t* k_nope, const uint16_t* k_pe_shared,
                                           const uint16_t* v, const int32_t* kv_len, int B,
                                           int H, int Tk, float softmax_scale, uint16_t* out,
                                           int* device_status, void* cuda_stream);

#ifdef __cplusplus
}
#endif

#endif /* MLA_ATTN_H_ */
