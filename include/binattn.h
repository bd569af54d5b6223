/*
 * binattn.h — C ABI of the BinaryAttention forward pass for NVIDIA B200 (sm_100a).
 *
 * The method (paper "BinaryAttention: One-Bit QK-Attention for Vision and Diffusion
 * Transformers", arXiv 2603.09582; cited below through its summary pages
 * gist.science/<lang>/paper/2603.09582):
 *   s_ij = alpha * x_ij + b_ij,     x_ij = d - 2 popc(sign bits of q_i XOR sign bits of k_j),
 *   alpha = softmax_scale * mu_q * mu_k,  mu = mean |x| of the (batch, head) slice,
 *   online softmax over key blocks of ba_kv_block() keys in ascending order,
 *   P_ij = rne(255 * exp(s_ij - m_t)) as uint8 (m_t = running row max after block t),
 *   V quantised per (batch, head, channel) to int8 with scale amax/127,
 *   O = (integer P.V accumulated per block, rescaled between blocks) * v_scale / (255 l).
 *
 * Conventions shared by every entry point:
 *   - Tensors are contiguous, row-major, [B][H][N][d] unless stated otherwise.
 *   - Every pointer argument is a DEVICE pointer owned by the caller, aligned to 16 bytes.
 *     The library never allocates, frees or keeps a pointer after the call returns.
 *   - Work is enqueued on `stream` (a cudaStream_t passed as void*; NULL = legacy default
 *     stream). No call synchronises the host. Calls on different streams are independent
 *     provided each uses its own workspace.
 *   - Arguments are validated before anything is launched; on an error nothing is
 *     enqueued and a status code is returned. Launch failures return BA_ERR_CUDA
 *     (ba_last_cuda_error() gives the cudaError_t).
 *   - Supported sizes: 1 <= d <= 128, 0 <= B, H, N; B*H <= 65536; N <= 1048576. Empty
 *     problems (B, H or N = 0) return BA_OK and launch nothing.
 */
#ifndef BINATTN_H
#define BINATTN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  BA_OK = 0,
  BA_ERR_INVALID_ARG = 1,   /* null pointer, negative size, bad enum, inconsistent bias */
  BA_ERR_UNSUPPORTED = 2,   /* d outside [1,128], sizes beyond the limits above */
  BA_ERR_ALIGNMENT = 3,     /* a pointer not aligned to 16 bytes */
  BA_ERR_WORKSPACE = 4,     /* workspace missing or smaller than required */
  BA_ERR_CUDA = 5,          /* a CUDA launch or runtime call failed */
  BA_ERR_TIMEOUT = 6        /* a bounded device-side wait expired (see ba_check_device_status) */
} ba_status;

typedef enum { BA_F16 = 0, BA_BF16 = 1, BA_F32 = 2 } ba_dtype;  /* F32 is accepted for O only */

typedef enum { BA_BIAS_NONE = 0, BA_BIAS_DENSE = 1, BA_BIAS_RELPOS2D = 2 } ba_bias_kind;

/*
 * The additive logit bias b_ij ("bias enhancement": gist.science/zh, technical summary
 * 2.2(2); gist.science/it, sintesi tecnica 2B — dense or position-sensitive). It is
 * added after the alpha scaling and is not scaled. Values must be finite.
 *   BA_BIAS_DENSE:    data = fp32 [H][N][N] for batch 0; batch b reads data + b*batch_stride
 *                     (batch_stride = 0 broadcasts one tensor over the batch).
 *   BA_BIAS_RELPOS2D: data = fp32 [H][(2*table_h-1)*(2*table_w-1)]. Token t >= n_prefix sits
 *                     at (y, x) = ((t-n_prefix) / grid_w, (t-n_prefix) % grid_w) with
 *                     grid_h*grid_w = N - n_prefix; b_ij = data[h][(y_i-y_j+table_h-1)*(2*table_w-1)
 *                     + (x_i-x_j+table_w-1)]; rows and columns of prefix tokens get 0.
 *                     Requires table_h >= grid_h and table_w >= grid_w.
 */
typedef struct {
  ba_bias_kind kind;
  const float* data;
  int64_t batch_stride;
  int grid_h, grid_w;
  int table_h, table_w;
  int n_prefix;
} ba_bias;

/* Words per packed sign row: 4 (128 bits, one 16-byte row) for 1 <= d <= 128, else 0. */
int ba_sign_words(int d);

/* Bytes per quantised V row: d rounded up to a multiple of 16 (pad bytes are 0). */
int ba_v_row_bytes(int d);

/* Key block of the online softmax: the 8-bit P codes depend on it (128). */
int ba_kv_block(void);

/*
 * The exact-code thresholds the tcgen05 kernel uses near a rounding tie: for 0 <= k <= 254, the
 * least double d whose code min(255, rne(fl32(255 * fl32(exp(d))))) exceeds k (the code of a
 * logit s against the running max m, with d = (double)s - (double)m; gist.science/zh 2.2(3)).
 * NaN for any other k. Host-side; computed once per process.
 */
double ba_p_code_threshold(int k);

/*
 * Preparation path ba_attention_fwd takes for this shape: 1 = one launch (one CTA per (b, h)
 * slice and tensor writes the sign bits and mu of q and k and the scales and int8 rows of v;
 * taken for many short slices with d a multiple of 8 and d >= 32), 0 = three launches
 * (128-token chunks with partial sums, a finalize kernel, the V quantiser). A host query: it
 * launches nothing and reports the choice only; both paths compute the same values.
 */
int ba_prep_fused(int B, int H, int N, int d);

/* Workspace sizes in bytes (0 for empty problems; -1 cast to size_t for unsupported d). */
size_t ba_pack_workspace_bytes(int B, int H, int N, int d);
size_t ba_quant_workspace_bytes(int B, int H, int N, int d);
size_t ba_workspace_bytes(int B, int H, int N, int d);

/*
 * Sign binarisation and the scale factor mu (gist.science/zh 2.2(1): s_i = mu_q sign(q_i),
 * mu averaging |x| over every token and channel of the (b, h) slice; gist.science/nl
 * Methodologie 2).
 *   x:    [B][H][N][d] in dt (BA_F16 or BA_BF16).
 *   bits: [B][H][N][4] uint32 out. Bit (c % 32) of word c/32 is 1 iff x_c < 0 (IEEE: -0.0,
 *         +0.0 and NaN give 0); bits at c >= d are 0.
 *   mu:   [B][H] fp32 out, mean of |x| over the N*d entries of each (b, h) slice (x must be
 *         finite: mu of a slice holding inf or NaN is unspecified).
 *   ws:   at least ba_pack_workspace_bytes(B,H,N,d) bytes of device memory (partial sums).
 */
ba_status ba_pack_signs(const void* x, ba_dtype dt, int B, int H, int N, int d, uint32_t* bits,
                        float* mu, void* ws, size_t ws_bytes, void* stream);

/*
 * Channel-aware 8-bit V (gist.science/zh 2.2(3); gist.science/nl Methodologie 2: a
 * channel-specific scale). Per (b, h, c): amax = max_j |v_jc|, inv = 127/amax (fp32),
 * q = clamp(rne(v * inv), -127, 127), v_scale = amax/127; a zero channel gives q = 0 and
 * v_scale = 0. v must be finite (the codes of a channel holding inf or NaN are unspecified).
 *   v:       [B][H][N][d] in dt (BA_F16 or BA_BF16).
 *   vq:      [B][H][N][ba_v_row_bytes(d)] int8 out, pad columns 0.
 *   v_scale: [B][H][d] fp32 out.
 *   ws:      at least ba_quant_workspace_bytes(B,H,N,d) bytes (per-chunk maxima).
 */
ba_status ba_quant_v(const void* v, ba_dtype dt, int B, int H, int N, int d, int8_t* vq,
                     float* v_scale, void* ws, size_t ws_bytes, void* stream);

/*
 * The fused forward on pre-packed operands (gist.science/zh 2.3 and gist.science/it
 * sintesi tecnica 2C: a FlashAttention-2-style tiled kernel with binary QK and an
 * unsigned-8-bit x signed-8-bit P.V accumulated in 32-bit integers).
 *   bits_q, bits_k: [B][H][N][4] from ba_pack_signs; mu_q, mu_k: [B][H].
 *   vq, v_scale:    from ba_quant_v.
 *   bias:           NULL or kind BA_BIAS_NONE for no bias.
 *   softmax_scale:  <= 0 selects 1/sqrt(d); alpha = (softmax_scale * mu_q) * mu_k in fp32.
 *   o:              [B][H][N][d] out in o_dt (BA_F16, BA_BF16 or BA_F32).
 *   dbg_logits:     NULL, or [B][H][N][N] int32 out receiving x_ij (debug; large).
 */
ba_status ba_attention_fwd_packed(const uint32_t* bits_q, const float* mu_q, const uint32_t* bits_k,
                                  const float* mu_k, const int8_t* vq, const float* v_scale, int B,
                                  int H, int N, int d, const ba_bias* bias, float softmax_scale,
                                  void* o, ba_dtype o_dt, int32_t* dbg_logits, void* stream);

/*
 * The whole forward pass: the results of ba_pack_signs(q), ba_pack_signs(k) and ba_quant_v(v)
 * into the workspace (in one launch for the shapes ba_prep_fused reports, else three), then
 * the fused step of ba_attention_fwd_packed.
 *   q, k, v: [B][H][N][d] in dt (BA_F16 or BA_BF16).
 *   ws:      at least ba_workspace_bytes(B,H,N,d) bytes; its contents on return are the
 *            packed operands (layout private to the library).
 */
ba_status ba_attention_fwd(const void* q, const void* k, const void* v, ba_dtype dt, int B, int H,
                           int N, int d, const ba_bias* bias, float softmax_scale, void* o,
                           ba_dtype o_dt, void* ws, size_t ws_bytes, int32_t* dbg_logits,
                           void* stream);

/*
 * ba_attention_fwd with debug outputs, for tests and diagnosis (slower; not for production use).
 *   dbg_logits:      NULL, or [B][H][N][N] int32 receiving x_ij.
 *   dbg_p:           NULL, or [B][H][N][N] uint8 receiving the 8-bit code P_ij of every key, taken
 *                    against the running maximum of the key's block (the codes the P.V product
 *                    uses; gist.science/zh 2.2(3)).
 *   check_all_codes: 0 = as ba_attention_fwd: the tensor-core kernel evaluates exp with the
 *                    hardware approximation and recomputes from the double-precision exponential
 *                    every code within its error band of a rounding tie in those blocks where a
 *                    changed code could move the output by more than a tenth of the 2e-3 error
 *                    bar (rows whose softmax sum is still small); 1 = in every block, so that every
 *                    code equals the definition's.  Other values: BA_ERR_INVALID_ARG.
 *   Other arguments and errors as ba_attention_fwd (dbg_p must be 16-byte aligned).
 */
ba_status ba_attention_fwd_debug(const void* q, const void* k, const void* v, ba_dtype dt, int B, int H,
                                 int N, int d, const ba_bias* bias, float softmax_scale, void* o,
                                 ba_dtype o_dt, void* ws, size_t ws_bytes, int32_t* dbg_logits,
                                 uint8_t* dbg_p, int check_all_codes, void* stream);

/*
 * ba_attention_fwd without a caller-supplied workspace (the paper has no counterpart; this
 * is a deployment convenience). For callers that cannot allocate device memory: a plugin that
 * is handed only its input and output buffers, or a runtime that fixes all device memory at
 * start-up and forbids cudaMalloc afterwards (it can synchronize the device and bypasses the
 * host's allocator). The workspace comes from a fixed array of BA_NOALLOC_SCRATCH_BYTES in the
 * library's device memory, held by every GPU that loads the library until the process exits.
 *   - Arguments as ba_attention_fwd, minus ws / ws_bytes.
 *   - Problems with ba_workspace_bytes(B,H,N,d) > BA_NOALLOC_SCRATCH_BYTES return
 *     BA_ERR_WORKSPACE before anything is launched.
 *   - All calls share the array: calls that can overlap on the GPU (unordered streams) race
 *     and must be ordered by the caller. Its contents persist between calls; none of it needs
 *     to start at zero.
 *   - The first call on each device looks up the array's device address (and caches it);
 *     make that first call before any stream capture. The cache assumes the device's primary
 *     context lives as long as the process (no cudaDeviceReset between calls).
 *   - Allocates nothing: no cudaMalloc, cudaFree or other allocating routine.
 */
#define BA_NOALLOC_SCRATCH_BYTES (32u * 1024u * 1024u)
ba_status ba_attention_fwd_noalloc(const void* q, const void* k, const void* v, ba_dtype dt, int B, int H,
                                   int N, int d, const ba_bias* bias, float softmax_scale, void* o,
                                   ba_dtype o_dt, int32_t* dbg_logits, void* stream);

/*
 * ------------------------------------------------------------------ paged KV cache
 * The binary attention of token sequences that grow: new K and V rows are quantised once, as
 * they are written into a paged cache, and attention of new tokens reads them there.
 *
 * The scale of a key and of a value row cannot wait for the rows that follow, so both are per
 * (token, head):
 *   k^_c = mu * (1 - 2 bit_c),  bit_c = 1 iff k_c < 0 (as ba_pack_signs),
 *          mu = mean_c |k_c| rounded to bf16;
 *   v^_c = code_c * 2^e,  e = the least integer with max_c |v_c| <= 127 * 2^e, held to
 *          [-24, 9], code_c = rne(v_c * 2^-e) held to [-127, 127]; a zero row has e = -24.
 * mu in bf16 makes every k^_c a bf16 number, and the power of two makes every v^_c an fp16
 * number (values beyond 127 * 2^9 = 65024 saturate there): the attention kernels feed both to
 * the tensor cores without another rounding. A row takes dp + 19 bytes (dp = ba_v_row_bytes(d)):
 * 147 at d = 128, where K and V in 16 bits take 512.
 *
 * Layout: data holds num_pages * n_kv_heads blocks [page][head] of ba_kv_block_bytes() bytes,
 * each with the rows of page_size tokens:
 *   int8   codes[page_size][dp]   (columns >= d are 0)
 *   uint32 bits[page_size][4]     (bits >= d are 0)
 *   bf16   mu[page_size]
 *   int8   e[page_size]
 * A token's slot is page * page_size + its offset in the page.
 */
typedef struct {
  void* data;        /* device memory, aligned to 16 bytes */
  int64_t num_pages; /* >= 0 */
  int page_size;     /* tokens per page: a multiple of 16, 16 to 1024 */
  int n_kv_heads;    /* 1 to 65535 */
  int d;             /* 1 to 128 */
} ba_kv_cache;

/* Bytes of one (page, head) block: page_size * (dp + 19), a multiple of 16; 0 for sizes outside
 * the limits above. */
size_t ba_kv_block_bytes(int page_size, int d);

/*
 * Quantises T new tokens and writes them into the cache.
 *   k, v:  row (t, h) starts at element t * stride_t + h * stride_h and has d contiguous elements
 *          of dt (BA_F16 or BA_BF16): slices of a fused projection are taken as they are. These
 *          two pointers need the alignment of their elements only (rows on 16-byte boundaries
 *          with d a multiple of 8 are read with wide loads). Values must be finite (a row with
 *          inf or NaN gets unspecified contents; other rows are not affected).
 *   slots: [T] int64 (aligned to 8 bytes), the slot of each token. A slot outside
 *          [0, num_pages * page_size) is skipped (padding: -1). A slot named twice in a call
 *          ends with an unspecified mixture of its rows: slots in range have to differ.
 */
ba_status ba_cache_write(const void* k, int64_t k_stride_t, int64_t k_stride_h, const void* v,
                         int64_t v_stride_t, int64_t v_stride_h, ba_dtype dt, int64_t T,
                         const int64_t* slots, const ba_kv_cache* cache, void* stream);

/*
 * Reads T rows back: k[t][h][c] = k^, v[t][h][c] = v^ of the token in slots[t], contiguous
 * [T][n_kv_heads][d] in dt (any ba_dtype; k^ is rounded to fp16 where dt is BA_F16, all else is
 * exact). Rows whose slot is out of range are 0. k or v may be NULL (not wanted). A slot may be
 * named any number of times.
 */
ba_status ba_cache_read(const ba_kv_cache* cache, const int64_t* slots, int64_t T, void* k, void* v,
                        ba_dtype dt, void* stream);

/*
 * Attention of new tokens over the paged cache, for any mix of sequence lengths: one token each
 * (decoding), a few (drafts), or a chunk of a prompt. The new tokens' own K and V rows are in the
 * cache already (ba_cache_write), as the last ones of their sequence.
 *
 * Sequence b has the rows cu_seqlens_q[b] .. cu_seqlens_q[b + 1] - 1 of q and o, n of them, and
 * kv_lens[b] tokens in the cache, token j in page page_table[b][j / page_size]. Its i-th new token
 * is at position p = kv_lens[b] - n + i and sees the tokens j < kv_lens[b] with
 *   causal:      j <= p
 *   window > 0:  j > p - window, or j < sinks  (the first tokens stay visible)
 * Query heads g * G .. g * G + G - 1 use KV head g, G = n_heads / n_kv_heads.
 *   s_j = softmax_scale * mu_q * mu_j * (d - 2 popc(sign bits of q XOR sign bits of k_j)),
 *   mu_q = mean |q| of the row in fp32;  o = sum_j exp(s_j) v^_j / sum_j exp(s_j),
 *   lse = log sum_j exp(s_j).
 * There is no 8-bit P here. For many rows the weights are rounded to fp16 for the product with V,
 * which accumulates in fp32: off by at most 2^-11 of themselves, or, far below the row's largest
 * weight, 2^-28 of that one. For few rows (max_q_len * G up to 32, or 128 where there
 * is little work) they are rounded to 16 bits below the largest weight * 2^e of 64 keys (2^-17 of it), products are exact and their
 * sums of 64 keys are added in fp32. Scores, maxima and sums are fp32. A row that sees nothing gets
 * o = 0 and lse = -inf.
 * Rows of the cache that no new token sees may hold anything. A row of o and lse is unspecified where
 * softmax_scale * mu_q * d or mu_j * d of a key that it sees is beyond fp32's range, or a score s_j beyond
 * +-2^24, where neighbouring fp32 numbers lie more than 1 apart.
 * BA_ERR_UNSUPPORTED where T * n_heads passes 2^31 - 4096, where the bounds make more than 2^31 - 1 tiles
 * (B * n_kv_heads * ceil(max_q_len * G / 256); 8 or 16 rows a tile with few), or where tiles * max_kv_len
 * passes some 2^44.
 */
typedef struct {
  int B;                       /* sequences */
  int64_t T;                   /* rows of q and o; rows of no sequence are left as they were */
  int n_heads;                 /* query heads, a multiple of the cache's n_kv_heads */
  int max_q_len;               /* >= every sequence's new tokens; rows beyond are left as they were */
  int64_t max_kv_len;          /* >= every kv_lens[b] (what is beyond it is not read); <= 2^28 */
  const int32_t* cu_seqlens_q; /* [B + 1] ascending, or NULL: sequence b has the one row b */
  const int32_t* kv_lens;      /* [B] */
  const int32_t* page_table;   /* [B] rows of table_stride entries, the first max_pages of them valid;
                                  a token whose page is outside [0, num_pages) is not seen */
  int64_t table_stride;
  int max_pages;
  int causal;                  /* 0 or 1 */
  int window;                  /* 0: none; > 0 wants causal = 1 */
  int sinks;                   /* >= 0 */
} ba_paged_seqs;

/* Workspace of ba_attention_paged in bytes (partial sums of a split key axis; 0 when none is
 * needed), or -1 cast to size_t for arguments that the call refuses. Reads no device memory. */
size_t ba_paged_workspace_bytes(const ba_kv_cache* cache, const ba_paged_seqs* seqs);

/*
 *   q:   row (t, h) starts at element t * q_stride_t + h * q_stride_h, d contiguous elements of dt
 *        (BA_F16 or BA_BF16), aligned to its elements; values must be finite.
 *   o:   [T][n_heads][d] contiguous in o_dt (any ba_dtype).
 *   lse: NULL, or [T][n_heads] fp32 out.
 *   softmax_scale: <= 0 selects 1/sqrt(d).
 *   The device arrays of seqs are aligned to 4 bytes. Lengths are read on the device, so a captured
 *   call can be replayed with other lengths within max_q_len and max_kv_len.
 */
ba_status ba_attention_paged(const void* q, int64_t q_stride_t, int64_t q_stride_h, ba_dtype dt,
                             const ba_kv_cache* cache, const ba_paged_seqs* seqs, float softmax_scale,
                             void* o, ba_dtype o_dt, float* lse, void* ws, size_t ws_bytes, void* stream);

/*
 * Kernel choice for the fused step, process-wide: 0 = automatic (the tcgen05 tensor-core
 * kernel where it supports the shape, else the CUDA-core kernel), 1 = the CUDA-core kernel,
 * 2 = the tcgen05 kernel (BA_ERR_UNSUPPORTED for shapes it does not take).
 */
ba_status ba_set_attention_impl(int impl);
int ba_get_attention_impl(void);

/* The kernel the last successful fused call on this thread ran: 1 CUDA-core, 2 tcgen05. */
int ba_last_attention_impl(void);

/*
 * Synchronises `stream` and reads (then clears) the device status words that kernels set
 * when a bounded wait expires. Returns BA_OK or BA_ERR_TIMEOUT (or BA_ERR_CUDA, with nothing cleared).
 */
ba_status ba_check_device_status(void* stream);

/*
 * Stage timing for measurement tools (off by default). While enabled, ba_attention_fwd
 * records a CUDA event on its stream before its first kernel and after each stage: the
 * q/k/v streaming pass, the finalize pass, the V quantiser and the fused attention kernel
 * (on the one-launch preparation path the finalize and quantiser stages are empty).
 * ba_stage_times synchronises on those events and writes the device time of each of the
 * four stages in milliseconds, summed over the calls since the last read, to ms[0..n-1]
 * (n <= 4), stores the number of calls in *calls, and forgets them.
 */
ba_status ba_stage_timing(int enable);
ba_status ba_stage_times(float* ms, int n, int* calls);

/* Human-readable status; the cudaError_t behind the last BA_ERR_CUDA on this thread. */
const char* ba_status_string(ba_status s);
int ba_last_cuda_error(void);

#ifdef __cplusplus
}
#endif

#endif /* BINATTN_H */
