/*
 * tsd_attention.h -- C ABI of the GB300 (sm_103a) multi-head scaled
 * dot-product attention library (libtsd_attention.so).
 *
 * The operation is eq. (1) of "Attention Is All You Need",
 *     Attention(Q, K, V) = softmax(Q K^T / sqrt(d_k)) V,
 * a query mapped against a set of key/value pairs to a weighted sum of the
 * values ("[논문 리뷰]Attention Is All You Need" (kimjiil.github.io),
 * section 3.2 / 3.2.1), applied per head, and multi-head attention
 *     MultiHead = Concat(head_1..head_h) W^O,
 *     head_i = Attention(X_q W_i^Q, X_kv W_i^K, X_kv W_i^V)
 * (same page, section 3.2.2). Masks set the illegal logits to -inf before
 * the softmax so their weight is exactly 0 (same page, section 3.2.3;
 * "Attention Is All You Need 해부" (sj-techlog), section "mask는 softmax
 * **전**에 더해야 한다").
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 *  - All tensor pointers are DEVICE pointers owned by the caller; the library
 *    never frees, retains or allocates device memory on a call. Every call is
 *    asynchronous on `stream` (a cudaStream_t; NULL is the legacy default
 *    stream) and returns before the GPU work finishes.
 *  - Layouts are row-major and contiguous. bf16 tensors hold IEEE bfloat16
 *    bit patterns (uint16); f32 tensors hold IEEE binary32.
 *  - Host-detected argument errors return before anything is launched.
 *  - kv_lens values are clamped on the device to [0, n_k]. A query row with
 *    no allowed key (kv_len = 0) produces an all-zero output row.
 *  - Kernels never trap or assert. Every wait inside a kernel is bounded;
 *    a kernel that gives up sets a device error word and exits cleanly,
 *    which attn_get_device_status() reports. A kernel whose warp groups
 *    trade registers is not launched when the build gave it fewer registers
 *    per thread than that trade assumes (ATTN_ERR_CUDA,
 *    cudaErrorInvalidConfiguration): it could otherwise wait for registers
 *    that are never released.
 */
#ifndef TSD_ATTENTION_H
#define TSD_ATTENTION_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* A cudaStream_t, declared without pulling in the CUDA headers. */
typedef struct CUstream_st *tsd_stream_t;

typedef enum attn_status {
    ATTN_OK = 0,
    ATTN_ERR_INVALID = 1,        /* an argument is invalid; nothing was launched */
    ATTN_ERR_UNSUPPORTED = 2,    /* valid for eq. (1) but outside what this build runs
                                    (e.g. a head size the bf16 kernel has no variant for) */
    ATTN_ERR_CUDA = 3,           /* a CUDA runtime/driver call failed; see attn_last_cuda_error() */
    ATTN_ERR_DEVICE_TIMEOUT = 4, /* a kernel's bounded wait ran out (attn_get_device_status) */
    ATTN_ERR_DEVICE_INDEX = 5,   /* a page index, or a new token's position, was out of range: its
                                    row was left out (attn_get_device_status) */
    ATTN_ERR_DEVICE_VALUE = 6    /* a beam's logits or score held a NaN or +infinity: the beam was
                                    left out (attn_get_device_status) */
} attn_status;

/* mask_kind bit flags */
enum {
    ATTN_MASK_NONE = 0,
    ATTN_MASK_CAUSAL = 1,       /* query i sees keys j <= i; requires n_q == n_k
                                   (decoder masked self-attention, section 3.2.3) */
    ATTN_MASK_KEY_PADDING = 2   /* keys j >= kv_lens[b] receive no attention
                                   ("Attention Is All You Need 해부", three-uses table) */
};

/*
 * attn_forward -- scaled dot-product attention, bf16 in/out, fp32 softmax and
 * accumulation, on the tcgen05 tensor cores.
 *
 *   q    [B, h, n_q, d_k]  bf16, device, 16-byte aligned
 *   k    [B, h, n_k, d_k]  bf16, device, 16-byte aligned
 *   v    [B, h, n_k, d_v]  bf16, device, 16-byte aligned
 *   out  [B, h, n_q, d_v]  bf16, device, 16-byte aligned, written in full
 *   d_k == d_v, and d_k in {16, 32, 64, 128, 256}   else ATTN_ERR_UNSUPPORTED
 *     (16, 32 and 256 are the head sizes of Table 3 (A), "[논문 리뷰]Attention
 *     Is All You Need" (kimjiil.github.io), section 6.2; 64 is the base model's)
 *   B, h, n_q, n_k >= 0                      else ATTN_ERR_INVALID
 *     (a zero size launches nothing; n_k = 0 writes all-zero output rows)
 *   mask_kind: OR of ATTN_MASK_* bits; CAUSAL needs n_q == n_k
 *   kv_lens: device int32[B]; required with ATTN_MASK_KEY_PADDING, ignored otherwise
 *   scale: the logit factor; 0 selects 1/sqrt(d_k) (eq. (1))
 * Errors: null/misaligned pointer, bad sizes or flags -> ATTN_ERR_INVALID;
 * a failed launch -> ATTN_ERR_CUDA.
 */
attn_status attn_forward(const void *q, const void *k, const void *v, void *out,
                         int B, int h, int n_q, int n_k, int d_k, int d_v,
                         int mask_kind, const int32_t *kv_lens, float scale,
                         tsd_stream_t stream);

/*
 * encoder_layer_forward -- one Transformer encoder layer, both sub-layers
 * wrapped post-LN as output = LayerNorm(x + Sublayer(x)) ("[논문 리뷰]
 * Attention Is All You Need" (kimjiil.github.io), sections 3.1 and 3.3;
 * LayerNorm(v) = gamma (v - mu) / sqrt(sigma^2 + eps) + beta over one token's
 * d_model features, "Attention Is All You Need 해부" (sj-techlog), section
 * "4. residual connection과 LayerNorm"):
 *   y   = LayerNorm_1(x + MultiHead(x, x))            (mha_forward, self-attention)
 *   out = LayerNorm_2(y + FFN(y)),  FFN(y) = max(0, y W_1 + b_1) W_2 + b_2
 *   x, out   [B, n, d_model] bf16, device; d_model in {256, 512, 1024, 2048}
 *            (else ATTN_ERR_UNSUPPORTED)
 *   w_q, w_k, w_v, w_o: as mha_forward with d_v = d_k (d_model x h*d_k, h*d_k x d_model)
 *   ln1_gamma, ln1_beta, ln2_gamma, ln2_beta: [d_model] bf16
 *   w_1 [d_model, d_ff], b_1 [d_ff], w_2 [d_ff, d_model], b_2 [d_model], bf16;
 *   d_ff a multiple of 8
 *   mask_kind, kv_lens, scale: as mha_forward (self-attention, n_q = n_k = n)
 *   eps: LayerNorm's epsilon (> 0; the pages do not give a value)
 *   workspace: device, 256-byte aligned, >= encoder_layer_workspace_bytes(...)
 *   bytes; scratch (it holds mha_forward's workspace, the attention output,
 *   y, the FFN's hidden layer and y + FFN(y)).
 * Errors: as mha_forward; eps <= 0 -> ATTN_ERR_INVALID. Launches: mha_forward's
 * plus four (LayerNorm, the two FFN GEMMs with their bias / ReLU / residual
 * epilogues, LayerNorm).
 */
size_t encoder_layer_workspace_bytes(int B, int n, int d_model, int h, int d_k, int d_ff);
attn_status encoder_layer_forward(const void *x,
                                  const void *w_q, const void *w_k, const void *w_v,
                                  const void *w_o,
                                  const void *ln1_gamma, const void *ln1_beta,
                                  const void *w_1, const void *b_1,
                                  const void *w_2, const void *b_2,
                                  const void *ln2_gamma, const void *ln2_beta,
                                  void *out,
                                  int B, int n, int d_model, int h, int d_k, int d_ff,
                                  int mask_kind, const int32_t *kv_lens, float scale, float eps,
                                  void *workspace, size_t workspace_bytes, tsd_stream_t stream);

/*
 * attn_decode -- one decoding step against a key/value cache ("Attention Is
 * All You Need 해부" (sj-techlog), section "KV cache는 추론의 같은 계산을
 * 반복하지 않게 한다"; "[논문 리뷰]Attention Is All You Need"
 * (kimjiil.github.io), section 3.7): only the newest tokens' queries are
 * computed; the keys and values of every position so far (theirs included)
 * come from the cache. With L = cache_lens[b] valid rows, query t sits at
 * position L - n_q + t and attends to the keys at positions <= its own (the
 * causal rule aligned to the end of the cache); a query at a negative
 * position sees no key and gets 0.
 *   q        [B, h, n_q, d_k] bf16, device        out [B, h, n_q, d_v] bf16
 *   k_cache  [B, h, n_max, d_k] bf16, device      v_cache [B, h, n_max, d_v]
 *   cache_lens: device int32[B] (clamped to [0, n_max]), or NULL for L = n_max
 *   1 <= n_q <= 8 and n_max <= 131072 (more -> ATTN_ERR_UNSUPPORTED);
 *   d_k == d_v in {64, 128}.
 *   workspace: device, 16-byte aligned, >= attn_decode_workspace_bytes(...)
 *   bytes (per-chunk partial results; scratch, caller-owned).
 *   scale: 0 -> 1/sqrt(d_k). Cache rows at or past L are never used.
 * Errors: as attn_forward; a short workspace -> ATTN_ERR_INVALID. Two
 * launches (per-chunk partials, then the merge), asynchronous on `stream`.
 */
size_t attn_decode_workspace_bytes(int B, int h, int n_q, int n_max, int d_v);
attn_status attn_decode(const void *q, const void *k_cache, const void *v_cache, void *out,
                        int B, int h, int n_q, int n_max, int d_k, int d_v,
                        const int32_t *cache_lens, float scale,
                        void *workspace, size_t workspace_bytes, tsd_stream_t stream);

/*
 * attn_forward_window -- restricted self-attention: query i considers only
 * the keys j with i - window_left <= j <= i + window_right ("[논문 리뷰]
 * Attention Is All You Need" (kimjiil.github.io), section "[4] Why
 * Self-Attention", Table 1, row "Self-Attention (restricted)": O(r n d) work
 * for a neighbourhood of r positions instead of O(n^2 d)). Table 1 sizes the
 * neighbourhood by r only; the bounds here are per side, so a neighbourhood
 * of size r centred on the query is window_left = window_right = (r - 1) / 2
 * and a radius-r window is window_left = window_right = r.
 *   Arguments, layouts, masks and errors as attn_forward, plus:
 *   window_left, window_right: >= 0, or -1 for no bound on that side
 *   (-1, -1 is attn_forward); < -1 -> ATTN_ERR_INVALID. A window needs
 *   n_q == n_k (query i and key i share a position), else ATTN_ERR_INVALID.
 *   The causal bit and key padding combine with the window; a row left with
 *   no key gets output 0. Key tiles outside every row's window are never
 *   loaded.
 */
attn_status attn_forward_window(const void *q, const void *k, const void *v, void *out,
                                int B, int h, int n_q, int n_k, int d_k, int d_v,
                                int mask_kind, const int32_t *kv_lens,
                                int window_left, int window_right,
                                float scale, tsd_stream_t stream);

/*
 * attn_forward_strided -- the same operation as attn_forward on tensors whose
 * (batch, head, row) strides are given in ELEMENTS (the head dimension stays
 * contiguous). This lets a caller read heads straight out of a [B, n, h*d]
 * projection output (head i = column block i, section 3.2.2) and write the
 * merged Concat(head_1..head_h) layout [B, n_q, h*d_v] without a copy.
 * Every stride must be a multiple of 8 elements (16 bytes); rows may not
 * overlap within a head. Other arguments and errors as attn_forward.
 */
attn_status attn_forward_strided(const void *q, int64_t q_sb, int64_t q_sh, int64_t q_sr,
                                 const void *k, int64_t k_sb, int64_t k_sh, int64_t k_sr,
                                 const void *v, int64_t v_sb, int64_t v_sh, int64_t v_sr,
                                 void *out, int64_t o_sb, int64_t o_sh, int64_t o_sr,
                                 int B, int h, int n_q, int n_k, int d_k, int d_v,
                                 int mask_kind, const int32_t *kv_lens, float scale,
                                 tsd_stream_t stream);

/*
 * attn_forward_f32 -- the same operation in fp32 throughout (FFMA, no TF32),
 * for callers that need results within 1e-4 of exact.
 *   q [B,h,n_q,d_k], k [B,h,n_k,d_k], v [B,h,n_k,d_v], out [B,h,n_q,d_v]: f32, device.
 *   1 <= d_k, d_v <= 128. Other arguments and errors as attn_forward.
 */
attn_status attn_forward_f32(const float *q, const float *k, const float *v, float *out,
                             int B, int h, int n_q, int n_k, int d_k, int d_v,
                             int mask_kind, const int32_t *kv_lens, float scale,
                             tsd_stream_t stream);

/*
 * mha_workspace_bytes -- size of the caller-owned device workspace that
 * mha_forward needs for the head-split projections Q, K, V and the merged
 * heads Concat(head_1..head_h) (bf16, each region 256-byte aligned).
 * Returns 0 for invalid sizes.
 */
size_t mha_workspace_bytes(int B, int n_q, int n_k, int h, int d_k, int d_v);

/*
 * mha_forward -- multi-head attention, section 3.2.2 (x.W convention, no
 * biases, as in the pages' formula):
 *   Q = x_q W_Q, K = x_kv W_K, V = x_kv W_V        (tensor-core GEMMs)
 *   head_i = Attention(Q_i, K_i, V_i)              (attn kernel; Q_i = column block i)
 *   out = Concat(head_1..head_h) W_O               (tensor-core GEMM)
 * Short sequences run all three in one or two kernels (mha_forward_launches).
 *
 *   x_q  [B, n_q, d_model] bf16      x_kv [B, n_k, d_model] bf16 (may equal x_q)
 *   w_q  [d_model, h*d_k]  bf16      w_k  [d_model, h*d_k]  bf16
 *   w_v  [d_model, h*d_v]  bf16      w_o  [h*d_v, d_model]  bf16
 *   out  [B, n_q, d_model] bf16
 *   d_k == d_v in {64, 128}; d_model a multiple of 8 (16-byte rows), >= 8.
 *   workspace: device, 256-byte aligned, >= mha_workspace_bytes(...) bytes;
 *   on return its last region holds the merged heads; the Q, K, V regions
 *   are scratch (short sequences -- n_q, n_k <= 128, d_k = d_v = 64, h even,
 *   d_model a multiple of 64 -- are projected and attended in one kernel
 *   and never write them; so is cross-attention, x_kv != x_q, with
 *   n_q <= 128 and 128 < n_k <= 192 source rows, the encoder-decoder
 *   attention of section 3.2.3 at the Transformer-base lengths). With
 *   thread-block clusters in flight, the
 *   merged-heads region is how the CTAs of one batch entry share their
 *   heads: calls running concurrently need distinct workspaces.
 *   mask_kind, kv_lens, scale: as attn_forward (the mask applies to every head).
 * Errors: as attn_forward; a short workspace -> ATTN_ERR_INVALID.
 */
attn_status mha_forward(const void *x_q, const void *x_kv,
                        const void *w_q, const void *w_k, const void *w_v, const void *w_o,
                        void *out,
                        int B, int n_q, int n_k, int d_model, int h, int d_k, int d_v,
                        int mask_kind, const int32_t *kv_lens, float scale,
                        void *workspace, size_t workspace_bytes, tsd_stream_t stream);

/*
 * mha_forward_launches -- how many kernels mha_forward launches for these
 * sizes on the current device (a planning query: no launch, no allocation;
 * it may ask the runtime how many thread-block clusters fit):
 *   1  short sequences, W_O applied in the same kernel (n_q, n_k <= 128, or
 *      cross-attention with n_q <= 128 and n_k <= 192; d_k = d_v = 64, h even,
 *      h/2 <= 8, d_model / (h/2) = 64 or 128, and a cluster of h/2 CTAs fits
 *      on the device);
 *   2  short sequences, then the W_O GEMM;
 *   3  the Q/K/V projection GEMM, the attention kernel, the W_O GEMM;
 *   0  nothing to do (B * n_q == 0);  -1  sizes mha_forward rejects.
 * self_attention: nonzero when x_kv will be passed equal to x_q.
 */
int mha_forward_launches(int B, int n_q, int n_k, int d_model, int h, int d_k, int d_v,
                         int self_attention);

/*
 * mha_concat_heads -- Concat(head_1, ..., head_h), head_i =
 * Attention(X_q W_i^Q, X_kv W_i^K, X_kv W_i^V): multi-head attention up to
 * (not including) the output projection W_O ("[논문 리뷰]Attention Is All You
 * Need" (kimjiil.github.io), section 3.2.2). mha_forward is this followed by
 * mha_project_out.
 *   Arguments and errors as mha_forward, with `concat` in place of w_o/out:
 *   concat: device bf16 [B, n_q, h*d_v] (head i = column block i), 16-byte
 *   aligned. The workspace (mha_workspace_bytes(...) bytes, 256-byte aligned)
 *   is scratch for the Q, K, V projections; short sequences (n_q, n_k <= 128,
 *   d_k = d_v = 64, h even, d_model a multiple of 64) run as one fused kernel
 *   and leave it untouched.
 */
attn_status mha_concat_heads(const void *x_q, const void *x_kv,
                             const void *w_q, const void *w_k, const void *w_v, void *concat,
                             int B, int n_q, int n_k, int d_model, int h, int d_k, int d_v,
                             int mask_kind, const int32_t *kv_lens, float scale,
                             void *workspace, size_t workspace_bytes, tsd_stream_t stream);

/*
 * mha_project_qkv -- the input projections of section 3.2.2, all positions at
 * once, in one launch:
 *   q_out = x_q W_Q  [B, n_q, h*d_k],  k_out = x_kv W_K  [B, n_k, h*d_k],
 *   v_out = x_kv W_V [B, n_k, h*d_v]   (bf16, fp32 accumulation)
 * Head i of each result is its column block i, so the outputs feed
 * attn_forward_strided directly. Shapes, alignment and errors as mha_forward
 * (every pointer device, 16-byte aligned; d_model a multiple of 8).
 */
attn_status mha_project_qkv(const void *x_q, const void *x_kv,
                            const void *w_q, const void *w_k, const void *w_v,
                            void *q_out, void *k_out, void *v_out,
                            int B, int n_q, int n_k, int d_model, int h, int d_k, int d_v,
                            tsd_stream_t stream);

/*
 * mha_project_out -- the output projection of section 3.2.2:
 *   out [B, n_q, d_model] = Concat(head_1..head_h) [B, n_q, h*d_v] . W_O [h*d_v, d_model]
 * (bf16, fp32 accumulation). Errors as mha_forward.
 */
attn_status mha_project_out(const void *concat, const void *w_o, void *out,
                            int B, int n_q, int d_model, int h, int d_v, tsd_stream_t stream);

/*
 * mha_forward_noalloc -- mha_forward for callers that cannot allocate device
 * memory. The pages have no counterpart: this is a deployment variant.
 *
 * Who needs it: a plugin whose host application owns the device-memory budget
 * and forbids allocation inside the plugin; a serving loop whose memory is
 * planned up front and must not call cudaMalloc/cudaFree on the request path
 * (they synchronise the device and stall other streams); a plain C caller
 * with no access to its framework's caching allocator. Such callers cannot
 * provide mha_forward's workspace, so this entry point uses a fixed
 * file-scope device array of TSD_MHA_NOALLOC_SCRATCH_BYTES instead and calls
 * no cudaMalloc, cudaFree or other allocating routine. The caller still
 * passes every input and output.
 *
 *   Arguments, layouts and errors as mha_forward, without the workspace.
 *   mha_workspace_bytes(B, n_q, n_k, h, d_k, d_v) must not exceed
 *   TSD_MHA_NOALLOC_SCRATCH_BYTES, else ATTN_ERR_UNSUPPORTED (before any
 *   CUDA call).
 *
 * The array belongs to the library's device image: every GPU that loads the
 * library holds it until the process exits. The first call on a device, with
 * that device current, looks up the array's device address
 * (cudaGetSymbolAddress) and caches it; make that first call before any
 * stream capture. A failed look-up returns ATTN_ERR_CUDA.
 *
 * All calls on a device share the one array, which keeps the last call's
 * contents; calls that overlap on the GPU (other streams or host threads
 * without ordering between them) race on it. No clearing is needed between
 * calls: every byte a call reads from the array is written by that call.
 */
#define TSD_MHA_NOALLOC_SCRATCH_BYTES (32u * 1024u * 1024u)

attn_status mha_forward_noalloc(const void *x_q, const void *x_kv,
                                const void *w_q, const void *w_k, const void *w_v,
                                const void *w_o, void *out,
                                int B, int n_q, int n_k, int d_model, int h, int d_k, int d_v,
                                int mask_kind, const int32_t *kv_lens, float scale,
                                tsd_stream_t stream);

/*
 * Host-buffer entry points -- attn_forward, attn_forward_window, mha_forward,
 * encoder_layer_forward and attn_decode with the step's inputs and result
 * in HOST memory (the pages' operations unchanged; a deployment variant).
 * Each call copies its host inputs into staging regions at the front of
 * `workspace`, runs the device entry point on the staged copies on
 * `stream`, and copies the result back to the host on `stream`. Weights,
 * LayerNorm parameters and the key/value cache stay DEVICE pointers: they
 * are state that lives on the GPU between steps.
 *
 *   *_host arguments: host memory (pinned -- cudaHostAlloc or
 *   cudaHostRegister -- for the copies to be asynchronous; pageable memory
 *   works and is copied synchronously). Sizes, layouts, masks and errors as
 *   the device entry point; kv_lens / cache_lens are host int32[B] here.
 *   workspace: device, 256-byte aligned, >= the matching
 *   *_host_workspace_bytes(...) (0 for invalid sizes); a workspace serves
 *   one stream at a time and only these calls.
 *
 * Ordering. The input copies run on a copy stream the library creates once
 * per device (non-blocking), after the last computation that read the same
 * workspace's staging region; the computation waits for them. The result
 * copy is on `stream`, so once `stream` has passed the call, the result is
 * in host memory and the host inputs may be reused. A caller that passes
 * two workspaces in turn over consecutive calls overlaps call i+1's input
 * copy with call i's computation and result copy. The first call with a
 * workspace (or after the library's table of 64 workspaces evicted it)
 * orders its copy after everything already on `stream`. Calls are
 * serialised by a library-wide lock while they enqueue (microseconds).
 * Errors: every argument error returns before anything is copied; a failed
 * copy or stream operation returns ATTN_ERR_CUDA.
 */
size_t attn_host_workspace_bytes(int B, int h, int n_q, int n_k, int d_k, int d_v);
attn_status attn_forward_host(const void *q_host, const void *k_host, const void *v_host,
                              void *out_host,
                              int B, int h, int n_q, int n_k, int d_k, int d_v,
                              int mask_kind, const int32_t *kv_lens_host, float scale,
                              void *workspace, size_t workspace_bytes, tsd_stream_t stream);

/* attn_forward_window with host q, k, v, out; the workspace as attn_forward_host's. */
attn_status attn_forward_window_host(const void *q_host, const void *k_host, const void *v_host,
                                     void *out_host,
                                     int B, int h, int n_q, int n_k, int d_k, int d_v,
                                     int mask_kind, const int32_t *kv_lens_host,
                                     int window_left, int window_right, float scale,
                                     void *workspace, size_t workspace_bytes,
                                     tsd_stream_t stream);

size_t mha_host_workspace_bytes(int B, int n_q, int n_k, int d_model, int h, int d_k, int d_v);
/* x_kv_host == x_q_host (with n_q == n_k) is self-attention: x is copied once. */
attn_status mha_forward_host(const void *x_q_host, const void *x_kv_host,
                             const void *w_q, const void *w_k, const void *w_v, const void *w_o,
                             void *out_host,
                             int B, int n_q, int n_k, int d_model, int h, int d_k, int d_v,
                             int mask_kind, const int32_t *kv_lens_host, float scale,
                             void *workspace, size_t workspace_bytes, tsd_stream_t stream);

/*
 * mha_forward_host_async -- mha_forward_host whose result copy runs on a
 * device-to-host stream the library creates once per device, after the
 * computation, instead of on `stream`: consecutive calls (two workspaces in
 * turn) then overlap call i's result copy with call i+1's computation, as a
 * serving loop wants. A call's result is in out_host, and its host inputs
 * may be reused, once `stream` has passed a later attn_host_join(stream).
 * A workspace's next computation waits for the result copy that last read
 * it. Arguments and errors as mha_forward_host.
 */
attn_status mha_forward_host_async(const void *x_q_host, const void *x_kv_host,
                                   const void *w_q, const void *w_k, const void *w_v,
                                   const void *w_o, void *out_host,
                                   int B, int n_q, int n_k, int d_model, int h, int d_k, int d_v,
                                   int mask_kind, const int32_t *kv_lens_host, float scale,
                                   void *workspace, size_t workspace_bytes, tsd_stream_t stream);

/* attn_host_join -- `stream` waits for every result copy the asynchronous
 * host-buffer calls issued so far on the current device (none: a no-op). */
attn_status attn_host_join(tsd_stream_t stream);

size_t encoder_layer_host_workspace_bytes(int B, int n, int d_model, int h, int d_k, int d_ff);
attn_status encoder_layer_forward_host(const void *x_host,
                                       const void *w_q, const void *w_k, const void *w_v,
                                       const void *w_o,
                                       const void *ln1_gamma, const void *ln1_beta,
                                       const void *w_1, const void *b_1,
                                       const void *w_2, const void *b_2,
                                       const void *ln2_gamma, const void *ln2_beta,
                                       void *out_host,
                                       int B, int n, int d_model, int h, int d_k, int d_ff,
                                       int mask_kind, const int32_t *kv_lens_host, float scale,
                                       float eps, void *workspace, size_t workspace_bytes,
                                       tsd_stream_t stream);
/* encoder_layer_forward_host_async -- encoder_layer_forward_host whose
 * result copy runs on the library's device-to-host stream, as
 * mha_forward_host_async: out_host is complete, and may be reused, once
 * `stream` has passed a later attn_host_join(stream). Arguments and errors as
 * encoder_layer_forward_host. */
attn_status encoder_layer_forward_host_async(const void *x_host,
                                             const void *w_q, const void *w_k, const void *w_v,
                                             const void *w_o,
                                             const void *ln1_gamma, const void *ln1_beta,
                                             const void *w_1, const void *b_1,
                                             const void *w_2, const void *b_2,
                                             const void *ln2_gamma, const void *ln2_beta,
                                             void *out_host,
                                             int B, int n, int d_model, int h, int d_k, int d_ff,
                                             int mask_kind, const int32_t *kv_lens_host,
                                             float scale, float eps, void *workspace,
                                             size_t workspace_bytes, tsd_stream_t stream);

size_t attn_decode_host_workspace_bytes(int B, int h, int n_q, int n_max, int d_k, int d_v);
/* q_host [B, h, n_q, d_k] and out_host [B, h, n_q, d_v] on the host; the
 * caches are device memory; cache_lens_host: host int32[B] or NULL. */
attn_status attn_decode_host(const void *q_host, const void *k_cache, const void *v_cache,
                             void *out_host,
                             int B, int h, int n_q, int n_max, int d_k, int d_v,
                             const int32_t *cache_lens_host, float scale,
                             void *workspace, size_t workspace_bytes, tsd_stream_t stream);
/* attn_decode_host_async -- attn_decode_host whose result copy runs on the
 * library's device-to-host stream, as mha_forward_host_async: out_host is
 * complete, and may be reused, once `stream` has passed a later
 * attn_host_join(stream). Arguments and errors as attn_decode_host. */
attn_status attn_decode_host_async(const void *q_host, const void *k_cache,
                                   const void *v_cache, void *out_host,
                                   int B, int h, int n_q, int n_max, int d_k, int d_v,
                                   const int32_t *cache_lens_host, float scale,
                                   void *workspace, size_t workspace_bytes, tsd_stream_t stream);

/*
 * Paged key/value caches. The rows of B sequences live in a pool of pages
 * that the caller hands out: row p of sequence b is slot p % page_size of
 * page page_table[b * max_pages + p / page_size]. ("Attention Is All You Need
 * 해부" (sj-techlog), section "KV cache는 추론의 같은 계산을 반복하지 않게
 * 한다", gives the cache itself; pages, grouped heads, the rotation and the
 * 4-bit form are this library's.)
 *
 *   page_table  device int32[B, max_pages]; entries past a sequence's last
 *               row are never read
 *   max_pages   the host sees this and not the lengths: a decoding step over
 *               short sequences is a few microseconds faster under a table
 *               no wider than they need (max_pages * page_size <= 1280 rows above all)
 *   page_size   a power of two, 16..256 (other powers -> ATTN_ERR_UNSUPPORTED);
 *               max_pages * page_size <= 2^30 and n_pages * h_kv * page_size < 2^36 - 16,
 *               else ATTN_ERR_UNSUPPORTED
 *   cache_lens  device int32[B]: rows of each sequence, the new tokens included
 *   new_lens    device int32[B]: how many of the call's n_new (n_q) tokens
 *               sequence b really has, clamped to [0, n_new]; NULL: all.
 *               Token t < new_lens[b] sits at position
 *               cache_lens[b] - new_lens[b] + t; the tokens past them are padding.
 *   h_kv        key/value heads, a divisor of h: query head i reads key head
 *               i / (h / h_kv)
 *   d           64 or 128 (else ATTN_ERR_UNSUPPORTED), of keys and values
 *   B, h        at most 65535, else ATTN_ERR_INVALID
 *
 * A bf16 cache is two pools [n_pages, h_kv, page_size, d] of bf16. A 4-bit
 * cache holds each of keys and values as
 *   codes   uint8 [n_pages, h_kv, page_size, d / 2]: two per byte, the even
 *           column in the low half. A code is a sign bit, two exponent bits
 *           and a mantissa bit (e2m1): 0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives
 *   scales  uint8 [n_pages, h_kv, page_size, d / 16]: an e4m3 number for each
 *           16 columns
 * and a factor f for the whole pool: value = code * scale * f. Values up to
 * 6 * 448 * f can be held; 2^-100 <= f <= 2^100, else ATTN_ERR_INVALID. All
 * pools are device memory, contiguous, 16-byte aligned.
 *
 * A page index outside [0, n_pages) where a row is needed: nothing is read
 * or written through it, that row takes no part, and attn_get_device_status
 * answers ATTN_ERR_DEVICE_INDEX once.
 */
enum {
    ATTN_ROPE_NONE = 0,
    ATTN_ROPE_HALVES = 1, /* columns i and i + rope_dim / 2 are a pair */
    ATTN_ROPE_PAIRS = 2   /* columns 2 i and 2 i + 1 are a pair */
};

/*
 * attn_cache_append -- writes the new tokens' keys and values into their
 * pages, the keys rotated by their positions, and returns the queries rotated
 * in the same way, in the layout that attn_decode_paged reads. Pair i of a
 * query's or key's first rope_dim columns, (x, y), becomes
 *   (x cos - y sin, y cos + x sin)
 * with the cosine and sine of the token's position; columns past rope_dim
 * and values are taken as they are. fp32, rounded once to bf16.
 *
 *   q   bf16, element (b, head, t, col) at b q_sb + head q_sh + t q_sr + col
 *       (strides in elements, multiples of 8, >= 0): a projection's output
 *       [B, n_new, h * d] has (n_new h d, d, h d). NULL (with q_out NULL): no queries
 *   k, v  likewise with kv_sb, kv_sh, kv_sr, h_kv heads
 *   q_out [B, h, n_new, d] bf16; may be q itself where q has that layout
 *   k_out [B, h_kv, n_new, d] bf16: the rotated keys, for attn_forward over
 *       a prompt; NULL: not wanted
 *   rope  device fp32 [rope_rows, rope_dim], 16-byte aligned: row p holds
 *       position p's rope_dim / 2 cosines, then their sines; ignored with
 *       ATTN_ROPE_NONE. rope_dim: even, <= d (else ATTN_ERR_INVALID), and a
 *       multiple of 32 (else ATTN_ERR_UNSUPPORTED)
 * Nothing is written for padding tokens or for tokens at negative positions.
 * A token whose position has no page table entry, no valid page or (when
 * rotated) no row in `rope` is left out whole, as the section above says.
 * Tokens of one call may not share a slot of a page. Errors as attn_forward.
 * One launch.
 */
attn_status attn_cache_append(const void *q, int64_t q_sb, int64_t q_sh, int64_t q_sr,
                              const void *k, const void *v,
                              int64_t kv_sb, int64_t kv_sh, int64_t kv_sr,
                              void *q_out, void *k_out, void *k_cache, void *v_cache,
                              const int32_t *page_table, const int32_t *cache_lens,
                              const int32_t *new_lens,
                              const float *rope, int rope_rows, int rope_dim, int rope_kind,
                              int B, int h, int h_kv, int n_new, int d,
                              int n_pages, int page_size, int max_pages, tsd_stream_t stream);

/*
 * attn_cache_append_q4 -- attn_cache_append into a 4-bit cache. For each 16
 * columns of a key (after the rotation, in fp32) or value x:
 *   scale = max|x| / (6 f) rounded to e4m3, at most 448;
 *   code  = x / (scale f) rounded to e2m1, at most 6 in magnitude
 * both to nearest, ties to even. Columns holding an infinity or a NaN make
 * their scale a NaN; a scale that rounds to 0 makes its codes 0. q_out and
 * k_out are bf16 as above.
 */
attn_status attn_cache_append_q4(const void *q, int64_t q_sb, int64_t q_sh, int64_t q_sr,
                                 const void *k, const void *v,
                                 int64_t kv_sb, int64_t kv_sh, int64_t kv_sr,
                                 void *q_out, void *k_out,
                                 void *k_codes, void *k_scales, void *v_codes, void *v_scales,
                                 float k_factor, float v_factor,
                                 const int32_t *page_table, const int32_t *cache_lens,
                                 const int32_t *new_lens,
                                 const float *rope, int rope_rows, int rope_dim, int rope_kind,
                                 int B, int h, int h_kv, int n_new, int d,
                                 int n_pages, int page_size, int max_pages, tsd_stream_t stream);

/*
 * attn_decode_paged -- attn_decode over a paged cache with grouped heads.
 *   q, out  [B, h, n_q, d] bf16; 1 <= n_q <= 8 (more -> ATTN_ERR_UNSUPPORTED);
 *       B h n_q < 2^31, else ATTN_ERR_INVALID
 *   cache_lens  as above, clamped to [0, max_pages * page_size]; NULL: that many
 *   mask_kind   ATTN_MASK_CAUSAL: query t sees the rows at positions <=
 *       cache_lens[b] - new_lens[b] + t, its own (the new tokens' keys are in
 *       the cache already). ATTN_MASK_NONE: every query sees all cache_lens[b]
 *       rows (cross-attention to encoder states kept in a cache). Others ->
 *       ATTN_ERR_INVALID
 *   scale       0 -> 1/sqrt(d); scale log2(e), with a 4-bit cache's k_factor, has
 *       to be finite in fp32, else ATTN_ERR_INVALID
 *   workspace   device, 16-byte aligned, >= attn_decode_paged_workspace_bytes(...)
 *       bytes of scratch (0 for sizes that the call refuses)
 * Rows of `out` that see no row, padding tokens' among them, are 0. Rows at
 * or past cache_lens[b] are never used, whatever they hold. An infinity in a
 * value that a query sees is one in its output (a NaN if the row's weight is
 * below fp32's range, or both infinities meet). The weighted values are added
 * up in fp32 before the division by the weights' sum, the largest weight being
 * 1 at most: a bf16 cache's |v| of one column have to add up to fp32's range.
 * Errors as attn_decode.
 */
size_t attn_decode_paged_workspace_bytes(int B, int h, int h_kv, int n_q, int d, int page_size,
                                         int max_pages);
attn_status attn_decode_paged(const void *q, const void *k_cache, const void *v_cache, void *out,
                              const int32_t *page_table, const int32_t *cache_lens,
                              const int32_t *new_lens,
                              int B, int h, int h_kv, int n_q, int d,
                              int n_pages, int page_size, int max_pages,
                              int mask_kind, float scale,
                              void *workspace, size_t workspace_bytes, tsd_stream_t stream);

/* attn_decode_paged_q4 -- attn_decode_paged over a 4-bit cache. */
attn_status attn_decode_paged_q4(const void *q, const void *k_codes, const void *k_scales,
                                 const void *v_codes, const void *v_scales,
                                 float k_factor, float v_factor, void *out,
                                 const int32_t *page_table, const int32_t *cache_lens,
                                 const int32_t *new_lens,
                                 int B, int h, int h_kv, int n_q, int d,
                                 int n_pages, int page_size, int max_pages,
                                 int mask_kind, float scale,
                                 void *workspace, size_t workspace_bytes, tsd_stream_t stream);

/*
 * Keeping a paged cache's pages. The calls below keep the page table that
 * attn_cache_append and attn_decode_paged read, between them: they give rows
 * of the table pages, share pages between rows, take them back and move them.
 * ("Attention Is All You Need 해부" (sj-techlog), section "KV cache는 추론의
 * 같은 계산을 반복하지 않게 한다", gives the cache; its pages are this library's.)
 * The state is two device arrays that the caller sets up and owns:
 *
 *   page_table  int32[B, max_pages]; -1 (any negative entry) holds no page
 *   ref_counts  int32[n_pages]: how many entries, of this and any other table
 *               over the same pool, name the page; 0: the page is free
 *
 * An empty table is all -1, an empty pool all 0. Row r of the table is a
 * sequence. Where a call takes new pages, it takes the free pages of the
 * lowest numbers, in the order of the rows and of each row's pages; what a
 * call does follows from its arguments alone, and nothing is kept between
 * calls. Counts that are not what the table says give wrong tables, never an
 * access out of range. An entry or a number that is out of range is left out and
 * attn_get_device_status answers ATTN_ERR_DEVICE_INDEX once. Calls that change
 * the same ref_counts have to be ordered by their stream.
 *   page_size, max_pages: as above; n_pages <= 2^30, else ATTN_ERR_UNSUPPORTED
 *   B           at most 65535, else ATTN_ERR_INVALID. B = 0 launches nothing and
 *               writes nothing (but for attn_cache_compact)
 *   every array: device memory, 4-byte aligned; a null or misaligned pointer
 *   or a bad size -> ATTN_ERR_INVALID
 *
 * A step of beam search over a paged cache is
 *   attn_cache_fork(table, lens, counts, parents, ...)  the rows beam_select chose
 *   attn_cache_reserve(...)     places for the new tokens; cache_lens with them
 *   attn_cache_copy(...)        the pages that reserve listed, all layers
 *   and then attn_cache_append and attn_decode_paged in every layer.
 */

/*
 * attn_cache_fork -- row r of the table becomes row parents[r], all rows at
 * once: rows that continue the same row share its pages, and pages that no row
 * names any more are free.
 *   parents     int32[B]: a row's number, its own to stay as it is, or -1: the
 *               row is empty afterwards
 *   cache_lens  int32[B], in place: lens[r] becomes lens[parents[r]] (0 for -1).
 *               NULL: not wanted
 *   B <= 32768, else ATTN_ERR_UNSUPPORTED
 * A parent out of range leaves its row as it is. One launch.
 */
attn_status attn_cache_fork(int32_t *page_table, int32_t *cache_lens, int32_t *ref_counts,
                            const int32_t *parents, int B, int n_pages, int max_pages,
                            tsd_stream_t stream);

/*
 * attn_cache_release -- row b keeps the pages of its first keep_lens[b] rows
 * of the cache and gives the others back: 0 frees a sequence, a smaller length
 * takes back speculated tokens, a negative number leaves the row as it is.
 *   keep_lens   int32[B], or NULL: all rows are freed
 * One launch.
 */
attn_status attn_cache_release(int32_t *page_table, int32_t *ref_counts, const int32_t *keep_lens,
                               int B, int n_pages, int page_size, int max_pages,
                               tsd_stream_t stream);

/*
 * attn_cache_reserve -- before attn_cache_append with the same cache_lens,
 * new_lens and n_new: every page that the new tokens are written into exists
 * and belongs to its row alone. The positions are cache_lens[b] - new_lens[b]
 * .. cache_lens[b] - 1; of the pages that hold them,
 *   a missing one is taken from the free pages;
 *   one that other entries name too, of this row or another, is left, and a
 *   free page taken in its place. Where all that name it are entries that this
 *   call's tokens are written into, the first of them (by row, then by place)
 *   keeps it. If the page holds earlier rows of the sequence (its first page
 *   can), a copy of them is listed.
 *   copies      int32[B, 3], written: (from page, to page, rows), in the order
 *               of the sequences; entries past n_copies[0] are left as they were.
 *               attn_cache_copy carries them out: no page is both from and to
 *   n_copies    int32[1], written
 *   n_missing   int32[1], written: 0, or how many pages are wanting. Then
 *               nothing is changed and nothing listed (but that an entry which
 *               names no page may be -1 afterwards)
 *   workspace   device, 16-byte aligned, >= attn_cache_pages_workspace_bytes(B,
 *               n_pages) bytes of scratch (0 for sizes that the calls refuse)
 * Positions past max_pages * page_size get no page. B times the pages that
 * n_new tokens of a row can lie in (max_pages at most) is at most 2^31, else
 * ATTN_ERR_UNSUPPORTED. One launch.
 */
size_t attn_cache_pages_workspace_bytes(int B, int n_pages);
attn_status attn_cache_reserve(int32_t *page_table, int32_t *ref_counts, const int32_t *cache_lens,
                               const int32_t *new_lens, int32_t *copies, int32_t *n_copies,
                               int32_t *n_missing, int B, int n_new, int n_pages, int page_size,
                               int max_pages, void *workspace, size_t workspace_bytes,
                               tsd_stream_t stream);

/*
 * attn_cache_compact -- moves the used pages to the front of the pool, so that
 * its end can be given up or used otherwise. With U used pages, the k-th
 * highest page from U on moves to the k-th lowest free page.
 *   table_out   int32[B, max_pages], counts_out int32[n_pages]: the table and
 *               the counts after the moves; may be page_table and ref_counts
 *               themselves, and do not overlap them otherwise. B may be 0
 *   copies      int32[max_copies, 3], written: (from, to, page_size) for
 *               attn_cache_copy, which has to follow before the cache is read;
 *               entries past n_copies[0] are left as they were
 *   max_copies  at most so many pages move; >= min(U, n_pages - U) moves all
 *   n_copies, n_used  int32[1], written: the moves, and U
 *   workspace   as attn_cache_reserve
 * All entries of tables that name pages of the pool have to be in page_table.
 * Two launches, or one where the table is small.
 */
attn_status attn_cache_compact(const int32_t *page_table, const int32_t *ref_counts,
                               int32_t *table_out, int32_t *counts_out, int32_t *copies,
                               int32_t *n_copies, int32_t *n_used, int B, int n_pages,
                               int page_size, int max_pages, int max_copies, void *workspace,
                               size_t workspace_bytes, tsd_stream_t stream);

/*
 * attn_cache_copy -- copies the first `rows` rows of page `from` to page `to`,
 * of every head, of keys and values, in all layers, for every (from, to, rows)
 * of a list.
 *   k_cache, v_cache  the first layer's pools [n_pages, h_kv, page_size, d]
 *               bf16; layer i's begin layer_rows * i rows of d columns further on
 *   copies      int32[max_copies, 3]; n_copies int32[1], how many of them there
 *               are (clamped to [0, max_copies]; above it is out of range), or
 *               NULL: all
 *   n_layers    0 .. 65535; layer_rows a multiple of 16, >= n_pages * h_kv *
 *               page_size, and times n_layers at most 2^50 (ignored for one
 *               layer), else ATTN_ERR_INVALID
 *   h_kv        1 .. 65535, else ATTN_ERR_INVALID; h_kv * page_size * d <= 2^29,
 *               else ATTN_ERR_UNSUPPORTED
 * No page may be `to` of two copies, or `from` of one and `to` of another. A
 * copy with a number out of range is left out. One launch.
 */
attn_status attn_cache_copy(void *k_cache, void *v_cache, const int32_t *copies,
                            const int32_t *n_copies, int max_copies, int n_layers,
                            int64_t layer_rows, int h_kv, int d, int n_pages, int page_size,
                            tsd_stream_t stream);

/* attn_cache_copy_q4 -- attn_cache_copy of a 4-bit cache's codes and scales. */
attn_status attn_cache_copy_q4(void *k_codes, void *k_scales, void *v_codes, void *v_scales,
                               const int32_t *copies, const int32_t *n_copies, int max_copies,
                               int n_layers, int64_t layer_rows, int h_kv, int d, int n_pages,
                               int page_size, tsd_stream_t stream);

/*
 * beam_select -- one step of beam search ("[논문 리뷰]Attention Is All You
 * Need" (kimjiil.github.io) and "Attention Is All You Need 해부" (sj-techlog)
 * decode with beams of 4 and a length penalty alpha = 0.6; how a step handles
 * ended hypotheses is this library's choice). Row b * beams + k of the logits is
 * what beam k of sentence b says of its next token. With s the beams' scores
 * (their tokens' summed log probabilities),
 *   total(k, v) = s_k + x_kv - log sum_u exp x_ku,
 * the 2 * beams best pairs of a sentence (`beams` without an end token; fewer
 * where fewer are above -infinity), by total and then by lowest k * vocab + v,
 * are its candidates.
 *   The first `beams` candidates that are not the end token are the next beams.
 *   Those that are the end token end there, with score total / ((5 + n) /
 *   6)^alpha at n = lengths[b] tokens; the best `beams` of them and of the
 *   hypotheses that ended before are kept, best first, earlier ones first among equals.
 *
 *   logits      bf16, 2-byte aligned; element (row, v) at row * row_stride + v,
 *               row_stride >= vocab (16-byte aligned rows are faster)
 *   scores      fp32[B, beams]; -infinity: no hypothesis (whatever its logits
 *               are). At a sentence's start: 0, and -infinity for the others
 *   lengths     int32[B]: tokens of the hypotheses, the one chosen now among
 *               them (less than 1 counts as 1)
 *   alpha       within fp32's range, else ATTN_ERR_INVALID (a double: 0.6 is no
 *               number of 32 bits)
 *   end         the end token (one from vocab on is never chosen), or -1: none;
 *               then lengths, alpha and the ended_* arrays are ignored
 *   tokens, parents  int32[B, beams], written: the token, and the row b * beams
 *               + k that it continues (as attn_cache_fork takes it)
 *   new_scores  fp32[B, beams], written: totals; may be `scores` itself.
 *               A beam without a candidate: -infinity, the end token (0 without
 *               one) and its own row
 *   ended_scores, ended_rows, ended_lengths  fp32, int32, int32 [B, beams], in
 *               place: score, the row that the end token continued, and n. The
 *               caller starts with scores of -infinity; a place without a
 *               hypothesis has that and keeps the other two as they were
 *   1 <= beams <= 16, vocab <= 2^20, and B * beams * ceil(vocab / 1024) <= 2^31 -
 *               2^20, else ATTN_ERR_UNSUPPORTED
 *   workspace   device, 16-byte aligned, >= beam_select_workspace_bytes(...)
 *               bytes of scratch (0 for sizes that the call refuses)
 * Logits of -infinity are tokens that are never chosen. A beam whose logits or
 * score hold a NaN or +infinity has no candidates, and attn_get_device_status
 * answers ATTN_ERR_DEVICE_VALUE once. Totals are formed and compared in 48 bits
 * from exponentials and partial sums in 32. beams = 1 is greedy decoding.
 * Errors as attn_forward. Two launches, or one where beams * ceil(vocab / 1024)
 * is small (16 for hundreds of sentences, 64 for a hundred, 128 for eight).
 */
size_t beam_select_workspace_bytes(int B, int beams, int vocab);
attn_status beam_select(const void *logits, int64_t row_stride, const float *scores,
                        const int32_t *lengths, int B, int beams, int vocab, int end, double alpha,
                        int32_t *tokens, int32_t *parents, float *new_scores, float *ended_scores,
                        int32_t *ended_rows, int32_t *ended_lengths, void *workspace,
                        size_t workspace_bytes, tsd_stream_t stream);

/* beam_select_f32 -- beam_select of fp32 logits (4-byte aligned). */
attn_status beam_select_f32(const float *logits, int64_t row_stride, const float *scores,
                            const int32_t *lengths, int B, int beams, int vocab, int end,
                            double alpha, int32_t *tokens, int32_t *parents, float *new_scores,
                            float *ended_scores, int32_t *ended_rows, int32_t *ended_lengths,
                            void *workspace, size_t workspace_bytes, tsd_stream_t stream);

/*
 * attn_get_device_status -- synchronises `stream`, then reads and clears the
 * device error words the kernels set when a bounded wait runs out, a page
 * index or position is out of range, or a beam's logits are no numbers. Returns
 * ATTN_OK, ATTN_ERR_DEVICE_TIMEOUT, ATTN_ERR_DEVICE_INDEX, ATTN_ERR_DEVICE_VALUE
 * (the first of them that happened, in this order), or ATTN_ERR_CUDA if the
 * synchronisation itself failed.
 */
attn_status attn_get_device_status(tsd_stream_t stream);

/* The last CUDA error code (cudaError_t as int) seen by this library on the
 * calling thread, 0 if none. */
int attn_last_cuda_error(void);

/* A static, human-readable name for a status code. */
const char *attn_status_string(attn_status s);

/*
 * attn_selftest_wait_timeout -- failure-detection self test. Launches one
 * small kernel whose bounded wait is on an mbarrier that nothing ever
 * arrives on, with a limit of `limit_us` microseconds (1..2000000). The
 * kernel records a timeout in the device error word and exits; the caller
 * reads it with attn_get_device_status(), and the context stays usable.
 * No tensor memory or asynchronous copy is involved.
 */
attn_status attn_selftest_wait_timeout(int limit_us, tsd_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* TSD_ATTENTION_H */
