/*
 * nystrom.h - C ABI of the Nyström self-attention forward library
 * (libnystrom.so, CUDA, sm_103a).
 *
 * What it computes, per head (b, h) of q, k, v in [B, H, n, d]:
 *
 *   Q~, K~ = segment means of Q and K over m contiguous segments; segment
 *            i is rows [floor(i n/m), floor((i+1) n/m)), i.e. n/m rows each
 *            when m divides n, else floor(n/m) or ceil(n/m) rows
 *            ("Nyströmformer" review page, Proposed method, bullet 4)
 *   A_S    = softmax(Q~ K~^T / sqrt(d))                       (bullet 2)
 *   Z      = iterative Moore-Penrose inverse of A_S, `iters` updates of
 *            Z <- 1/4 Z (13I - A_S Z (15I - A_S Z (7I - A_S Z)))
 *            from Z_0 = A_S^T / (||A_S||_1 ||A_S||_inf)       (bullet 5)
 *   out    = softmax(Q K~^T / sqrt(d)) Z softmax(Q~ K^T / sqrt(d)) V
 *            + DWConv(V)                                      (bullets 3, 6)
 *
 * DWConv is a depthwise convolution along the sequence: one odd-width filter
 * of conv_ks taps per head, shared by the d channels, cross-correlation with
 * (conv_ks-1)/2 zero rows of padding on each side, no bias:
 *   conv[t] = sum_{j<conv_ks} conv_w[h][j] * V[t + j - (conv_ks-1)/2].
 * conv_ks = 0 drops the term (the output is then the attention alone).
 *
 * Conventions shared by every entry point below:
 *  - Device pointers unless a name says "host". The caller owns every
 *    buffer; the library never frees or keeps a caller pointer.
 *  - q, k, v, out: [B][H][n][d] contiguous, d innermost, element type
 *    `dtype` (NYS_FP32: float; NYS_BF16: bfloat16 bit patterns). Each base
 *    address 16-byte aligned. out is fully overwritten; it may not alias
 *    q, k or v.
 *  - conv_w: [H][conv_ks] float32 (for both dtypes); may be NULL when
 *    conv_ks == 0.
 *  - Shape rules (else NYS_ERR_SHAPE, nothing launched): B, H, n, d, m >= 1;
 *    m <= n; m <= 256; d % 8 == 0 and d <= 128; for NYS_BF16 also
 *    d in {32, 64, 128}; 0 <= iters <= 64; conv_ks == 0 or odd and <= 127;
 *    B*H*n*d < 2^40.
 *  - Scale: every softmax uses 1/sqrt(d).
 *  - Asynchrony: compute entry points enqueue work on `stream` (0 = the
 *    legacy default stream) and return without waiting. A negative return
 *    means nothing was enqueued (argument errors) or that a launch failed
 *    (NYS_ERR_CUDA; see nystrom_last_error_string). Device-side failures
 *    (a bounded wait that ran out) are reported by nystrom_get_status after
 *    the stream has finished.
 *  - Thread safety: calls may come from several host threads; the cached
 *    workspace of nystrom_attn_fwd is shared per device, so concurrent calls
 *    on different streams of one device must use nystrom_attn_fwd_ws with
 *    their own workspaces. nystrom_qk_norm_rope_bwd, nystrom_kv4_attn_fwd,
 *    nystrom_q8_matmul, nystrom_add_rms_norm_bwd, nystrom_gated_ff_fwd and
 *    nystrom_gated_ff_bwd share another one where none is given. Those calls may
 *    come from any threads and streams: one whose stream is not the last one's
 *    waits there, on the device, for the last one's kernels. Calls that shall
 *    run side by side are given workspaces.
 */
#ifndef NYSTROM_H_
#define NYSTROM_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same type as the CUDA runtime's cudaStream_t. */
typedef struct CUstream_st* nys_stream_t;

typedef enum { NYS_FP32 = 0, NYS_BF16 = 1 } nys_dtype_t;

typedef enum {
  NYS_OK = 0,
  NYS_ERR_ARG = -1,         /* NULL pointer, bad dtype, negative size      */
  NYS_ERR_SHAPE = -2,       /* shape outside the rules above               */
  NYS_ERR_ALIGN = -3,       /* a pointer is not 16-byte aligned            */
  NYS_ERR_UNSUPPORTED = -4, /* no GPU of compute capability 10.3 current   */
  NYS_ERR_NOMEM = -5,       /* workspace allocation failed / too small     */
  NYS_ERR_CUDA = -6,        /* a CUDA runtime call or launch failed        */
  NYS_ERR_TIMEOUT = -7,     /* a device-side bounded wait ran out          */
  NYS_ERR_INDEX = -8        /* a device-side index (page, position, length)
                               lay outside its range and was skipped       */
} nys_status_t;

/*
 * nystrom_attn_fwd - the forward pass (see the top of this file).
 * Uses a workspace the library allocates and caches per device (grown with
 * cudaMalloc when a call needs more; growing synchronises the device).
 * iters: number of pseudo-inverse updates ("about 6", Proposed method,
 * bullet 5); run exactly, no early exit. For NYS_BF16 inputs up to 8 updates
 * run on the tensor cores (tf32 products, fp32 storage); with more, the
 * pseudo-inverse runs in fp32 on the CUDA cores, since the iteration
 * amplifies tf32 rounding by the condition number of A_S as it inverts more
 * of its small singular values (slower, same result bar).
 * Returns NYS_OK or a negative nys_status_t.
 */
int nystrom_attn_fwd(const void* q, const void* k, const void* v,
                     const float* conv_w, void* out, int B, int H, int n,
                     int d, int m, int iters, int conv_ks, int dtype,
                     nys_stream_t stream);

/*
 * nystrom_attn_workspace_bytes - bytes of device workspace that
 * nystrom_attn_fwd_ws needs for this shape (0 if the shape is invalid).
 * Host arithmetic only; launches nothing. The size depends on the SM count
 * of the current device (the plan spreads work over its SMs; 152, a GB300,
 * when no device can be queried), so ask with the device current that will
 * run the call.
 */
size_t nystrom_attn_workspace_bytes(int B, int H, int n, int d, int m,
                                    int dtype);

/*
 * nystrom_attn_fwd_ws - as nystrom_attn_fwd, with a caller-owned device
 * workspace of ws_bytes >= nystrom_attn_workspace_bytes(...) bytes,
 * 256-byte aligned. The library allocates nothing. The workspace must stay
 * valid and unused by others until the stream has finished the call.
 * Returns NYS_ERR_NOMEM if ws_bytes is too small.
 */
int nystrom_attn_fwd_ws(const void* q, const void* k, const void* v,
                        const float* conv_w, void* out, int B, int H, int n,
                        int d, int m, int iters, int conv_ks, int dtype,
                        void* workspace, size_t ws_bytes, nys_stream_t stream);

/*
 * nystrom_attn_fwd_noalloc - as nystrom_attn_fwd, but allocates nothing:
 * no cudaMalloc, cudaFree or allocating library call. The paper has no
 * counterpart; this entry point exists for callers that cannot allocate
 * device memory at call time, such as plugins inside a host application that
 * owns all device memory through its own allocator, or latency-critical
 * loops where a cudaMalloc/cudaFree would synchronise the device.
 * Its scratch is a fixed 32 MiB device array inside the library, reserved on
 * every GPU that loads the library until the process exits. Shapes whose
 * workspace (nystrom_attn_workspace_bytes) exceeds 32 MiB are rejected with
 * NYS_ERR_NOMEM before anything is enqueued.
 * The first call on a device looks up the array's device address (once per
 * device, with that device current); make that first call before any stream
 * capture. The first call on a device of a shape whose plan runs on more
 * than one stream (see nystrom_plan_describe) also creates the library's
 * auxiliary streams and events for that device, as every entry point does;
 * they hold no device memory of the caller's and live until exit. All calls
 * share the one array and it keeps the previous call's
 * contents; the library clears what must start at zero on every call. Calls
 * that overlap on the GPU (different streams, or different host threads,
 * same device) race on the array: serialise them.
 */
int nystrom_attn_fwd_noalloc(const void* q, const void* k, const void* v,
                             const float* conv_w, void* out, int B, int H,
                             int n, int d, int m, int iters, int conv_ks,
                             int dtype, nys_stream_t stream);

/*
 * nystrom_attn_fwd_ex - the forward pass with the two variants the page
 * leaves open (Proposed method, bullets 4 and 6), as readings of it:
 *  - conv_layout NYS_CONV_PER_HEAD: conv_w is [H][conv_ks], one filter per
 *    head shared by its d channels (as nystrom_attn_fwd);
 *    NYS_CONV_PER_CHANNEL: conv_w is [H][d][conv_ks] float32, channel c of
 *    head h has its own taps conv_w[h][c][.] ("depthwise": one filter per
 *    channel).
 *  - lengths_host: HOST int32 [B], or NULL. Batch entry b holds
 *    lengths_host[b] real tokens in rows [0, lengths_host[b]) of its n rows,
 *    the rest is padding, which takes part in nothing: the landmarks are the
 *    segment means of the real tokens (segments over lengths_host[b] rows),
 *    padded keys are masked out of softmax(Q~ K^T / sqrt(d)), padded rows of
 *    V read as zero in the convolution, and the output rows of padding are
 *    zero. The real rows' result equals that of the unpadded sequence. Each
 *    length must satisfy m <= lengths_host[b] <= n (else NYS_ERR_SHAPE).
 *    Padded rows of q, k, v must hold finite values (they are read, then
 *    masked). The array is copied to the device inside the call.
 * workspace: caller-owned device workspace of ws_bytes >=
 * nystrom_attn_workspace_bytes(...) bytes, 256-byte aligned, as for
 * nystrom_attn_fwd_ws; or NULL to use the library's cached workspace (as
 * nystrom_attn_fwd does).
 * With NYS_CONV_PER_HEAD and no lengths the result is that of
 * nystrom_attn_fwd. The variants run the token pass for the attention term
 * alone and add the convolution (and zero the padding rows) in a pass of
 * their own, on the CUDA cores.
 * Returns NYS_OK or a negative nys_status_t (NYS_ERR_ARG for an unknown
 * conv_layout).
 */
typedef enum { NYS_CONV_PER_HEAD = 0, NYS_CONV_PER_CHANNEL = 1 } nys_conv_layout_t;
int nystrom_attn_fwd_ex(const void* q, const void* k, const void* v,
                        const float* conv_w, void* out, int B, int H, int n,
                        int d, int m, int iters, int conv_ks, int dtype,
                        int conv_layout, const int* lengths_host,
                        void* workspace, size_t ws_bytes, nys_stream_t stream);

/*
 * nystrom_mha_fwd - the multi-head attention module around the op (the
 * page's model uses Nyström self-attention in place of softmax attention,
 * abstract and Proposed method bullet 6): with D = H*d,
 *   [Q | K | V] = x w_qkv + b_qkv,  Q, K, V split into H heads of d columns
 *   (head h = columns [h*d, (h+1)*d) of each), O_h = the forward pass of the
 *   top of this file on head h (m landmarks, iters updates, conv_w [H][conv_ks]),
 *   y = [O_1 | ... | O_H] w_o + b_o.
 * x, y: [B][n][D], w_qkv: [D][3D] (columns: the Q block, then K, then V),
 * w_o: [D][D], all row-major in `dtype` (device); b_qkv [3D] and b_o [D]
 * float32 device arrays, or NULL for no bias. Pointers 16-byte aligned.
 * The projections run in cuBLAS (fp32 accumulation into the workspace); the
 * head split and merge, the biases and the attention in this library's
 * kernels. No residual connection, normalisation or dropout: those belong to
 * the layer around the module.
 * workspace: device, 256-byte aligned, ws_bytes >= nystrom_mha_workspace_bytes,
 * or NULL to use a buffer the library allocates and caches per device.
 * Returns NYS_OK or a negative nys_status_t (shape rules as the top of this
 * file, with n, H, d, m of the attention).
 */
size_t nystrom_mha_workspace_bytes(int B, int n, int H, int d, int m, int dtype);
int nystrom_mha_fwd(const void* x, const void* w_qkv, const float* b_qkv,
                    const void* w_o, const float* b_o, const float* conv_w,
                    void* y, int B, int n, int H, int d, int m, int iters,
                    int conv_ks, int dtype, void* workspace, size_t ws_bytes,
                    nys_stream_t stream);

/*
 * Clustered attention, centroid path ("Fast Transformers with Clustered
 * Attention" review page, Proposed method, bullets 1, 2 and 4): per head
 * (b, h) the queries Q [n, d] are grouped into C clusters by K-means and
 * attention is computed once per centroid:
 *   mu      = segment means of Q over C contiguous segments (as Q~ above)
 *   iters x:  a(i) = argmin_c |q_i - mu_c|^2 (ties: the lowest c), then
 *             mu_c = mean of the queries with a(i) = c (none: unchanged)
 *   out[i]  = softmax(mu_{a(i)} K^T / sqrt(d)) V
 * K-means: for NYS_BF16 with d in {64, 128} and C <= 128 on the tensor
 * cores (distances to fp32 accuracy: the centroids split into three bf16
 * terms; the members' sums as a one-hot product with fp32 accumulation,
 * added across CTAs in a fixed order: deterministic), otherwise in fp32 on
 * the CUDA cores (the update sums a cluster's queries in index order). The
 * centroid rows run in the landmark-row kernels of the forward pass (bf16
 * tensor cores for NYS_BF16, with the centroids rounded to bf16; fp32 CUDA
 * cores for NYS_FP32).
 * q, k, v, out: [B][H][n][d] in `dtype`, device, 16-byte aligned; shape rules
 * as the top of this file with C in place of m; 1 <= iters <= 64.
 * workspace: device, 256-byte aligned, ws_bytes >=
 * nystrom_clustered_workspace_bytes(...), or NULL for the library's cached
 * workspace. Asynchronous on `stream`; nystrom_get_status reports bounded
 * waits that ran out.
 * nystrom_clustered_stage_offset: byte offset in the workspace, after a
 * call with these sizes has finished, of NYS_CSTAGE_ASSIGN (int32
 * [B*H][n], the last assignment), NYS_CSTAGE_CENTROIDS_PREV (float32
 * [B*H][C][d], the centroids that assignment used), NYS_CSTAGE_CENTROIDS
 * (float32 [B*H][C][d], after the last update), NYS_CSTAGE_G (float32
 * [B*H][C][d], the centroid rows); -1 for invalid sizes or stage.
 */
typedef enum {
  NYS_CSTAGE_ASSIGN = 0,
  NYS_CSTAGE_CENTROIDS_PREV = 1,
  NYS_CSTAGE_CENTROIDS = 2,
  NYS_CSTAGE_G = 3
} nys_cstage_t;
size_t nystrom_clustered_workspace_bytes(int B, int H, int n, int d, int C,
                                         int dtype);
long long nystrom_clustered_stage_offset(int B, int H, int n, int d, int C,
                                         int iters, int dtype, int stage);
int nystrom_clustered_attn_fwd(const void* q, const void* k, const void* v,
                               void* out, int B, int H, int n, int d, int C,
                               int iters, int dtype, void* workspace,
                               size_t ws_bytes, nys_stream_t stream);

/*
 * nystrom_attn_fwd_host - the whole forward pass from and to HOST memory:
 * copies q, k, v, conv_w to the device, runs the forward pass on `stream`,
 * copies out back and waits for the stream. The batch is processed in up
 * to four chunks of whole batch entries, pipelined: a chunk's inputs are
 * copied up (on a library stream) while the previous chunk is computed on
 * `stream` and the one before it is copied back (on another library
 * stream). Host buffers should be pinned (page-locked) for full copy speed;
 * pageable memory works but is slower. Device staging buffers are
 * allocated and cached per device (grown with cudaMalloc when needed); one
 * host-entry call per device runs at a time. Synchronous: out_host is
 * complete on return; nystrom_get_status then reports the status of all
 * chunks.
 */
int nystrom_attn_fwd_host(const void* q_host, const void* k_host,
                          const void* v_host, const float* conv_w_host,
                          void* out_host, int B, int H, int n, int d, int m,
                          int iters, int conv_ks, int dtype,
                          nys_stream_t stream);

/*
 * Stage export, for testing the intermediate results against a reference.
 * After a nystrom_attn_fwd_ws call has finished, the workspace holds, as
 * float32 arrays per head (b*H + h major):
 *   NYS_STAGE_Q_TILDE [m][d], NYS_STAGE_K_TILDE [m][d], NYS_STAGE_G [m][d]
 *   (= softmax(Q~ K^T/sqrt d) V), NYS_STAGE_A_S [m][m], NYS_STAGE_W [m][d]
 *   (= Z G), NYS_STAGE_Z [m][m] (Z after `iters` updates).
 * nystrom_attn_stage_offset returns the byte offset of `stage` in the
 * workspace for this shape, or -1 for an invalid shape or stage.
 */
typedef enum {
  NYS_STAGE_Q_TILDE = 0,
  NYS_STAGE_K_TILDE = 1,
  NYS_STAGE_G = 2,
  NYS_STAGE_A_S = 3,
  NYS_STAGE_W = 4,
  NYS_STAGE_Z = 5
} nys_stage_t;
long long nystrom_attn_stage_offset(int B, int H, int n, int d, int m,
                                    int dtype, int stage);

/*
 * nystrom_plan_describe - the kernels a forward call of this shape
 * launches, in order, as one line of text: the plan ("serial": each step
 * after the previous one; "z-beside-rows": the pseudo-inverse's chain of
 * products on a second stream beside the landmark-row pass, then the merge
 * of G and W = Z G; "head-groups": the batch split into groups of whole
 * batch entries, each group's steps on its own stream), the number of head
 * groups, and per step the kernel with its host-side sizes (the landmark-row
 * pass's CTAs, key ranges per head and 128-key tiles per CTA; the
 * pseudo-inverse's CTAs and, beside the rows, the SMs they take). The plan is
 * a function of the shape and of the current device's SM count (152, a
 * GB300, when no device can be queried).
 * Host only: launches nothing.
 * buf: host memory of `len` bytes (may be NULL when len == 0); receives at
 * most len - 1 characters and a terminating NUL.
 * Returns the length of the full description (without the NUL), or a
 * negative nys_status_t: NYS_ERR_SHAPE / NYS_ERR_ARG for a shape the forward
 * call would reject, NYS_ERR_ARG for len < 0 or a NULL buf with len > 0.
 */
int nystrom_plan_describe(int B, int H, int n, int d, int m, int iters,
                          int conv_ks, int dtype, char* buf, int len);

/*
 * Queries and keys on their way into attention, and the cache that keeps keys
 * and values for later queries. These operators take heads of any stride:
 * a row is the d contiguous channels of one (batch entry, head, token), and
 * nys_strides_t gives the distance between rows in ELEMENTS along each of the
 * three, so [B][H][n][d] (the layout of the forward pass) and [B][n][H][d]
 * (a projection's output, or a slice of a packed one) are both read and
 * written in place. Row addresses are 16-byte aligned (else NYS_ERR_ALIGN),
 * strides are not negative, and rows of an output do not overlap one another or
 * another output's. Where an output may be an input, it has the same address and
 * strides; the same address with other strides, or of two outputs, is refused
 * (NYS_ERR_ARG).
 */
typedef struct { long long batch, head, token; } nys_strides_t;

/*
 * nystrom_qk_norm_rope_fwd - per-head RMS norm of queries and keys and the
 * rotation of their positions, in one pass. For each row x of q (k alike):
 *   z = w * x / sqrt(mean(x^2) + eps)      (norm = 0: z = x)
 *   (y_a, y_b) = (z_a cos t - z_b sin t, z_b cos t + z_a sin t)
 * for the rot/2 pairs (a, b) of channels among the first `rot`, with the angle
 *   t = position on pair i's axis * inv_freq[i];
 * channels from rot on pass through. Pair i is channels (i, i + rot/2) for
 * NYS_ROPE_HALVES and (2i, 2i + 1) for NYS_ROPE_PAIRS. The first section[0]
 * pairs turn with axis 0, the next section[1] with axis 1, and so on (text:
 * one axis; images and video: time, height, width).
 * positions: device int32 [axes][B][n], any value; or NULL for positions
 *   0 .. n-1 on every axis. inv_freq_host: HOST double [rot/2], radians per
 *   position (read during the call). Angles are reduced exactly, as 64-bit
 *   fractions of a turn, so far positions lose nothing.
 * q_weight, k_weight: device float [d], or NULL for all ones.
 * q, k in `dtype` with strides p->q, p->k; q_out, k_out likewise with
 *   p->q_out, p->k_out. An output may be its own input (same pointer, same
 *   strides), else they do not overlap. k (and k_out) may be NULL with Hk = 0.
 * Arithmetic in fp32, one rounding to dtype at the end.
 * Shape rules (else NYS_ERR_SHAPE): B, n, Hq >= 1, Hk >= 0, d % 8 == 0,
 *   8 <= d <= 128, rot even, 0 <= rot <= d, 1 <= axes <= 4, sections >= 0 that
 *   sum to rot/2, B*n < 2^31, (Hq + Hk) <= 65535. NYS_ERR_ARG for NULL
 *   pointers, an unknown pairing or dtype, a negative or non-finite eps, a
 *   non-finite frequency.
 *
 * nystrom_qk_norm_rope_bwd - its gradients: from the inputs q, k (strides
 * p->q, p->k) and the gradients gq, gk of the outputs (strides p->q_out,
 * p->k_out), with g the rotation undone on a row of gq, h = x / sqrt(mean(x^2)
 * + eps):
 *   dx = (w g - h mean(w g h)) / sqrt(mean(x^2) + eps),  dw = sum of g h
 * over all rows (norm = 0: dx = g). dq, dk in `dtype`, strides p->dq, p->dk;
 * dq may be gq and dk may be gk (same strides). dq_weight, dk_weight: device
 * float [d], overwritten, two arrays; NULL if not wanted. The sums are fp32 in a
 * fixed order: the same call gives the same bits.
 * workspace: device, 256-byte aligned, ws_bytes >=
 * nystrom_qk_norm_rope_workspace_bytes(p); needed only when a weight gradient
 * is asked for. NULL uses the library's cached workspace, which a stream
 * under capture may not do (NYS_ERR_ARG): a captured call brings its own.
 */
typedef enum { NYS_ROPE_HALVES = 0, NYS_ROPE_PAIRS = 1 } nys_rope_pairing_t;
typedef struct {
  int B, n, Hq, Hk, d;
  int rot;        /* rotated channels, from channel 0 on */
  int axes;       /* 1 .. 4 */
  int section[4]; /* pairs per axis */
  int pairing;    /* nys_rope_pairing_t */
  int norm;       /* 1: RMS norm first; 0: rotation alone */
  int dtype;
  float eps;
  nys_strides_t q, k, q_out, k_out;
  nys_strides_t dq, dk; /* backward only */
} nys_qk_rope_t;
int nystrom_qk_norm_rope_fwd(const nys_qk_rope_t* p, const void* q, const void* k,
                             const float* q_weight, const float* k_weight, const int* positions,
                             const double* inv_freq_host, void* q_out, void* k_out,
                             nys_stream_t stream);
size_t nystrom_qk_norm_rope_workspace_bytes(const nys_qk_rope_t* p);
int nystrom_qk_norm_rope_bwd(const nys_qk_rope_t* p, const void* q, const void* k,
                             const void* gq, const void* gk, const float* q_weight,
                             const float* k_weight, const int* positions,
                             const double* inv_freq_host, void* dq, void* dk, float* dq_weight,
                             float* dk_weight, void* workspace, size_t ws_bytes,
                             nys_stream_t stream);

/*
 * A key/value cache held in 4 bits. Each 32 consecutive channels of a token's
 * key (or value) share one scale: with a the largest magnitude among them,
 *   scale = a * (1/7), both and the product rounded to fp32, then rounded
 *           towards zero to bfloat16,
 *   code  = x / scale rounded to the nearest integer (ties to even), in -7..7,
 * and the cache stands for code * scale, so nothing grows in magnitude and no
 * value is off by more than half a scale. A block that holds an infinity or a
 * NaN gets a NaN scale and reads back as NaN.
 * The cache is a pool of pages; page p of sequence b is block_table[b][p], an
 * index into the pool, and holds tokens [p page_size, (p+1) page_size). In
 * memory the pool is [num_pages][Hk][page_size/16] blocks of 16 tokens, 18*d
 * bytes each (4.5 bits per value):
 *   key codes 8d bytes | key scales d | value codes 8d | value scales d.
 * Scales are bfloat16 [d/32][16 tokens]. A code + 8 is a 4-bit field; even
 * channels sit in the low half of a byte. With token r of the block, channel
 * c, group y = c/32, w = c%32: the key field is in byte
 *   r (d/2) + (w/8)(d/8) + 4y + (w%8)/2
 * of the key codes, the value field in byte
 *   (r/8) 4d + ((w/4) 4 + (r%8)/2)(d/8) + (r%2)(d/16) + 2y + (w%4)/2
 * of the value codes (the order in which the attention's matrix instructions
 * take them).
 * data: device, 16-byte aligned, nystrom_kv4_cache_bytes(...) bytes, never
 * initialised by the library: tokens that were not written hold whatever the
 * memory held, and no operator lets them into a result.
 * block_table: device int32 [B][max_pages]. Sequences may share pages that
 * are only read. Shape rules: num_pages, max_pages, Hk >= 1; page_size a
 * multiple of 16 in 16 .. 4096; d in {32, 64, 128}; max_pages * page_size <=
 * 2^31 - 2^16; nystrom_kv4_cache_bytes(...) <= 2^47.
 */
typedef struct {
  void* data;
  const int* block_table;
  int num_pages, max_pages, page_size, Hk, d;
} nys_kv4_cache_t;
size_t nystrom_kv4_cache_bytes(int num_pages, int page_size, int Hk, int d);

/*
 * nystrom_kv4_write - quantises rows i < counts[b] of k, v [B, Hk, n, d] (any
 * strides, NYS_FP32 or NYS_BF16) into the cache at positions starts[b] + i.
 * nystrom_kv4_read - the reverse: what the cache holds at positions starts[b]
 * + i, in `dtype`, to rows i < counts[b] of k, v; rows behind are left as they
 * were. (Read into [B][H][n][d], a cached context is the k and v of
 * nystrom_attn_fwd.)
 * starts: device int32 [B], or NULL for 0. counts: device int32 [B], or NULL
 * for n; a count above n is taken as n, one below 0 as 0.
 * A page outside the pool or a position outside the block table is skipped
 * (its rows of a read come back as zeros) and makes nystrom_get_status report
 * NYS_ERR_INDEX. Two sequences of one write must not name the same
 * page for positions they write.
 * B, n >= 1, B <= 65535, n * Hk < 2^33 (else NYS_ERR_SHAPE).
 */
int nystrom_kv4_write(const nys_kv4_cache_t* cache, const void* k, const void* v,
                      const nys_strides_t* k_strides, const nys_strides_t* v_strides,
                      const int* starts, const int* counts, int B, int n, int dtype,
                      nys_stream_t stream);
int nystrom_kv4_read(const nys_kv4_cache_t* cache, void* k, void* v,
                     const nys_strides_t* k_strides, const nys_strides_t* v_strides,
                     const int* starts, const int* counts, int B, int n, int dtype,
                     nys_stream_t stream);

/*
 * nystrom_kv4_attn_fwd - attention of nq new queries of each sequence over its
 * cached keys and values:
 *   out = softmax(q K^T * scale) V
 * q, out [B, Hq, nq, d] in `dtype`, any strides (out may be q, with the same
 * ones); query head h reads cache head h / (Hq/Hk). lengths: device int32 [B],
 * the tokens of each sequence in the cache (the new ones included). q_counts: device int32 [B], the real queries
 * of each sequence (NULL: nq); rows of out behind them are left as they were.
 * causal = 1: query i of c sees keys 0 .. length - c + i; causal = 0: all
 * `length` keys. A query that sees no key gives zeros. max_length: an upper
 * bound of the lengths that the host knows; the launch is planned by it.
 * A length outside 0 .. min(max_length, max_pages * page_size) is brought to
 * the nearer end, a page outside the pool counts as keys that are not seen;
 * both make nystrom_get_status report NYS_ERR_INDEX. scale: 0 means 1/sqrt(d).
 * Scores, the softmax and all sums are fp32. For NYS_BF16 the probabilities
 * enter the product with V as bf16; with more than 48 query rows per cache
 * head (nq * Hq/Hk, d in {64, 128}) they, and codes times scales, enter as
 * fp16 scaled by powers of two, or as bf16 where the value scales of 32 tokens
 * span more than 2^29. With x the largest, over a row's keys, of the probability
 * times the largest value scale of its 32 tokens, a probability there keeps fp16's
 * 11 bits down to 2^-25 x and is off by at most 2^-36 x below. Queries enter the scores as fp16 scaled by a power of two
 * per row, which loses nothing of channels down to 2^-26 of the row's largest. In
 * the calls of more rows keys lose nothing down to 2^-29 of the largest key scale
 * among the same 32 tokens; a smaller one is off by at most 2^-37 of that scale.
 * For NYS_FP32 queries and probabilities enter as sums of
 * 16-bit terms that keep at least 22 and 24 bits.
 * Shape rules: B, nq, Hk >= 1, Hq a multiple of Hk, Hq <= 65535, B <= 65535,
 * max_length >= 0, nq * (Hq/Hk) < 2^30, and the key tiles that all items could
 * have (32 keys x 16 query rows per cache head; more than 48 rows in bf16: 128 x
 * 256) below 2^31 (else NYS_ERR_SHAPE); scale * log2(e) finite (else NYS_ERR_ARG).
 * Magnitudes: in calls of few rows probabilities are kept up to 2^8 above 1, so
 * cached values beyond 2^100 may give infinities, as may bf16 queries that times
 * the scale go beyond 2^114. In calls of more rows scales below 2^-97 lose bits,
 * and value scales of 2^58 and more have no common measure with those of 32
 * tokens that are all below 2^-68 (or zero).
 * workspace: device, 256-byte aligned, ws_bytes >=
 * nystrom_kv4_attn_workspace_bytes(...) (which may be 0), not shared with a
 * call that may run at the same time. NULL uses the library's cached
 * workspace, which a stream under capture may not do (NYS_ERR_ARG).
 * nystrom_get_status reports NYS_ERR_INDEX and NYS_ERR_TIMEOUT of these cache
 * operators until they are read: they are not cleared by a later call. A first
 * call of a process may be captured, of these operators and of the norm and
 * rotation.
 */
size_t nystrom_kv4_attn_workspace_bytes(const nys_kv4_cache_t* cache, int B, int nq, int Hq,
                                        int max_length, int dtype);
int nystrom_kv4_attn_fwd(const nys_kv4_cache_t* cache, const void* q, void* out,
                         const nys_strides_t* q_strides, const nys_strides_t* out_strides,
                         const int* lengths, const int* q_counts, int B, int nq, int Hq,
                         int max_length, int causal, float scale, int dtype, void* workspace,
                         size_t ws_bytes, nys_stream_t stream);

/*
 * Around the attention module in a Transformer layer: the residual's addition
 * with the norm that follows it, projections in 8 bits, the gated feed-forward
 * product. These operators take matrices: rows are tokens (or a weight's output
 * channels), each a run of contiguous elements, `stride` elements apart, so a
 * slice of a wider matrix is read and written in place. Addresses are 16-byte
 * aligned and strides multiples of 16 bytes (else NYS_ERR_ALIGN). Rows of an
 * output do not overlap, nor those of a factor of nystrom_q8_matmul (a, w) and
 * nystrom_gated_ff (x, the weights): a stride below the row's length, with more
 * than one row, is NYS_ERR_ARG. Rows of other inputs may, down to a stride of 0
 * (one row for all). The stride of a single row does not matter. Outputs overlap
 * neither one another nor an input, except where an operator says so; one at the
 * very address of another, or of an input it may not be, is refused (NYS_ERR_ARG).
 */

/*
 * A matrix in 8 bits: `rows` rows of K e4m3 codes (4 exponent bits, 3 of
 * mantissa, largest 448), and for each row and block of 128 consecutive channels
 * (the last one of a row may be shorter) one scale, a power of two 2^(byte - 127)
 * (byte 255: NaN). The matrix stands for code * scale. scales: device, 32-bit
 * words [ceil(K/512)][rows], contiguous; byte j (from the low end) of word g of a
 * row is the scale of its block 4 g + j (0 behind the last block).
 * With a the largest magnitude of a block, its scale is the smallest power of two
 * with a <= 448 * scale, at least 2^-127 (a block of zeros), and a code is the
 * value over the scale, rounded to nearest, ties to even: nothing saturates, and
 * a value is off by at most 2^-4 of itself, or by 2^-10 * scale below 2^-6 * scale.
 * A block that holds an infinity or a NaN gets scale 255 and reads back as NaN.
 * Shape rules (else NYS_ERR_SHAPE): rows, K >= 1, K % 16 == 0, K <= 2^20,
 * rows < 2^31 - 2^10.
 */
typedef struct {
  void* codes;  /* device, 16-byte aligned */
  void* scales; /* device, 4-byte aligned, nystrom_q8_scales_bytes(rows, K) bytes */
  int rows, K;
  long long stride; /* bytes between rows of codes, a multiple of 16 */
} nys_q8_t;
size_t nystrom_q8_scales_bytes(int rows, int K);

/*
 * nystrom_q8_write - quantises x, [rows][K] in `dtype`, element (r, k) at
 * x[r row_stride + k channel_stride]; one of the two strides is 1 (a weight kept
 * as [K][rows], the order of nystrom_mha_fwd, is read as it lies), the other a
 * multiple of 16 bytes. Where row_stride is 1 and channel_stride is not, rows
 * must be a multiple of 8 (else NYS_ERR_SHAPE). block_rows: 1, or 128: the rows
 * 128 i .. 128 i + 127 share one scale per block of channels (weights).
 * nystrom_q8_read - the reverse: code * scale, rounded to `dtype`, to
 * out[r stride + k].
 */
int nystrom_q8_write(const nys_q8_t* q, const void* x, long long row_stride,
                     long long channel_stride, int block_rows, int dtype, nys_stream_t stream);
int nystrom_q8_read(const nys_q8_t* q, void* out, long long stride, int dtype,
                    nys_stream_t stream);

/*
 * nystrom_q8_matmul - out[t][n] = sum over k of A[t][k] W[n][k], the values that
 * the two 8-bit matrices stand for: a [T][K], w [N][K], out [T][N] in `dtype`
 * (row stride out_stride). Products are exact and summed in fp32 by the matrix
 * units (at most 32768 of a result, NYS_FP32: 1024, then in registers: the units
 * cut off towards zero), which apply the scales; one rounding to dtype. a's K and
 * w's are equal (else NYS_ERR_SHAPE); N a multiple of 8.
 * workspace: device, 256-byte aligned, ws_bytes >= nystrom_q8_matmul_workspace_bytes
 * (which may be 0), not shared with a call that may run at the same time. NULL
 * uses the library's cached workspace, which a stream under capture may not do
 * (NYS_ERR_ARG) where one is needed.
 */
size_t nystrom_q8_matmul_workspace_bytes(int T, int N, int K, int dtype);
int nystrom_q8_matmul(const nys_q8_t* a, const nys_q8_t* w, void* out, long long out_stride,
                      int dtype, void* workspace, size_t ws_bytes, nys_stream_t stream);

/*
 * nystrom_add_rms_norm_fwd - the residual's addition and the norm of the sum:
 *   s = x + residual, rounded to dtype (residual NULL: s = x, sum NULL)
 *   y = weight * s / sqrt(mean(s^2) + eps)
 * The sum of squares is fp32: a row whose sum passes 3.4e38 (values of 1e17 and more)
 * has y = 0, and with eps = 0 one whose sum is below 1e-45 has infinities or NaN.
 * x, residual, sum, y: [rows][d] in `dtype`, row strides p->x, p->residual,
 * p->sum, p->y. weight: device float [d], or NULL for all ones. sum and y may each
 * be x or residual (same address and stride). In place of y, y8: an 8-bit
 * matrix of rows x d (see nys_q8_t), quantised from y in fp32; exactly one of y
 * and y8 is given. sum may be NULL with a residual too: s is then not kept.
 * Shape rules (else NYS_ERR_SHAPE): rows >= 1, d % 8 == 0 (16 with y8),
 * 8 <= d <= 16384. NYS_ERR_ARG for a negative or non-finite eps.
 *
 * nystrom_add_rms_norm_bwd - its gradients: from s (stride p->sum), the gradient
 * gy of y (stride p->y) and gs of s from elsewhere (stride p->gs; NULL: none),
 * with r = 1 / sqrt(mean(s^2) + eps), h = r s:
 *   dx = gs + r (weight gy - h mean(weight gy h)),   dweight = sum over rows of gy h
 * dx [rows][d] in `dtype`, stride p->dx, is the gradient of x and of the residual
 * alike; it may be gy or gs (same address and stride). dweight: device float
 * [d], or NULL. Sums are fp32 in a fixed order: the same call gives the same
 * bits. workspace: as above, nystrom_add_rms_norm_workspace_bytes(p), needed for
 * dweight only.
 */
typedef struct {
  int rows, d, dtype;
  float eps;
  long long x, residual, sum, y; /* row strides in elements */
  long long gs, dx;              /* backward only */
} nys_add_rms_norm_t;
int nystrom_add_rms_norm_fwd(const nys_add_rms_norm_t* p, const void* x, const void* residual,
                             const float* weight, void* sum, void* y, const nys_q8_t* y8,
                             nys_stream_t stream);
size_t nystrom_add_rms_norm_workspace_bytes(const nys_add_rms_norm_t* p);
int nystrom_add_rms_norm_bwd(const nys_add_rms_norm_t* p, const void* s, const void* gy,
                             const void* gs, const float* weight, void* dx, float* dweight,
                             void* workspace, size_t ws_bytes, nys_stream_t stream);

/*
 * nystrom_gated_ff_fwd - both projections of a gated feed-forward block, the
 * activation and the product:
 *   g = x W_gate, u = x W_up, h = act(g) * u
 * x [T][d], h [T][f] in `dtype`, row strides p->x, p->h; weights in `dtype`:
 * NYS_FF_IN_OUT: [d][f], NYS_FF_OUT_IN: [f][d], row stride p->w, both alike.
 * gate, up: [T][f], row strides p->gate, p->up, receive g and u for the
 * backward pass; both or neither (NULL).
 * act: NYS_ACT_SILU g / (1 + e^-g); NYS_ACT_GELU g (1 + erf(g / sqrt 2)) / 2;
 * NYS_ACT_GELU_TANH g (1 + tanh(sqrt(2/pi) (g + 0.044715 g^3))) / 2;
 * NYS_ACT_RELU max(g, 0).
 *
 * nystrom_gated_ff_bwd - its gradients, from x, the weights, the kept g and u,
 * and the gradient gh of h (stride p->h):
 *   dg = gh u act'(g), du = gh act(g)     (act'(0) = 0 for RELU)
 *   dx = dg W_gate^T + du W_up^T, dW_gate = x^T dg, dW_up = x^T du
 * dx: stride p->dx, NULL if not wanted; dw_gate, dw_up: the weights' layout, row
 * stride p->dw, both or neither NULL.
 *
 * Sums are fp32 in the matrix units, in a fixed order; one rounding to dtype. The
 * units cut sums off towards zero, so they add up at most 16384 products of a result
 * (NYS_FP32: 64), which loses 2^-13 of the products' magnitudes at most, and registers
 * what is longer. For
 * NYS_BF16 dg and du enter the products rounded to bf16, of up to 128 tokens to two
 * bf16 terms (16 bits). Up to 24 tokens of NYS_FP32 are multiplied in fp32 (but for
 * the weights' gradients); else NYS_FP32 operands enter as sums of three bfloat16
 * terms (24 bits; six of the nine products, all that matter at 2^-24), so an
 * infinity gives NaN where a finite sum could not, values beyond 3.38e38 are
 * infinite, and bits below 2^-133 are lost.
 * Shape rules (else NYS_ERR_SHAPE): T, d, f >= 1, d % 8 == f % 8 == 0, d, f <= 2^20,
 * T <= 2^30.
 * workspace: as above (back: 0 forward, 1 backward).
 */
typedef enum { NYS_ACT_SILU = 0, NYS_ACT_GELU = 1, NYS_ACT_GELU_TANH = 2, NYS_ACT_RELU = 3 } nys_act_t;
typedef enum { NYS_FF_IN_OUT = 0, NYS_FF_OUT_IN = 1 } nys_ff_layout_t;
typedef struct {
  int T, d, f;
  int act, layout, dtype;
  long long x, w, h, gate, up; /* row strides in elements */
  long long dx, dw;            /* backward only */
} nys_gated_ff_t;
size_t nystrom_gated_ff_workspace_bytes(const nys_gated_ff_t* p, int back);
int nystrom_gated_ff_fwd(const nys_gated_ff_t* p, const void* x, const void* w_gate,
                         const void* w_up, void* h, void* gate, void* up, void* workspace,
                         size_t ws_bytes, nys_stream_t stream);
int nystrom_gated_ff_bwd(const nys_gated_ff_t* p, const void* x, const void* w_gate,
                         const void* w_up, const void* gate, const void* up, const void* gh,
                         void* dx, void* dw_gate, void* dw_up, void* workspace, size_t ws_bytes,
                         nys_stream_t stream);

/*
 * nystrom_get_status - waits for `stream`, then returns and clears the
 * device-side status word of the most recent forward call on the current device
 * (NYS_OK, or NYS_ERR_TIMEOUT if a bounded wait inside a kernel ran out; the
 * word is the library's, not part of a workspace, and a call that runs at the
 * same time on another stream sets the same one), then that of the cache operators and of those around the attention module
 * (NYS_ERR_INDEX of nystrom_kv4_*, NYS_ERR_TIMEOUT since it was last read).
 * Returns NYS_ERR_CUDA if the stream reports an error.
 */
int nystrom_get_status(nys_stream_t stream);

/*
 * Launch accounting and per-kernel timing, for benchmarks.
 * nystrom_launch_count: kernels this library has launched in this process
 * (all devices, all threads).
 * nystrom_profile_enable(1): from now on every kernel launch is bracketed
 * by two CUDA events recorded on the launch's own stream (adds two event
 * records per launch). nystrom_profile_enable(0) stops recording.
 * nystrom_profile_read: waits for the recorded events, returns the number of
 * distinct kernels seen since the last read (at most max_kernels are
 * written), and for kernel i writes its name to names + i*name_len
 * (NUL-terminated, truncated), its summed duration in ms to total_ms[i] and
 * its launch count to launches[i]; then forgets the records. Returns
 * NYS_ERR_CUDA if an event query fails.
 */
unsigned long long nystrom_launch_count(void);
int nystrom_profile_enable(int on);
int nystrom_profile_read(int max_kernels, char* names, int name_len,
                         double* total_ms, long long* launches);

/*
 * nystrom_debug_stall_pinv - testing the device-side timeout path. With
 * on = 1, every later forward call whose pseudo-inverse runs in the
 * tensor-core kernel for m <= 128 (bf16 inputs) makes that kernel wait, at
 * its start and before any copy or product is in flight, on a barrier phase
 * that nothing completes; the bounded wait runs out after 1 ms, the kernel
 * records NYS_ERR_TIMEOUT in the status word and skips its remaining work
 * (its outputs, and the call's output, are then undefined), and
 * nystrom_get_status reports NYS_ERR_TIMEOUT with the CUDA context intact.
 * on = 0 (the default) turns it off. Process-wide; not for production use.
 * Returns NYS_OK, or NYS_ERR_ARG for on other than 0 or 1.
 */
int nystrom_debug_stall_pinv(int on);

/* Static description of a status code. Never NULL. */
const char* nystrom_strerror(int code);

/* Text of the last CUDA error seen by this host thread ("" if none). */
const char* nystrom_last_error_string(void);

#ifdef __cplusplus
}
#endif

#endif /* NYSTROM_H_ */
