/*
 * psa_attn.h -- C ABI of the GB300 (sm_103a) PSA self-attention library.
 *
 * PSA attention runs two softmax-attention calls, "lo" and "hi", over one
 * packed per-(batch, head) buffer.  The calls share the Q and K sections, and
 * each owns one V section ("Struct PsaFa2Backward", vision_rs yolo attention
 * psa page: description and "Atomicity" paragraphs).  It is self-attention:
 * the query and key counts are both N (same page, description).  Because the
 * two calls share Q, K and therefore one softmax P, this library runs them as
 * ONE attention with a 2d-wide value [V_lo | V_hi]; the gradients it returns are
 * exactly those of the two calls, with dQ and dK summed over both.
 *
 * Notation, per (b, h) slice, all matrices [N, d] row-major:
 *   S = scale * Q K^T, LSE_i = ln sum_j exp(S_ij), P = exp(S - LSE 1^T),
 *   O_lo = P V_lo, O_hi = P V_hi.
 *
 * Common conventions
 *   - BH = B * heads slices; the slice index is the outermost index of every
 *     tensor.  packed / d_packed are [BH, 4, N, d]: sections 0..3 are
 *     Q, K, V_lo, V_hi (resp. dQ, dK, dV_lo, dV_hi).  o_lo, o_hi, do_lo, do_hi
 *     are [BH, N, d]; lse is [BH, N] fp32 (natural log, always fp32, whatever
 *     the storage type).  All contiguous, no padding.
 *   - Storage dtype: PSA_F32 or PSA_BF16 for every non-lse tensor; arithmetic
 *     accumulates in fp32.
 *   - head_dim (d) is one of 16, 32, 64.
 *   - All pointers are DEVICE pointers, 16-byte aligned.  The caller allocates
 *     and owns every buffer, including the backward workspace; the library
 *     allocates no device memory per call.
 *   - `stream` is a cudaStream_t (NULL = legacy default stream).  Calls are
 *     asynchronous on it and do not synchronise the host.
 *   - Return: 0 on success, a negative psa_status on error.  Arguments are
 *     checked before anything is launched; on an argument error nothing is
 *     launched and no buffer is touched.  psa_attn_last_error() returns a
 *     message for the calling thread's last error.
 *   - B*heads == 0 or N == 0 is a valid empty call (returns 0, launches nothing).
 */
#ifndef PSA_ATTN_H
#define PSA_ATTN_H

#include <stddef.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { PSA_F32 = 0, PSA_BF16 = 1, PSA_E4M3 = 2 /* of a rolling cache only */ } psa_dtype;

typedef enum {
    PSA_OK = 0,
    PSA_ERR_ARG = -1,          /* null pointer, negative size, non-finite scale, bad dtype */
    PSA_ERR_ALIGN = -2,        /* a pointer is not 16-byte aligned */
    PSA_ERR_UNSUPPORTED = -3,  /* head_dim not in {16, 32, 64}, or a size over the limits */
    PSA_ERR_WORKSPACE = -4,    /* workspace missing or smaller than psa_attn_bwd_workspace_bytes */
    PSA_ERR_CUDA = -5,         /* a CUDA launch / driver call failed (message has the CUDA error) */
    PSA_ERR_TIMEOUT = -6       /* a device-side bounded wait gave up (see psa_attn_sync_status) */
} psa_status;

/* Backward kernel choice.  AUTO picks the tensor-core (tcgen05) path where it
 * exists for the (dtype, head_dim) and the CUDA-core (SIMT) path elsewhere.
 *   PSA_ALGO_TC        one key-outer pass; dQ partial sums are added to an
 *                      fp32 accumulator by bulk reduce operations, and the
 *                      dK/dV products of neighbouring query sub-tiles come
 *                      from two issuing threads, in orders that can differ
 *                      from run to run, and so can the rounding of dQ, dK and
 *                      dV.  (The units of its last, partial wave are split
 *                      along the queries; their dK/dV partials are summed in
 *                      a fixed order.)
 *   PSA_ALGO_TC_2PASS  a key-outer dK/dV pass and a query-outer dQ pass
 *                      (the split of "Struct PsaFa2Backward", description:
 *                      query gradients from a sweep over keys, key gradients
 *                      from a sweep over queries); no atomics,
 *                      bit-for-bit reproducible.  Backward only (the forward
 *                      entry points reject it). */
typedef enum { PSA_ALGO_AUTO = 0, PSA_ALGO_SIMT = 1, PSA_ALGO_TC = 2, PSA_ALGO_TC_2PASS = 3 } psa_algo;

/*
 * psa_attn_fwd -- PSA forward: O_lo = P V_lo, O_hi = P V_hi and LSE.
 * Produces the forward outputs that the backward consumes; "Struct
 * PsaFa2Backward", "Grid" paragraph (the backward shares the forward pass's
 * decomposition).
 *   packed  [BH,4,N,d] dtype, read
 *   o_lo, o_hi [BH,N,d] dtype, written
 *   lse     [BH,N] fp32, written (natural log of the softmax denominator of scale*q.k)
 *   scale   softmax scale applied to q.k (finite)
 */
int psa_attn_fwd(const void* packed, void* o_lo, void* o_hi, float* lse,
                 int B, int heads, int N, int head_dim, float scale,
                 int dtype, void* stream);

/* Like psa_attn_fwd, with an explicit kernel choice (psa_algo): the
 * tensor-core forward (bf16 storage) or the CUDA-core forward (any storage).
 * PSA_ALGO_TC returns PSA_ERR_UNSUPPORTED for fp32 storage. */
int psa_attn_fwd_algo(const void* packed, void* o_lo, void* o_hi, float* lse,
                      int B, int heads, int N, int head_dim, float scale,
                      int dtype, int algo, void* stream);

/*
 * Bytes of device workspace psa_attn_bwd needs for these sizes and the kernel
 * AUTO would pick: the fp32 row statistics D (the CUDA-core and two-pass
 * paths), or on the fused tensor-core path 8 bytes of row statistics per query
 * (LSE and D, padded to whole 64-query tiles), an fp32 dQ accumulator and room
 * for the fp32 dK/dV partials of split units.  The size does not depend on the
 * GPU.  Returns 0 for an empty or invalid problem.
 */
size_t psa_attn_bwd_workspace_bytes(int B, int heads, int N, int head_dim, int dtype);

/*
 * psa_attn_bwd -- PSA backward (the lo/hi pair of FA2 backward calls).
 * "Struct PsaFa2Backward": description (P is recomputed from Q, K and the row
 * statistics; query gradients need a sweep over keys, key gradients a sweep
 * over queries),
 * "Atomicity" (dQ, dK summed over lo and hi; each call owns its dV section).
 *   packed       [BH,4,N,d] dtype, read (Q, K, V_lo, V_hi)
 *   o_lo, o_hi   [BH,N,d] dtype, read (forward outputs)
 *   lse          [BH,N] fp32, read (from psa_attn_fwd)
 *   do_lo, do_hi [BH,N,d] dtype, read (upstream gradients)
 *   d_packed     [BH,4,N,d] dtype, OVERWRITTEN with dQ, dK, dV_lo, dV_hi
 *                (the page's kernel adds into a zeroed buffer; this call writes
 *                the gradients, so d_packed need not be zeroed first)
 *   workspace    device scratch of at least workspace_bytes; contents on entry
 *                are ignored, contents on exit are unspecified
 * Calls that share a workspace must not overlap on the GPU.
 */
int psa_attn_bwd(const void* packed, const void* o_lo, const void* o_hi, const float* lse,
                 const void* do_lo, const void* do_hi, void* d_packed,
                 void* workspace, size_t workspace_bytes,
                 int B, int heads, int N, int head_dim, float scale,
                 int dtype, void* stream);

/* Like psa_attn_bwd, with an explicit kernel choice (psa_algo).  PSA_ALGO_TC
 * and PSA_ALGO_TC_2PASS return PSA_ERR_UNSUPPORTED where no tensor-core kernel
 * exists for the (dtype, head_dim). */
int psa_attn_bwd_algo(const void* packed, const void* o_lo, const void* o_hi, const float* lse,
                      const void* do_lo, const void* do_hi, void* d_packed,
                      void* workspace, size_t workspace_bytes,
                      int B, int heads, int N, int head_dim, float scale,
                      int dtype, int algo, void* stream);

/*
 * psa_attn_view -- a strided view of a [B, heads, N, d] tensor: element
 * (b, h, n, j) (batch, head, position, feature) is at
 *   base + b*batch_stride + h*head_stride + n*pos_stride + j*feat_stride
 * with strides in elements.  Row-major rows ([N, d] per slice, as
 * psa_attn_bwd takes dO): feat_stride = 1, pos_stride >= d (a padded row when
 * larger).  Channel-major ([d, N] per slice, as a [B, c, H, W] feature map
 * holds it): pos_stride = 1, feat_stride >= N.
 */
typedef struct {
    const void* base;
    long long batch_stride, head_stride, pos_stride, feat_stride;
} psa_attn_view;

/*
 * psa_attn_bwd_ex -- psa_attn_bwd on strided layouts.  "Struct
 * PsaMergeAttnRuntimeOp" (forward_output_row_stride,
 * backward_grad_output_row_stride: a buffer's row stride may be rounded up
 * past the row length so that every row starts on a 16-byte boundary, as TMA
 * copies need) and the channel-major feature maps of the model around the op.
 *   packed          [BH, 4, N, qkv_row_stride] dtype, read: rows of d used
 *                   (section stride N*qkv_row_stride, slice stride 4*N*qkv_row_stride)
 *   qkv_row_stride  >= head_dim; also the row stride of d_packed
 *   o_lo, o_hi      [BH, N, o_row_stride] dtype, read; o_row_stride >= head_dim
 *   lse             [BH, N] fp32, read
 *   do_lo, do_hi    views (above) of the upstream gradients, read
 *   d_packed        [BH, 4, N, qkv_row_stride] dtype: the first head_dim
 *                   elements of every row are OVERWRITTEN, the padding is not
 *                   touched
 *   workspace       at least psa_attn_bwd_ex_workspace_bytes(...) bytes
 *   algo            PSA_ALGO_AUTO, PSA_ALGO_TC (fused tensor-core kernel, bf16)
 *                   or PSA_ALGO_SIMT; the two-pass mode takes contiguous
 *                   tensors only (psa_attn_bwd_algo)
 * Alignment: every pointer 16-byte aligned.  The tensor-core path also needs
 * every stride other than a unit one to be a multiple of 16 bytes (TMA); the
 * CUDA-core path needs qkv_row_stride = o_row_stride = head_dim (it gathers
 * strided dO views into the workspace first).  Violations return
 * PSA_ERR_ALIGN or PSA_ERR_UNSUPPORTED before anything is launched.
 * Other arguments, results and errors as psa_attn_bwd_algo.
 */
int psa_attn_bwd_ex(const void* packed, long long qkv_row_stride,
                    const void* o_lo, const void* o_hi, long long o_row_stride,
                    const float* lse, const psa_attn_view* do_lo, const psa_attn_view* do_hi,
                    void* d_packed, void* workspace, size_t workspace_bytes,
                    int B, int heads, int N, int head_dim, float scale,
                    int dtype, int algo, void* stream);

/* Workspace bytes psa_attn_bwd_ex needs (0 for an empty or invalid problem). */
size_t psa_attn_bwd_ex_workspace_bytes(const psa_attn_view* do_lo, const psa_attn_view* do_hi,
                                       int B, int heads, int N, int head_dim, int dtype, int algo);

/*
 * psa_merge_bwd -- the backward of the PSA attention merge alone
 * ("Struct PsaMergeAttnRuntimeOp", pack_backward_args: d_merged, d_lo, d_hi,
 * c, H, W, num_heads; backward_grid: one block per (batch*head, position)).
 * The merged tensor is [B, c, H, W], c = 2 * heads * head_dim, N = H * W;
 * its channels hold the lo outputs of every head in the low half and the hi
 * outputs in the high half, head-major in each half (a reading: the pages
 * name the arguments, not the order):
 *   d_lo[b*heads + h, n, j] = d_merged[b, h*head_dim + j, n]
 *   d_hi[b*heads + h, n, j] = d_merged[b, heads*head_dim + h*head_dim + j, n]
 *   d_merged  [B, c, H, W] dtype, read;  d_lo, d_hi  [B*heads, N, d] dtype, written
 */
int psa_merge_bwd(const void* d_merged, void* d_lo, void* d_hi, int B, int heads, int H, int W,
                  int head_dim, int dtype, void* stream);

/*
 * psa_merge_attn_bwd -- the merge's backward fused into the attention
 * backward: the kernels read dO_lo and dO_hi straight out of d_merged (the
 * views of psa_merge_bwd's mapping), so d_lo / d_hi are never written.
 * Arguments as psa_attn_bwd, with d_merged [B, 2*heads*head_dim, H, W] in
 * place of do_lo / do_hi and N = H * W; the workspace is
 * psa_merge_attn_bwd_workspace_bytes(...) bytes.  The tensor-core path needs
 * H * W a multiple of 8 (rows of d_merged 16-byte aligned).
 */
int psa_merge_attn_bwd(const void* packed, const void* o_lo, const void* o_hi, const float* lse,
                       const void* d_merged, void* d_packed, void* workspace, size_t workspace_bytes,
                       int B, int heads, int H, int W, int head_dim, float scale,
                       int dtype, int algo, void* stream);
size_t psa_merge_attn_bwd_workspace_bytes(int B, int heads, int H, int W, int head_dim, int dtype, int algo);

/*
 * psa_attn_bwd_noalloc -- the backward for callers that cannot allocate device
 * memory.  (The pages have no counterpart of this entry point; it is a
 * convenience of this library.)
 *
 * Some callers cannot call cudaMalloc or any allocating routine: a plugin that
 * is handed only its input and output buffers by a host runtime that owns all
 * device memory, or an application whose memory budget is fixed after start-up
 * and forbids libraries from allocating later.  psa_attn_bwd needs a workspace
 * from its caller; this variant needs none.  It runs the CUDA-core backward
 * (PSA_ALGO_SIMT) and keeps its only scratch -- the fp32 row statistics D, one
 * value per query row -- in a static array inside this library's device
 * memory, 2 MiB per GPU, which every GPU that loads the library holds until the
 * process exits.  The call itself allocates nothing (no cudaMalloc, cudaFree or
 * allocating library routine).
 *   Arguments and results are those of psa_attn_bwd without the workspace.
 *   Limit: B*heads*N <= psa_attn_bwd_noalloc_max_rows() (524288); larger
 *   problems return PSA_ERR_UNSUPPORTED before anything is launched.
 *   Set-up: the first call on each device looks up the device address of the
 *   static array (with that device current) and caches it; make that first
 *   call before any stream capture.
 *   Sharing: every call on a device uses the same array.  D is rewritten in
 *   full by each call before it is read, so a call never sees an earlier
 *   call's values, but calls that overlap on the GPU (different streams, or
 *   different host threads, without ordering between them) race on it.
 */
int psa_attn_bwd_noalloc(const void* packed, const void* o_lo, const void* o_hi, const float* lse,
                         const void* do_lo, const void* do_hi, void* d_packed,
                         int B, int heads, int N, int head_dim, float scale,
                         int dtype, void* stream);

/* Largest B*heads*N psa_attn_bwd_noalloc accepts. */
long long psa_attn_bwd_noalloc_max_rows(void);

/* ------------------------------------------------------------------------
 * Sliding-window attention with sinks, rotary positions and a rolling cache
 * (the pages have no counterpart of these entry points).
 *
 * Attention of q_heads query heads over kv_heads key/value heads (head h reads
 * key head h / (q_heads / kv_heads)), causal, where a row sees the last
 * `window` positions and the first `sinks` positions of its sequence:
 *   row i of sequence b has the position p = L_b - Q_b + i, Q_b = q_lens[b]
 *   query rows and L_b = kv_lens[b] keys, and sees key j when
 *   j <= p and (j > p - window or j < sinks).
 *   O_i = sum_j P_ij V_j,  P_ij = exp(scale q_i.k_j - LSE_i),
 *   LSE_i = ln sum over the visible j of exp(scale q_i.k_j).
 * A row that sees no key (p < 0: more rows than keys) has O = 0, LSE = -inf and
 * zero gradients.  Rows i >= Q_b are padding: their O, dQ are written as 0 and
 * their LSE as -inf; keys j >= L_b are padding: their dK, dV are written as 0.
 * What padding holds (NaN too) has no effect, but whole tiles of it may be read:
 * a view is readable memory up to its N rows.  A non-finite value in a
 * real token may reach the outputs of any row of its sequence.
 *   dtype, pointers, streams, empty calls and errors as above; tensors are
 *   psa_attn_view views [B, heads, N, head_dim] with any non-negative strides
 *   (an output's must not make two elements coincide), bases 16-byte aligned; no
 *   output overlaps another tensor, but where an operator says so.
 *   head_dim is 16, 32, 64 or 128; at most 2^30 rows, keys or cache slots.
 */
typedef struct {
    int B, q_heads, kv_heads; /* q_heads a multiple of kv_heads */
    int Nq, Nk;               /* rows of q, o, dO, dQ; rows of k, v, dK, dV */
    int head_dim;
    int window;               /* >= 1; >= Nk: plain causal attention */
    int sinks;                /* >= 0; 0: a plain sliding window */
    float scale;
    int dtype;
} psa_win_shape;

/*
 * psa_win_attn_fwd -- O and LSE.
 *   q, k, v   views, read;  o  view, written (its base is written through)
 *   lse       [B, q_heads, Nq] fp32, written, contiguous, 16-byte aligned
 *   q_lens, kv_lens   DEVICE int32 [B] or NULL (NULL: Nq resp. Nk for every
 *             sequence); values outside 0..Nq resp. 0..Nk are clamped to them
 *   algo      PSA_ALGO_AUTO, PSA_ALGO_SIMT (products by warps, for both dtypes and
 *             any strides, fp32 in fp32's accuracy) or PSA_ALGO_TC (tcgen05: bf16,
 *             scale >= 1e-30, every feat_stride 1 and every other stride of a
 *             dimension longer than 1 a non-zero multiple of 16 bytes; else
 *             PSA_ERR_UNSUPPORTED).  AUTO picks TC where it is supported.
 */
int psa_win_attn_fwd(const psa_win_shape* shape, const psa_attn_view* q, const psa_attn_view* k,
                     const psa_attn_view* v, const psa_attn_view* o, float* lse, const int* q_lens,
                     const int* kv_lens, int algo, void* stream);

/*
 * psa_win_attn_bwd -- dQ, dK, dV of a loss whose gradient in O is dO; dK and dV
 * are summed over the query heads that share a key head, in a fixed order (no
 * atomics: the same inputs give the same bits).
 *   o, lse    psa_win_attn_fwd's outputs, read;  d_o  view, read
 *   dq, dk, dv  views, OVERWRITTEN
 *   workspace  as for psa_attn_bwd; psa_win_attn_bwd_workspace_bytes bytes,
 *              the same for every algo
 *   other arguments as psa_win_attn_fwd (the layout rule of PSA_ALGO_TC covers
 *   every view)
 */
int psa_win_attn_bwd(const psa_win_shape* shape, const psa_attn_view* q, const psa_attn_view* k,
                     const psa_attn_view* v, const psa_attn_view* o, const float* lse, const psa_attn_view* d_o,
                     const psa_attn_view* dq, const psa_attn_view* dk, const psa_attn_view* dv, const int* q_lens,
                     const int* kv_lens, void* workspace, size_t workspace_bytes, int algo, void* stream);

/* Workspace bytes of psa_win_attn_bwd (0 for an empty or invalid problem). */
size_t psa_win_attn_bwd_workspace_bytes(const psa_win_shape* shape);

/*
 * Rotary positions with up to three axes (say time, row, column).  The first
 * rot_dim features of a head form rot_dim / 2 pairs; pair i belongs to axis
 * a(i) (the first sections[0] pairs to axis 0, the next sections[1] to axis 1,
 * ...) and turns by the angle pos[a(i)] * f_i:
 *   y1 = x1 cos - x2 sin,  y2 = x2 cos + x1 sin.
 * PSA_ROPE_SHARED: f_i = theta^(-i / n), n = rot_dim / 2, one ladder of
 * frequencies over all axes.  PSA_ROPE_PER_AXIS: every axis has a ladder of its
 * own, f = theta^(-k / s) for its pair k of s.  Pair i is the features i and
 * i + n, or 2i and 2i + 1 when interleaved.  Features past rot_dim are copied.
 *
 * A plan holds the frequencies in units of 2^-64 turns, rounded, so that an angle
 * modulo a turn is off by at most 2^-34 turns at any 32-bit position; it is plain
 * host memory, made once by psa_rope_plan_init and passed to the calls, which copy it.
 */
enum { PSA_ROPE_SHARED = 0, PSA_ROPE_PER_AXIS = 1 };
#define PSA_ROPE_MAX_PAIRS 64
typedef struct {
    int head_dim, rot_dim, n_axes, interleaved;
    unsigned long long turn[PSA_ROPE_MAX_PAIRS]; /* f_i / 2 pi in units of 2^-64 turns */
    unsigned char axis[PSA_ROPE_MAX_PAIRS];
} psa_rope_plan;

/* sections: n_axes (1..3) pair counts >= 0 that add up to rot_dim / 2; rot_dim
 * even, 2..head_dim; head_dim 16, 32, 64 or 128; theta > 1 and finite. */
int psa_rope_plan_init(psa_rope_plan* plan, int head_dim, int rot_dim, int n_axes, const int* sections,
                       double theta, int ladder, int interleaved);

/*
 * psa_rope -- y = rotated x and (x2 not NULL) y2 = rotated x2, say the queries
 * and the keys, in one launch; inverse != 0 turns back, which is the gradient
 * (dx from dy).
 *   x, y    views [B, heads, N, head_dim], read / written; in place when y is
 *           the same view as x (a partial overlap gives undefined values)
 *   x2, y2  views [B, heads2, N, head_dim], both NULL or both given
 *   pos     DEVICE int32, element (axis a, sequence b, row n) at
 *           a*pos_axis_stride + b*pos_batch_stride + n (strides >= 0: a batch
 *           stride of 0 shares the positions); any value, negative ones too
 */
int psa_rope(const psa_rope_plan* plan, const psa_attn_view* x, const psa_attn_view* y, int heads,
             const psa_attn_view* x2, const psa_attn_view* y2, int heads2, int B, int N, const int* pos,
             long long pos_axis_stride, long long pos_batch_stride, int inverse, int dtype, void* stream);

/*
 * A rolling key/value cache [B, kv_heads, capacity, head_dim]: position p of a
 * sequence lives in slot p for p < sinks, else in slot
 * sinks + (p - sinks) mod (capacity - sinks), so that the sinks and the newest
 * capacity - sinks positions are kept.  capacity >= sinks + window.  A capacity
 * no sequence outgrows makes it a plain cache (slot = position).
 */
typedef struct {
    void* k;
    void* v;
    int B, kv_heads, capacity, head_dim, window, sinks, dtype;
    long long batch_stride, head_stride, slot_stride; /* elements, of k and of v; features adjacent */
} psa_win_cache;

/*
 * psa_win_cache_append -- writes the keys and values of new positions into
 * their slots: row t of sequence b is position start[b] + t, t < n_new[b] <= T;
 * of the rows that share a slot only the newest is written.  Slots of other
 * positions are not touched.
 *   k_new, v_new  views [B, kv_heads, T, head_dim], read
 *   start         DEVICE int32 [B], >= 0 (a sequence with a negative start, or
 *                 whose last position would pass 2^31 - 1, is skipped; position
 *                 2^31 - 1 itself is written, but psa_win_decode's lens ends there)
 *   n_new         DEVICE int32 [B] or NULL (T rows each); clamped to 0..T
 *   plan, pos     NULL, or the rotation applied to the keys on the way, as in
 *                 psa_rope (pos element (a, b, t))
 */
int psa_win_cache_append(const psa_win_cache* cache, const psa_attn_view* k_new, const psa_attn_view* v_new, int T,
                         const int* start, const int* n_new, const psa_rope_plan* plan, const int* pos,
                         long long pos_axis_stride, long long pos_batch_stride, void* stream);

/*
 * psa_win_decode -- attention of one query row per sequence, at position
 * lens[b] - 1, over the cache: it sees the positions p < lens[b] with p < sinks
 * or p >= lens[b] - window (which the cache holds by its capacity).
 *   q, o   views [B, q_heads, 1, head_dim] (pos_stride is not used)
 *   lse    [B, q_heads] fp32 or NULL
 *   lens   DEVICE int32 [B], positions appended so far, the newest included;
 *          <= 0: the sequence is empty, O = 0 and LSE = -inf
 *   workspace  psa_win_decode_workspace_bytes bytes (0: none is needed), as for
 *          psa_attn_bwd
 * The same inputs give the same bits.
 */
int psa_win_decode(const psa_win_cache* cache, const psa_attn_view* q, const psa_attn_view* o, float* lse,
                   int q_heads, const int* lens, float scale, void* workspace, size_t workspace_bytes,
                   void* stream);
size_t psa_win_decode_workspace_bytes(const psa_win_cache* cache, int q_heads);

/*
 * The cache in 8 bits, drafted tokens, and reading a cache back.
 *
 * An 8-bit cache is a psa_win_cache of dtype PSA_E4M3 (k, v: e4m3 codes, strides in
 * bytes) with psa_win_scales: a stored row is its d codes times its scale.  Rows are
 * quantised as they are written: the scale is the smallest power of two s >= 2^-100 with
 * max|x| <= 448 s, the codes are x / s rounded to e4m3 (to nearest, ties to even); a row with
 * an element that is not finite gets the scale NaN.  (A number above 248 * 2^120 becomes 2^128,
 * which reads back as an infinity.)  Caches filled in another way may have
 * any finite scales >= 0; one below 2^-126 may count as 0.  Attention on the tensor
 * cores (psa_win_tree_attn) takes a cached element as its code times its scale rounded to bf16:
 * exact where the scale has at most 4 significant bits, as the writes' powers of two have, off by up to
 * 2^-8 of the element otherwise.  Everything else here takes the scales as they are, in fp32.
 *   The functions below take caches of all three types, `scales` NULL for PSA_F32 and
 * PSA_BF16; psa_win_cache_append and psa_win_decode take the latter two only.  `dtype`
 * is the type of the other tensors, PSA_F32 or PSA_BF16; it is the cache's, unless that is
 * PSA_E4M3 (psa_win_read converts between all types).
 */
typedef struct {
    float* k; /* [B, kv_heads, capacity] */
    float* v;
    long long batch_stride, head_stride, slot_stride; /* elements, of k and of v */
} psa_win_scales;

/*
 * psa_win_store -- psa_win_cache_append for caches of every type, with the new rows
 * taken by index, say those of an accepted path through a tree of drafts:
 *   k_new, v_new  views [B, kv_heads, T, head_dim] of dtype, read
 *   rows          NULL, or DEVICE int32: position start[b] + i is row
 *                 rows[b * rows_stride + i] of sequence b, i < n_new[b] <= R.  A position
 *                 whose row is not in 0..T-1 is left as it was.  NULL: row i, R = T
 *   R             positions per sequence at most (given with rows NULL too)
 *   plan, pos     as in psa_win_cache_append; pos belongs to the rows of k_new
 *   other arguments as psa_win_cache_append
 */
int psa_win_store(const psa_win_cache* cache, const psa_win_scales* scales, const psa_attn_view* k_new,
                  const psa_attn_view* v_new, int T, const int* rows, long long rows_stride, int R, const int* start,
                  const int* n_new, const psa_rope_plan* plan, const int* pos, long long pos_axis_stride,
                  long long pos_batch_stride, int dtype, void* stream);

/*
 * psa_win_read -- the positions first[b] .. first[b] + N - 1 of every sequence, in order.
 *   k, v    views [B, kv_heads, N, head_dim] of dtype, written: 0 where the cache does not
 *           hold a position (p < 0, p >= lens[b], or overwritten: p >= sinks and
 *           p < lens[b] - (capacity - sinks))
 *   first   DEVICE int32 [B];  lens  DEVICE int32 [B], positions appended so far
 */
int psa_win_read(const psa_win_cache* cache, const psa_win_scales* scales, const psa_attn_view* k, const psa_attn_view* v,
                 int N, const int* first, const int* lens, int dtype, void* stream);

/*
 * psa_win_decode_any -- psa_win_decode for caches of every type (q, o of dtype).
 */
int psa_win_decode_any(const psa_win_cache* cache, const psa_win_scales* scales, const psa_attn_view* q,
                       const psa_attn_view* o, float* lse, int q_heads, const int* lens, float scale, void* workspace,
                       size_t workspace_bytes, int dtype, void* stream);
size_t psa_win_decode_any_workspace_bytes(const psa_win_cache* cache, int q_heads, int dtype);

/*
 * psa_win_tree_attn -- attention of T new tokens per sequence, which the cache does not
 * hold, over the cache and over each other: a tree of drafts, or a run of tokens.
 *   Node t of sequence b has the parent parents[b * parents_stride + t], one of
 * 0..t-1; any other value makes it a root, a child of the cache's last position.  It sits at
 * position p = lens[b] + (number of its ancestors).  It sees the cached positions j < lens[b]
 * with j < sinks or j > p - window, and of its ancestors and itself those whose position
 * is below sinks or above p - window.  (So a node sees what psa_win_decode would, had its path
 * been appended.)
 *   q, o    views [B, q_heads, T, head_dim];  k_new, v_new  views [B, kv_heads, T, head_dim]
 *           (keys rotated already, where positions are rotary)
 *   lse     [B, q_heads, T] fp32 or NULL
 *   parents DEVICE int32 or NULL: a run, each token's parent is the one before it;
 *           parents_stride 0 shares one tree
 *   n_new   DEVICE int32 [B] or NULL (T each), clamped to 0..T: nodes t >= n_new[b] are
 *           padding, whose O is 0 and LSE -inf and whose contents have no effect
 *   lens    DEVICE int32 [B], positions that the cache holds; <= 0: none
 *   T       at most PSA_TREE_MAX
 *   algo    PSA_ALGO_AUTO, PSA_ALGO_SIMT (products by warps) or PSA_ALGO_TC (tcgen05; where
 *           it does not take the call, PSA_ERR_UNSUPPORTED); AUTO takes the tensor
 *           cores where they can, but for up to 32 rows per key head over an 8-bit cache, where
 *           sequences, key heads, window and head_dim decide.  Over an 8-bit
 *           cache whose scales are no powers of two they differ by the rounding that the tensor
 *           cores' kernel makes (above); PSA_ALGO_SIMT makes none
 *   workspace  psa_win_tree_attn_workspace_bytes bytes (0: none is needed), the same for
 *           every algo, as for psa_attn_bwd
 * The same inputs give the same bits.  A value that is not finite may reach the nodes of
 * its sequence that do not see it, where others do (as 0 times it); a key does not.
 */
#define PSA_TREE_MAX 256
int psa_win_tree_attn(const psa_win_cache* cache, const psa_win_scales* scales, const psa_attn_view* q,
                      const psa_attn_view* k_new, const psa_attn_view* v_new, const psa_attn_view* o, float* lse, int q_heads,
                      int T, const int* parents, long long parents_stride, const int* n_new, const int* lens, float scale,
                      void* workspace, size_t workspace_bytes, int algo, int dtype, void* stream);
size_t psa_win_tree_attn_workspace_bytes(const psa_win_cache* cache, int q_heads, int T, int dtype);

/* Workspace bytes for an explicit kernel choice (0 if unsupported). */
size_t psa_attn_bwd_workspace_bytes_algo(int B, int heads, int N, int head_dim, int dtype, int algo);

/*
 * psa_attn_bwd_host -- the backward on HOST buffers: copies the inputs to the
 * device, runs psa_attn_bwd_algo and copies d_packed back, all enqueued on
 * `stream`.  (The pages have no counterpart; it is this library's end-to-end
 * entry point.)  The (batch*head) slices are independent, so they are split
 * into `chunks` groups whose copy in, backward and copy back are pipelined:
 * the copies run on two streams this library creates once per device, and the
 * kernels on `stream`.
 *   packed ... d_packed  HOST pointers, layouts as in psa_attn_bwd (d_packed is
 *                written).  Page-locked memory (cudaHostAlloc or
 *                cudaHostRegister) makes the copies asynchronous; with pageable
 *                memory the call still works, but the copies block the host.
 *   dev_buf      DEVICE scratch, 256-byte aligned, at least
 *                psa_attn_bwd_host_buffer_bytes(...) bytes: the device copies of
 *                every input and of d_packed, then the backward workspace.
 *                Contents on entry are ignored; on exit unspecified.
 *   algo         as psa_attn_bwd_algo.
 *   chunks       0 = chosen by the library from the sizes and the GPU
 *                (psa_attn_bwd_host_chunks); else 1..64, capped at B*heads.
 *                With N % 4 != 0 the call runs as one chunk (every chunk's lse
 *                must start on a 16-byte boundary).
 *   stream       the call starts after earlier work on `stream`; work enqueued
 *                on `stream` after the call starts after d_packed has landed in
 *                host memory.  Asynchronous: synchronise `stream` before reading
 *                d_packed.
 * Returns as psa_attn_bwd (PSA_ERR_WORKSPACE: dev_buf missing or too small;
 * PSA_ERR_ALIGN: dev_buf not 256-byte aligned).  An empty problem returns 0
 * and touches nothing.  Calls that share dev_buf must not overlap on the GPU;
 * calls from several host threads are serialised while they enqueue.
 */
int psa_attn_bwd_host(const void* packed, const void* o_lo, const void* o_hi, const float* lse,
                      const void* do_lo, const void* do_hi, void* d_packed,
                      void* dev_buf, size_t dev_buf_bytes,
                      int B, int heads, int N, int head_dim, float scale,
                      int dtype, int algo, int chunks, void* stream);

/* Device buffer bytes psa_attn_bwd_host needs (0 for an empty or invalid
 * problem); they do not depend on the chunk count. */
size_t psa_attn_bwd_host_buffer_bytes(int B, int heads, int N, int head_dim, int dtype, int algo);

/* The chunk count psa_attn_bwd_host uses for chunks = 0 on the current device
 * (1 when no device is available). */
int psa_attn_bwd_host_chunks(int B, int heads, int N, int head_dim, int dtype, int algo);

/*
 * Synchronises `stream`, then reports whether any kernel of this library gave
 * up on a bounded device-side wait since the last check (PSA_ERR_TIMEOUT, and
 * the flag is cleared), or whether the stream has a CUDA error (PSA_ERR_CUDA).
 * Returns 0 otherwise.
 */
int psa_attn_sync_status(void* stream);

/*
 * Failure-detection self-test (the pages have no counterpart).  Launches, on
 * `stream`, one small kernel that waits -- through the same bounded device-side
 * wait the backward kernels use -- on a barrier nothing ever arrives on, with
 * a 20 ms limit.  The wait gives up, records the timeout in the device error
 * word and the kernel exits normally; no fault, no trap, and the CUDA context
 * stays usable.  A following psa_attn_sync_status(stream) returns
 * PSA_ERR_TIMEOUT and clears the word.  Returns 0 if the launch succeeded.
 */
int psa_attn_selftest_wait_timeout(void* stream);

/*
 * Kernel timing (instrumentation; it changes no result and skips no work).
 * While enabled, every launch this library makes records a pair of CUDA events
 * around itself on the call's stream, tagged with a slot: 0 = forward,
 * 1 = backward preprocess (D), 2 = backward main (dK/dV, and dQ on the
 * tensor-core path), 3 = backward dQ (CUDA-core path) / dQ finalize.  The
 * window attention uses the same slots (its sink rows' sums are in 2), the
 * attention of single and of drafted tokens slot 0; the rotation, the cache's
 * writes and its reads have none.
 * psa_attn_profile_read() synchronises those events, writes per-slot total
 * milliseconds and launch counts into the caller's arrays (length >= 4) and
 * clears the records.  Returns the number of slots, or a negative psa_status.
 * Without timing, the tensor-core backward's main and finalize kernels start
 * as programmatic dependents of the kernel before them (their blocks are
 * scheduled while it finishes); with timing on they start after it, one by
 * one, so that each pair of events measures one kernel.
 */
int psa_attn_profile_enable(int on);
int psa_attn_profile_read(float* total_ms, int* launches, int n_slots);
const char* psa_attn_profile_slot_name(int slot);

/* Message for the calling thread's most recent error ("" if none). */
const char* psa_attn_last_error(void);

/* Library version as MAJOR*10000 + MINOR*100 + PATCH. */
int psa_attn_version(void);

#ifdef __cplusplus
}
#endif

#endif /* PSA_ATTN_H */
