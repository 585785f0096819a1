/*
 * txl_attn.h -- C ABI of the GB300 (sm_103a) Transformer-XL relative
 * attention library (libtxl.so).
 *
 * The operation is relative multi-head attention over a per-layer recurrence
 * memory, as defined by:
 *   - "Transformer-XL" course notes (zty624.github.io), sections
 *     "Segment-Level Recurrence", "Batched Tensor Contract",
 *     "Causal Mask With Memory", "Relative Positional Encoding" and
 *     "Relative Shift Trick";
 *   - "Transformer-XL模型 核心源码阅读笔记" (CSDN source-reading notes),
 *     section "Build the model": RelPartialLearnableMultiHeadAttn.forward and
 *     MemTransformerLM._forward / _update_mems.
 *
 * Conventions shared by every entry point
 *   - All tensors are dense, contiguous, row-major, on the current CUDA
 *     device; every pointer argument is a DEVICE pointer unless the call says
 *     otherwise.  The caller owns every buffer; the library never allocates,
 *     frees or retains them.
 *   - Calls are asynchronous on `stream` (a cudaStream_t; NULL = legacy
 *     default stream) and never synchronise the host, except
 *     txl_sync_status().
 *   - Return value: TXL_OK (0) on success, a negative txl_status otherwise.
 *     Argument errors are detected on the host before anything is launched.
 *     No kernel traps or asserts: a device-side wait that runs past its
 *     time limit records TXL_ERR_DEVICE_TIMEOUT in a device status word,
 *     which txl_sync_status() reports and clears.
 *   - dtype: TXL_BF16 (inputs and output bf16, fp32 accumulation on the
 *     tensor cores) or TXL_F32 (inputs and output fp32, fp32 CUDA-core path).
 */
#ifndef TXL_ATTN_H
#define TXL_ATTN_H

#include <stddef.h>

#ifdef __cplusplus
extern "C" {
#endif

enum txl_dtype {
    TXL_F32 = 0,
    TXL_BF16 = 1
};

enum txl_status {
    TXL_OK = 0,
    TXL_ERR_INVALID_ARG = -1,    /* null pointer, B/H/L <= 0, M < 0, bad dtype */
    TXL_ERR_UNSUPPORTED = -2,    /* a size the library has no kernel for (see each call) */
    TXL_ERR_MISALIGNED = -3,     /* a base pointer is not 16-byte aligned */
    TXL_ERR_ALIAS = -4,          /* an output overlaps an input it must not overlap */
    TXL_ERR_LAUNCH = -5,         /* the CUDA launch itself failed */
    TXL_ERR_DEVICE_TIMEOUT = -6, /* a bounded device-side wait expired (reported by txl_sync_status) */
    TXL_ERR_WORKSPACE = -7,      /* workspace pointer null/misaligned or smaller than required */
    TXL_ERR_CUDA = -8,           /* a CUDA runtime/driver call failed (e.g. tensor-map encoding) */
    TXL_ERR_SCRATCH_LIMIT = -9,  /* the call needs more scratch than txl_attn_fwd_noalloc holds */
    TXL_ERR_OUT_OF_BOUNDS = -10  /* a bounds-checked build skipped an out-of-range access */
};

/*
 * Relative attention forward for one layer and one segment.
 *
 *   q      [B, H, L, d_h]      queries of the current segment only
 *   k, v   [B, H, M+L, d_h]    keys / values: rows 0..M-1 are the memory
 *                              (previous segment, stop-gradient), rows
 *                              M..M+L-1 the current segment
 *   r_k    [M+L, H, d_h]       projected sinusoid position table; row r holds
 *                              relative distance M+L-1-r (distance 0 last)
 *   u_bias [H, d_h]            global content bias u   (r_w_bias)
 *   v_bias [H, d_h]            global position bias v  (r_r_bias)
 *   out    [B, H, L, d_h]      result
 *
 * For query i in [0,L) and key j in [0,M+L):
 *   visible(i,j) <=> j <= M+i          (all memory keys, causal current keys)
 *   s(i,j) = scale * ((q_i+u).k_j + (q_i+v).r_k[M+L-1-(M+i-j)])
 *   out_i  = sum_j softmax_j(s(i,.)) v_j   over visible j only.
 * M = 0 is ordinary causal attention with a relative bias.
 *
 * bf16: d_h must be 64 (TXL_ERR_UNSUPPORTED otherwise); fp32: 1 <= d_h <= 256.
 * All pointers 16-byte aligned (TXL_ERR_MISALIGNED).  `out` must not overlap
 * any input (TXL_ERR_ALIAS).  This entry point allocates nothing and never
 * splits the keys of a query tile across CTAs; txl_attn_fwd_ws may.
 */
int txl_attn_fwd(const void* q, const void* k, const void* v, const void* r_k,
                 const void* u_bias, const void* v_bias,
                 int B, int H, int L, int M, int d_h, float scale, void* out,
                 int dtype, void* stream);

/*
 * txl_attn_fwd_ex: txl_attn_fwd with the same_length mask of
 * "Transformer-XL模型 核心源码阅读笔记" (MemTransformerLM._forward): every query
 * attends over the same number of keys.  With klen = M+L and mask_len = klen -
 * mem_len, query i additionally ignores keys j <= i - mask_shift_len, where
 * mask_shift_len = L - mask_len if mask_len > 0, else L; when M = mem_len each
 * query sees its mem_len most recent positions, itself included.  mem_len is
 * the configured memory length (M <= mem_len; M < mem_len while the memory is
 * still filling), else TXL_ERR_INVALID_ARG.  Key tiles that no query of a
 * 128-row query tile sees are skipped.  same_length = 0 is txl_attn_fwd.
 * Everything else (layouts, sizes, errors) as for txl_attn_fwd.
 */
int txl_attn_fwd_ex(const void* q, const void* k, const void* v, const void* r_k,
                    const void* u_bias, const void* v_bias, int B, int H, int L, int M, int d_h,
                    float scale, int same_length, int mem_len, void* out, int dtype, void* stream);

/*
 * Scratch bytes txl_attn_fwd_ws needs for these sizes (0 when the call runs
 * without splitting the keys).  Never negative; 0 also for invalid sizes.
 */
size_t txl_attn_workspace_bytes(int B, int H, int L, int M, int d_h, int dtype);

/*
 * txl_attn_fwd with caller-provided scratch: `workspace` (device, 256-byte
 * aligned, at least txl_attn_workspace_bytes(...) bytes) holds the partial
 * results of the split-key path, which the bf16 kernel takes when the call has
 * fewer (b, h, 128-row query tile) items than the GPU has SMs: each item's key
 * tiles are split over several CTAs, each writes its unnormalised partial O
 * and (max, sum) per row, and a combine pass merges them (the online-softmax
 * merge).  Nothing in the workspace needs to start at zero; every value read
 * is written earlier in the same call.  With a size of 0 the workspace is not
 * touched and may be null.  The library allocates nothing.
 * TXL_ERR_WORKSPACE if the buffer is missing, misaligned or too small;
 * TXL_ERR_ALIAS if it overlaps q, k, v or out.  Concurrent calls must use
 * distinct workspaces.
 */
int txl_attn_fwd_ws(const void* q, const void* k, const void* v, const void* r_k,
                    const void* u_bias, const void* v_bias,
                    int B, int H, int L, int M, int d_h, float scale, void* out,
                    int dtype, void* workspace, size_t ws_bytes, void* stream);

/*
 * Bytes of the static device scratch that txl_attn_fwd_noalloc uses.
 */
#define TXL_NOALLOC_SCRATCH_BYTES (16u << 20)

/*
 * txl_attn_fwd_ws without a caller workspace and without any allocation: the
 * split-key path (see txl_attn_fwd_ws) takes its partial results from one
 * file-scope static device buffer of TXL_NOALLOC_SCRATCH_BYTES (16 MiB) per
 * device.  The library looks its device address up (cudaGetSymbolAddress)
 * on every call that is not inside a stream capture and keeps the last
 * address per device for calls made during a capture.  The pages have no
 * counterpart of this entry point: it exists for callers that cannot hand
 * out a workspace (for example a fixed launch sequence).
 *
 *   - Same arguments, results and errors as txl_attn_fwd_ws; a call whose
 *     txl_attn_workspace_bytes(...) exceeds TXL_NOALLOC_SCRATCH_BYTES returns
 *     TXL_ERR_SCRATCH_LIMIT and launches nothing.
 *   - Nothing in the scratch needs to start at zero: every value read is
 *     written earlier in the same call.
 *   - The first call on each device that needs scratch must not be inside a
 *     stream capture (there is no cached address yet: TXL_ERR_CUDA).  After
 *     cudaDeviceReset (or any teardown of the device's context) the module is
 *     loaded again at a new address: make one call outside a capture before
 *     capturing again, or a capture would launch on the stale address.
 *   - Calls that overlap in time on one device (different streams, or
 *     threads) share the buffer and race: order them, e.g. on one stream.
 *   - Calls that need no scratch (txl_attn_workspace_bytes(...) == 0) do not
 *     touch it.
 */
int txl_attn_fwd_noalloc(const void* q, const void* k, const void* v, const void* r_k,
                         const void* u_bias, const void* v_bias,
                         int B, int H, int L, int M, int d_h, float scale, void* out,
                         int dtype, void* stream);

/*
 * Projections feeding txl_attn_fwd, bf16 in and out, fp32 accumulation, on
 * the tensor cores ("Transformer-XL模型 核心源码阅读笔记",
 * RelPartialLearnableMultiHeadAttn.forward: qkv_net over the concatenation of
 * memory and current hidden states, r_net over the position embedding).
 *
 * txl_qkv_proj:
 *   h     [B, L, d]     current hidden states (layer input), d = H * d_h
 *   mem   [B, M, d]     the layer's memory (may be null when M = 0)
 *   w_qkv [3d, d]       stacked weights, rows [0,d) W_q, [d,2d) W_k, [2d,3d) W_v
 *                       (output = input x W^T, the nn.Linear layout)
 *   q     [B, H, L, d_h]      q = h W_q^T, split into heads
 *   k, v  [B, H, M+L, d_h]    rows 0..M-1 from mem, rows M.. from h, split into
 *                             heads (no [mem; h] concatenation is formed)
 * txl_r_proj:
 *   emb   [K, d]   position embedding rows (the sinusoid of distances K-1..0)
 *   w_r   [d, d]   W_r (nn.Linear layout)
 *   r_k   [K, H, d_h] = emb W_r^T (row-major [K, d])
 *
 * Supported sizes (TXL_ERR_UNSUPPORTED otherwise): d_h = 64, H a multiple of
 * 4, L, M and K multiples of 128 (M may be 0).  Pointers 16-byte aligned
 * (TXL_ERR_MISALIGNED); outputs must not overlap inputs (TXL_ERR_ALIAS).
 * Asynchronous on `stream`; nothing is allocated.  Bounded device waits
 * report TXL_ERR_DEVICE_TIMEOUT through txl_sync_status.
 */
int txl_qkv_proj(const void* h, const void* mem, const void* w_qkv, int B, int L, int M, int H,
                 int d_h, void* q, void* k, void* v, void* stream);

/*
 * txl_qkvr_proj: one layer's projections in one launch -- txl_qkv_proj_ring's
 * q, k, v (same arguments and contract) and txl_r_proj's r_k = emb W_r^T over
 * K = M + L rows of the position embedding emb [M+L, d] (same contract) --
 * dealt from one tile list, so the small position projection rides in the
 * q/k/v launch instead of occupying a few SMs of a launch of its own
 * ("Transformer-XL模型 核心源码阅读笔记", RelPartialLearnableMultiHeadAttn.forward:
 * w_heads = qkv_net(cat), r_head_k = r_net(r)).  r_k must not overlap any
 * other argument (TXL_ERR_ALIAS).
 */
int txl_qkvr_proj(const void* h, int h_layout, const void* mem, int mem_layout, int mem_start,
                  const void* w_qkv, const void* emb, const void* w_r, int B, int L, int M, int H,
                  int d_h, void* q, void* k, void* v, void* r_k, void* stream);

/*
 * txl_qkv_proj_ex: txl_qkv_proj with the layout of h and mem chosen per
 * argument.  TXL_LAYOUT_ROWS: [B, T, d] as above.  TXL_LAYOUT_HEADS:
 * [B, H, T, d_h], the layout txl_attn_fwd writes its output in, so a stack of
 * layers feeds one layer's attention output (and the memory rolled from it)
 * straight into the next layer's projections; row t of head h is columns
 * h*d_h .. h*d_h+d_h-1 of the row-major view.  Other layouts return
 * TXL_ERR_INVALID_ARG; sizes, alignment and aliasing as for txl_qkv_proj.
 */
#define TXL_LAYOUT_ROWS 0
#define TXL_LAYOUT_HEADS 1
int txl_qkv_proj_ex(const void* h, int h_layout, const void* mem, int mem_layout,
                    const void* w_qkv, int B, int L, int M, int H, int d_h, void* q, void* k,
                    void* v, void* stream);

/*
 * Ring-buffer memory (an alternative to the Tail_M copy): a memory
 * of M rows whose logical row t is stored at row (start + t) mod M.
 *
 * txl_qkv_proj_ring: txl_qkv_proj_ex reading mem as a ring starting at
 *   mem_start (0 <= mem_start < M, a multiple of 128: every 128-row tile of
 *   the ring is then contiguous; TXL_ERR_UNSUPPORTED otherwise).  Same result
 *   as txl_qkv_proj_ex on the logical (unrotated) memory.
 * txl_mem_ring_push: the ring counterpart of txl_mem_update.  For L < M the
 *   L rows of hids [B, L, d] overwrite the ring's L oldest rows (hids row r
 *   at ring row (start + r) mod M) and *new_start = (start + L) mod M: L rows
 *   are written instead of M moved.  For L >= M the ring is refilled with the
 *   newest M rows and *new_start = 0.  The logical memory afterwards equals
 *   txl_mem_update's result.  Arguments and errors as txl_mem_update, plus
 *   start in [0, M) (TXL_ERR_INVALID_ARG) and new_start a host pointer.
 */
int txl_qkv_proj_ring(const void* h, int h_layout, const void* mem, int mem_layout, int mem_start,
                      const void* w_qkv, int B, int L, int M, int H, int d_h, void* q, void* k,
                      void* v, void* stream);
int txl_mem_ring_push(void* ring, const void* hids, int B, int L, int M, int d, int start,
                      int* new_start, int dtype, void* stream);
int txl_r_proj(const void* emb, const void* w_r, int K, int H, int d_h, void* r_k, void* stream);

/*
 * txl_attn_bwd: gradients of sum(out * dout) for the attention of
 * txl_attn_fwd / txl_attn_fwd_ex (same inputs, same mask options), for
 * training with a stop-gradient memory ("Transformer-XL" notes: the memory is
 * a constant input of the segment; its rows' dk, dv are returned and the
 * caller drops them).  Inputs in dtype (TXL_BF16 or TXL_F32), d_h <= 256;
 * gradients in fp32, device buffers the call overwrites:
 *   dq [B, H, L, d_h], dk, dv [B, H, M+L, d_h], dr [M+L, H, d_h] (summed
 *   over the batch), du, dvb [H, d_h] (summed over batch and query rows).
 * P is recomputed from q, k, r_k, u, v (no forward state is kept).  CUDA-core
 * arithmetic with fp32 atomics for the summed gradients: a correctness path
 * whose summation order is not fixed.  Errors as txl_attn_fwd; gradient
 * buffers must not overlap the inputs or each other (TXL_ERR_ALIAS).
 */
int txl_attn_bwd(const void* q, const void* k, const void* v, const void* r_k, const void* u_bias,
                 const void* v_bias, const void* dout, int B, int H, int L, int M, int d_h, float scale,
                 int same_length, int mem_len, float* dq, float* dk, float* dv, float* dr, float* du,
                 float* dvb, int dtype, void* stream);

/*
 * txl_attn_bwd_ws: the gradients of txl_attn_bwd (same arguments, layouts,
 * outputs and errors) on the tensor cores, for bf16 inputs with d_h = 64 and
 * the plain causal mask with memory (same_length = 0).  Any other call needs
 * no workspace and runs txl_attn_bwd.
 *
 * The pass follows the derivative of the attention of "Transformer-XL模型 核心
 * 源码阅读笔记", section "Build the model" (RelPartialLearnableMultiHeadAttn.
 * forward: AC + shifted BD, masked softmax, P V) with the memory a constant
 * input ("Transformer-XL" notes, section "Segment-Level Recurrence"), in four
 * launches on `stream`: the forward kernel of txl_attn_fwd_lse writes the
 * output and each query row's log2-sum-exp into the workspace; a small
 * kernel computes D = dout . out per row, writes (q+u) and (q+v) scaled by
 * scale * log2 e in bf16 and zeroes dr, du, dvb; a query-major pass recomputes P, dP and dS
 * per 128-row query tile and writes dq and accumulates dr, du, dvb; a
 * key-major pass recomputes them per 128-key tile and writes dk, dv (it may
 * start on the SMs the query-major pass leaves; the call's last launch
 * completes after both).  dr, du and dvb are accumulated with fp32 atomics
 * (summation order not fixed); dq, dk and dv are written once per element.  Contractions in bf16 with fp32
 * accumulation: P and dS are rounded to bf16 before their products.
 *
 * workspace: device memory owned by the caller, 256-byte aligned, at least
 * txl_attn_bwd_workspace_bytes(...) bytes (0 when the call runs
 * txl_attn_bwd); it must not overlap an input or a gradient (TXL_ERR_ALIAS).
 * TXL_ERR_WORKSPACE when it is null, misaligned or too small.
 */
size_t txl_attn_bwd_workspace_bytes(int B, int H, int L, int M, int d_h, int dtype, int same_length);

/*
 * txl_attn_fwd_lse: txl_attn_fwd (bf16, d_h = 64) that also writes each query
 * row's log2-sum-exp of its scores, lse [B, H, L] fp32 (log2 units: with s_ij
 * the score of "Transformer-XL模型 核心源码阅读笔记", RelPartialLearnableMultiHead
 * Attn.forward, P_ij = 2^(s_ij log2 e - lse_i)), the state a backward pass
 * needs besides `out`.  lse: device memory, 16-byte aligned, not overlapping
 * any other argument (TXL_ERR_ALIAS); TXL_ERR_UNSUPPORTED for TXL_F32.
 *
 * txl_attn_bwd_saved: the gradients of txl_attn_bwd_ws from the forward's
 * saved state instead of a recomputed forward: out [B, H, L, d_h] (bf16) and
 * lse as written by txl_attn_fwd_lse for the same inputs, D = dout . out per
 * row.  bf16, d_h = 64, no same_length (TXL_ERR_UNSUPPORTED otherwise); the
 * workspace of txl_attn_bwd_workspace_bytes(..., same_length = 0); the
 * gradients must overlap neither the inputs, out, lse nor the workspace.
 */
int txl_attn_fwd_lse(const void* q, const void* k, const void* v, const void* r_k, const void* u_bias,
                     const void* v_bias, int B, int H, int L, int M, int d_h, float scale, void* out, float* lse,
                     int dtype, void* stream);
int txl_attn_bwd_saved(const void* q, const void* k, const void* v, const void* r_k, const void* u_bias,
                       const void* v_bias, const void* out, const float* lse, const void* dout, int B, int H, int L,
                       int M, int d_h, float scale, float* dq, float* dk, float* dv, float* dr, float* du,
                       float* dvb, int dtype, void* workspace, size_t ws_bytes, void* stream);
int txl_attn_bwd_ws(const void* q, const void* k, const void* v, const void* r_k, const void* u_bias,
                    const void* v_bias, const void* dout, int B, int H, int L, int M, int d_h, float scale,
                    int same_length, int mem_len, float* dq, float* dk, float* dv, float* dr, float* du,
                    float* dvb, int dtype, void* workspace, size_t ws_bytes, void* stream);

/*
 * The rest of a decoder layer ("Transformer-XL模型 核心源码阅读笔记":
 * RelPartialLearnableMultiHeadAttn.forward after the attention, PositionwiseFF,
 * RelPartialLearnableDecoderLayer), bf16 with fp32 accumulation:
 *
 * txl_linear: out [B, T, N] = relu?(x W^T + bias) + resid (nn.Linear layout,
 *   w [N, K]); x [B, T, K] (TXL_LAYOUT_ROWS) or [B, K/64, T, 64]
 *   (TXL_LAYOUT_HEADS: an attention output read directly as attn_vec, the
 *   o_net input); bias [N] and resid [B, T, N] may be null.  Covers o_net
 *   (no bias), the two CoreNet layers (bias, ReLU on the first) and, in the
 *   pre-norm layer, their residual adds.  T a multiple of 128, K of 64, N of
 *   256 (TXL_ERR_UNSUPPORTED); out may be resid itself, no other overlap
 *   (TXL_ERR_ALIAS).
 * txl_layer_norm: out [rows, d] = LayerNorm(x + y) * gamma + beta over each
 *   row (y may be null; nn.LayerNorm: biased variance, eps inside the square
 *   root).  d in {256, 512, 768, 1024, 1536, 2048}; out may be x or y.
 *
 * All pointers are device pointers, 16-byte aligned (TXL_ERR_MISALIGNED).
 * Asynchronous on `stream`; nothing is allocated.
 */
int txl_linear(const void* x, int x_layout, int B, int T, int K, const void* w, int N,
               const void* bias, const void* resid, int relu, void* out, void* stream);
int txl_layer_norm(const void* x, const void* y, const void* gamma, const void* beta, long long rows,
                   int d, float eps, void* out, void* stream);

/*
 * LayerNorm for training: txl_layer_norm's forward that also keeps each row's
 * statistics, and its gradients.  Any row length 1 <= d <= 16384 and
 * 0 <= rows < 2^31 (TXL_ERR_UNSUPPORTED beyond); dtype TXL_BF16 or TXL_F32 for
 * x, y, gamma, beta, out, dout, dres and dx; statistics and parameter gradients
 * fp32.
 *
 * txl_layer_norm_fwd: with z = x + y (y may be null),
 *   mean[r] = sum z / d, rstd[r] = (sum (z - mean)^2 / d + eps)^(-1/2),
 *   out = (z - mean) rstd gamma + beta.  mean, rstd: [rows].
 * txl_layer_norm_bwd: from dout, the gradient of out, and the forward's inputs
 *   and statistics: dx [rows, d], the gradient of x and of y alike, plus dres
 *   (may be null: the gradient that reaches z along a residual path);
 *   dgamma, dbeta [d], summed over the rows in a fixed order (the same inputs
 *   give the same bits; zeros when rows = 0).
 *
 * All pointers 16-byte aligned (TXL_ERR_MISALIGNED; with rows = 0 only those of
 * dgamma and dbeta are looked at).  Outputs overlap neither inputs nor each other
 * (TXL_ERR_ALIAS).  workspace: device memory, 256-byte aligned, at least
 * txl_layer_norm_bwd_workspace_bytes(...) bytes (TXL_ERR_WORKSPACE), overlapping
 * no other argument (TXL_ERR_ALIAS); concurrent calls use distinct ones.  0 bytes:
 * none needed, not touched.
 */
int txl_layer_norm_fwd(const void* x, const void* y, const void* gamma, const void* beta, long long rows,
                       int d, float eps, void* out, float* mean, float* rstd, int dtype, void* stream);
size_t txl_layer_norm_bwd_workspace_bytes(long long rows, int d, int dtype);
int txl_layer_norm_bwd(const void* dout, const void* x, const void* y, const void* gamma, const float* mean,
                       const float* rstd, const void* dres, long long rows, int d, void* dx, float* dgamma,
                       float* dbeta, int dtype, void* workspace, size_t ws_bytes, void* stream);

/*
 * txl_linear_bwd: gradients of txl_linear's out = x W^T + bias, bf16 with fp32
 * accumulation on the tensor cores.  dy [B, T, N] is the gradient of out, x
 * [B, T, K] (TXL_LAYOUT_ROWS) or [B, K/64, T, 64] (TXL_LAYOUT_HEADS), w [N, K]:
 *   dx = dy W, bf16 in x's layout (an attention output's gradient comes out in
 *        the layout txl_attn_bwd takes as dout); with relu_in, where x is the
 *        output of a ReLU, the gradient of the ReLU's input: exactly 0 where x
 *        is not above 0 (a NaN among them), whatever dy and W hold
 *   dw = dy^T x, fp32 [N, K];  db = sum of dy over the rows, fp32 [N]
 * dx may be null, db may be null, dw may be null if db is (TXL_ERR_INVALID_ARG:
 * db without dw, or nothing asked for).  Sums over rows are added in a fixed
 * order: the same inputs give the same bits.
 *
 * Any B, T >= 1; K and N multiples of 8, K of 64 in the heads layout
 * (TXL_ERR_UNSUPPORTED; as are B T above 2^28, K or N above 2^20 and more than
 * 2^30 output tiles of 128 x 128).  Pointers 16-byte aligned
 * (TXL_ERR_MISALIGNED); outputs overlap neither inputs nor each other
 * (TXL_ERR_ALIAS).  workspace as for txl_layer_norm_bwd, of
 * txl_linear_bwd_workspace_bytes(...) bytes.
 */
size_t txl_linear_bwd_workspace_bytes(int x_layout, int B, int T, int K, int N, int want_dx, int want_dw,
                                      int want_db);
int txl_linear_bwd(const void* dy, const void* x, int x_layout, int B, int T, int K, const void* w, int N,
                   int relu_in, void* dx, float* dw, float* db, void* workspace, size_t ws_bytes, void* stream);

/*
 * txl_token_logprobs: from logits x of `rows` rows of V (row r at logits + r ld, in
 * elements, ld >= V) and a token per row (int64; negative: the row has none),
 *   lse[r] = ln sum e^x,  logprob[r] = x_token - lse (0 without a token, NaN for a
 *   token >= V),  entropy[r] = -sum p ln p with p = e^(x - lse);
 *   with 0 < top <= min(V, 32): top_index[r, i], the indexes of the `top` largest
 *   logits in their order, of equal ones the lower index first (NaN above all others),
 *   and top_logprob[r, i] = x - lse.  top = 0: both null.
 * fp32 arithmetic, each logit read once; logits of dtype TXL_BF16 or TXL_F32, results
 * fp32, indexes int64.  A row of nothing but -inf: lse, logprob and top_logprob -inf,
 * entropy 0.  A row that holds a NaN or +inf: lse, logprob (of a token), entropy and
 * top_logprob NaN.
 * txl_token_logprobs_bwd: with the gradients of logprob, lse and entropy (fp32 [rows],
 * each may be null: zeros, but not all three),
 *   dx_j = dlogprob (delta_j,token - p_j) + dlse p_j - dentropy p_j ((x_j - lse) + entropy),
 * dlogprob taken as 0 where there is no token.  lse and entropy (null without dentropy)
 * as the forward call gave them (p carries lse's rounding, 2^-24 of it).  dlogits (rows ldd elements apart) may be logits with
 * the same distance of rows: the gradient then takes their place.  A row whose gradients
 * are all 0 gets zeros whatever its logits hold, as does a row of nothing but -inf (lse
 * -inf); dlogprob other than 0 at a token >= V makes any other row NaN.  What lies between the rows
 * is left as it was.
 *
 * 0 <= rows < 2^31, 1 <= V <= 2^24, rows * max(ld, ldd) <= 2^40 (TXL_ERR_UNSUPPORTED
 * beyond, as for top > 32; top > V is TXL_ERR_INVALID_ARG).  Pointers need the alignment
 * of their elements (TXL_ERR_MISALIGNED).  What is written overlaps nothing else
 * (TXL_ERR_ALIAS), but for dlogits as said.
 */
int txl_token_logprobs(const void* logits, long long ld, const long long* tokens, long long rows, int V, int top,
                       float* logprob, float* lse, float* entropy, long long* top_index, float* top_logprob,
                       int dtype, void* stream);
int txl_token_logprobs_bwd(const void* logits, long long ld, const long long* tokens, const float* lse,
                           const float* entropy, const float* dlogprob, const float* dlse, const float* dentropy,
                           long long rows, int V, void* dlogits, long long ldd, int dtype, void* stream);

/*
 * txl_linear_logprobs: txl_token_logprobs of the logits z = x W^T + bias without the
 * logits: x [rows, K], w [V, K] and bias [V] (may be null) bf16, products on the tensor
 * cores with fp32 accumulation (which cuts off some 2^-26 of the sum per 16 elements of K), z
 * never rounded to fewer bits; the row statistics lse,
 * logprob and entropy (fp32 [rows]) and their special cases are those of
 * txl_token_logprobs (a bias of -inf masks a column).  For scoring; the gradient goes over
 * txl_linear's logits and txl_token_logprobs_bwd.  The same inputs give the same bits.
 *
 * 0 <= rows <= 2^28, K a multiple of 8 up to 2^20, 1 <= V <= 2^24, rows * V <= 2^40
 * (TXL_ERR_UNSUPPORTED beyond).  x and w 16-byte aligned, the others to their elements
 * (TXL_ERR_MISALIGNED); outputs overlap neither inputs nor each other (TXL_ERR_ALIAS).
 * workspace as for txl_layer_norm_bwd, of txl_linear_logprobs_workspace_bytes(...) bytes.
 */
size_t txl_linear_logprobs_workspace_bytes(long long rows, int K, int V);
int txl_linear_logprobs(const void* x, const void* w, const void* bias, const long long* tokens, long long rows, int K,
                        int V, float* logprob, float* lse, float* entropy, void* workspace, size_t ws_bytes,
                        void* stream);

/*
 * txl_adamw_step: one AdamW step over n_tensors tensors.  `tensors` is an array
 * in HOST memory, read during the call; tensor i has n elements (0: skipped),
 * a parameter, a gradient and a weight decay of its own.  With g the gradient
 * times the clip factor and t the step's number (the first step is 1),
 *   m = beta1 m + (1 - beta1) g,   v = beta2 v + (1 - beta2) g^2,
 *   p = p - lr (weight_decay p + m / (1 - beta1^t) / (sqrt(v / (1 - beta2^t)) + eps)),
 * in fp32.  param_dtype TXL_F32: p is the parameter (master null).  TXL_BF16: p
 * is the fp32 copy in `master`, and the parameter is written as its rounding.
 * grad_dtype: TXL_F32 or TXL_BF16.
 *
 * Flat state: tensor i's state starts at element 256 * (sum over j < i of
 * ceil(n_j / 256)) of master, exp_avg and exp_avg_sq; the elements between a
 * tensor's end and the next start are the library's (start them at zero).
 * txl_adamw_state_elements gives the length (-1: invalid or above 2^38).
 *   state_bits 32: exp_avg, exp_avg_sq hold m and v in fp32 (the scales null).
 *   state_bits 8: exp_avg holds e4m3 codes of m, exp_avg_sq of sqrt(v), each
 *     block of 256 elements with one fp32 scale in exp_avg_scale and
 *     exp_avg_sq_scale (value = code * scale); codes are rounded up or down at
 *     random, the mean kept, from `seed`, the step's number and the element's index.
 * All of it starts at zero, master at the parameters' values.
 *
 * steps (device): number of steps done, advanced by the call.  lr (device): the
 * learning rate.  Both are read when the step runs, so a captured step can be
 * replayed and lr changed between replays.  max_norm > 0: gradients are scaled
 * by min(1, max_norm / norm) with norm the 2-norm of all gradients (their sum of
 * squares must stay in fp32's range), written to grad_norm (device, may be
 * null); a norm that is not finite leaves parameters, states and steps as
 * they were.  max_norm = 0: no clipping, grad_norm untouched.
 *
 * Parameters, gradients and flat buffers 16-byte aligned, steps 8-byte
 * (TXL_ERR_MISALIGNED).  What is written overlaps nothing else
 * (TXL_ERR_ALIAS); gradients may share memory.  workspace as for
 * txl_layer_norm_bwd, of txl_adamw_workspace_bytes(...) bytes.  betas in
 * [0, 1), eps 0 or at least 2^-126, max_norm >= 0, both finite
 * (TXL_ERR_INVALID_ARG).
 */
typedef struct txl_adamw_tensor {
    void* param;
    const void* grad;
    long long n;
    float weight_decay;
    int reserved; /* 0 */
} txl_adamw_tensor;
long long txl_adamw_state_elements(const txl_adamw_tensor* tensors, int n_tensors);
size_t txl_adamw_workspace_bytes(const txl_adamw_tensor* tensors, int n_tensors);
int txl_adamw_step(const txl_adamw_tensor* tensors, int n_tensors, int param_dtype, int grad_dtype,
                   int state_bits, float* master, void* exp_avg, float* exp_avg_scale, void* exp_avg_sq,
                   float* exp_avg_sq_scale, long long* steps, const float* lr, double beta1, double beta2,
                   double eps, double max_norm, unsigned seed, float* grad_norm, void* workspace,
                   size_t ws_bytes, void* stream);

/*
 * txl_grad_norm: the 2-norm of n_tensors tensors together (norm, device fp32 [1]), that
 * of each one (norms, fp32 [n_tensors], may be null) and, with max_norm > 0, their scaling
 * in place by max_norm / norm where norm > max_norm.  `tensors` is an array in HOST memory,
 * read during the call; tensor i has n elements (0: its norm is 0) of type dtype (TXL_F32
 * or TXL_BF16, which may differ from tensor to tensor).  Products and sums in fp32 over
 * values scaled by powers of two where their squares would leave its range, added in a
 * fixed order (the same inputs give the same bits).  A scaled value is its product with
 * max_norm / norm in fp32, whatever the quotient's size, rounded to its type.
 * norm and norms are those before the scaling.  A norm that is not finite in fp32 leaves
 * the tensors as they were, as does one of at most max_norm.  max_norm = 0: nothing is
 * scaled, and tensors may overlap each other.
 *
 * Tensors 16-byte aligned, norm and norms 4-byte (TXL_ERR_MISALIGNED); what is written
 * overlaps nothing else (TXL_ERR_ALIAS).  At most 2^38 elements per tensor, 2^40 in all
 * (TXL_ERR_UNSUPPORTED).  workspace as for txl_layer_norm_bwd, of
 * txl_grad_norm_workspace_bytes(...) bytes.  max_norm >= 0 and finite, and 0 or at least
 * 2^-126 (TXL_ERR_INVALID_ARG).
 */
typedef struct txl_grad_tensor {
    void* grad;
    long long n;
    int dtype;
    int reserved; /* 0 */
} txl_grad_tensor;
size_t txl_grad_norm_workspace_bytes(const txl_grad_tensor* tensors, int n_tensors);
int txl_grad_norm(const txl_grad_tensor* tensors, int n_tensors, double max_norm, float* norm, float* norms,
                  void* workspace, size_t ws_bytes, void* stream);

/*
 * Tail_M memory roll, in place ("Transformer-XL" notes, section
 * "Segment-Level Recurrence": M_{tau+1} = Tail_M([M_tau; H_tau]); source notes
 * MemTransformerLM._update_mems with ext_len = 0 and a full memory).
 *
 *   mems [B, M, d]   memory of one layer, overwritten with the newest M rows
 *                    of the sequence-axis concatenation [mems; hids]
 *   hids [B, L, d]   hidden states of the current segment (layer input)
 *
 * When L >= M the result is hids[:, L-M:]; when L < M it is
 * [mems[:, L:]; hids].  Bit-exact copy for any element type; dtype only
 * fixes the element size (TXL_BF16: 2 bytes, TXL_F32: 4 bytes).  M = 0 is a
 * no-op.  `mems` must not overlap `hids` (TXL_ERR_ALIAS).  Any alignment is
 * accepted; 16-byte aligned rows of a multiple of 16 bytes take the
 * vectorised path.
 */
int txl_mem_update(void* mems, const void* hids, int B, int L, int M, int d,
                   int dtype, void* stream);

/*
 * txl_mem_update_ext: txl_mem_update keeping the last ext_len rows of hids
 * out of the memory ("Transformer-XL模型 核心源码阅读笔记",
 * MemTransformerLM._update_mems: the cached span of [mems; hids] ends ext_len
 * rows before its end, those rows serving as extended context of the next
 * segment instead).  The result is the Tail_M roll with hids[:, :L-ext_len]
 * (an unchanged memory when ext_len >= L); hids is still [B, L, d].
 * ext_len < 0 returns TXL_ERR_INVALID_ARG.  ext_len = 0 is txl_mem_update.
 *
 * txl_mem_reset: mems [B, rows, d] (any layout whose batch rows are
 * contiguous, e.g. [B, H, M, d_h] with rows = H*M, d = d_h); every batch row
 * b with flags[b] != 0 (flags: B bytes in device memory) is set to zero bits
 * ("Transformer-XL" notes, section "Batched Streams": a row whose stream
 * enters a new document gets an empty memory; the flag is per row, not per
 * batch).  Other rows are untouched.  Asynchronous on `stream`.
 */
int txl_mem_update_ext(void* mems, const void* hids, int B, int L, int M, int d, int ext_len,
                       int dtype, void* stream);
int txl_mem_reset(void* mems, const void* flags, int B, int rows, int d, int dtype, void* stream);

/*
 * Waits for `stream`, then reports and clears the device status word:
 * TXL_ERR_DEVICE_TIMEOUT if a kernel gave up on a bounded wait since the last
 * call, TXL_ERR_CUDA if the stream reports a CUDA error, TXL_OK otherwise.
 */
int txl_sync_status(void* stream);

/*
 * Bounds-checked builds (the library compiled with -DTXL_CHECKED, shipped as
 * libtxl_checked.so beside libtxl.so): every kernel routes its computed
 * global-memory indexes and shared-memory addresses through a check; an
 * access outside its buffer is skipped, never performed, and the first such
 * access per source file is recorded (no trap, no fault).  TMA copies are
 * bounded by their tensor maps in hardware and are not re-checked.
 * txl_bounds_status synchronises the device, then returns TXL_OK when no
 * access was out of range since the last call, or TXL_ERR_OUT_OF_BOUNDS with
 * the first record in *first: bit 63 set, bits 40..62 the check site (the
 * hundreds digit names the source file), bits 0..39 the offending index
 * (mod 2^40).  The records are cleared.  TXL_ERR_UNSUPPORTED from a library
 * built without checks.  A debugging aid, not for production launches.
 */
int txl_bounds_status(unsigned long long* first);

/* Human-readable name of a txl_status value (static string). */
const char* txl_status_string(int status);

/* ABI version: (major << 16) | minor. */
int txl_version(void);

/*
 * Test hook for the failure-detection path.  kind = 1 makes the NEXT bf16
 * attention launch made by the calling host thread withhold one internal
 * completion signal, so its waiting warps hit their time limit, record
 * TXL_ERR_DEVICE_TIMEOUT and exit cleanly (the GPU context stays usable).
 * kind = 0 clears it.  The hook is per host thread (launches from other
 * threads never consume it) and disarms itself after one launch.  Not for
 * production use.
 */
int txl_debug_inject(int kind);

#ifdef __cplusplus
}
#endif

#endif /* TXL_ATTN_H */
