/*
 * txl.h -- C ABI of libtxl: Transformer-XL segment-level relative multi-head
 * attention and the per-layer memory rollover on one GB300 GPU (sm_103a), and
 * what a training step needs around them (projections, the embedding, layer
 * norm, the output layer's losses, the optimiser step).
 *
 * Every pointer argument named "device" is a CUDA device pointer owned by the
 * caller; the library never frees caller memory and keeps no pointer to it
 * after the call returns.  Calls are asynchronous on the given stream (a
 * cudaStream_t passed as void*, NULL = the legacy default stream): the library
 * never synchronises the device inside a compute call.  Argument errors are
 * detected on the host before any launch and nothing is launched then.
 *
 * Notation (Transformer-XL, Section 3.2 and Appendix B): B batch, H heads,
 * D head dimension, L segment length, M memory length, T = M + L the extended
 * context [memory (M rows, oldest first); current segment (L rows)].
 * Row-major layouts, D innermost:
 *     q, out : [L][B][H][D]      k, v : [T][B][H][D]
 *     r      : [T][H][D]  -- row t holds W_kR R_{T-1-t} (the reversed table Q
 *                            of Appendix B); shared by every sequence
 *     u_bias, v_bias : [H][D] float32 (the global biases u and v of
 *                            Section 3.3, one vector per head)
 */
#ifndef TXL_H_
#define TXL_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    TXL_OK = 0,
    TXL_ERR_INVALID = 1,     /* bad argument: NULL, negative size, misaligned, overlap */
    TXL_ERR_UNSUPPORTED = 2, /* valid but not built: d_head too large, unknown dtype */
    TXL_ERR_CUDA = 3,        /* a CUDA runtime/driver call failed (also: no GPU) */
    TXL_ERR_TIMEOUT = 4      /* a bounded in-kernel wait gave up (see txl_check) */
} txl_status;

typedef enum {
    TXL_F32 = 0,             /* float32 in, float32 accumulate, float32 out */
    TXL_BF16 = 1             /* bfloat16 in, float32 accumulate, bfloat16 out */
} txl_dtype;

/*
 * txl_rel_attn_fwd -- one layer of relative attention (Transformer-XL,
 * Section 3.3, the computing procedure; Appendix B, the linear-cost route).
 *
 * For every b < batch, h < heads and query position i < seg_len:
 *     s_ij = ((q_i + u).k_j + (q_i + v).r[T-1-(M+i-j)]) / sqrt(d_head)
 *                                          for key j = 0 .. M+i (causal)
 *     out_i = sum_j softmax_j(s_ij) v_j
 * where j indexes the extended context [memory; segment] and M+i-j is the
 * relative distance of the pair.
 *
 * q, k, v, r, out : device, dtype elements, layouts above; base addresses
 *                   16-byte aligned; out must not overlap any input.
 * u_bias, v_bias  : device, float32 [heads][d_head], 4-byte aligned; either
 *                   may be NULL, which drops its term: with both NULL the
 *                   score is terms (a) + (b) only, the form of Shaw et al.
 *                   the paper contrasts in Section 3.3 (r may then be any
 *                   table, e.g. a learned R^ in place of W_kR R).  NULL needs
 *                   heads*d_head <= 65536 (else TXL_ERR_UNSUPPORTED).
 * batch, heads, seg_len >= 0 (0 => nothing to do, TXL_OK, pointers unused);
 * mem_len >= 0; 1 <= d_head <= 128 for TXL_F32, 1 <= d_head <= 64 for
 * TXL_BF16 (larger: TXL_ERR_UNSUPPORTED).
 * stream          : cudaStream_t as void*.
 * Returns TXL_OK once the work is enqueued.  TXL_ERR_INVALID /
 * TXL_ERR_UNSUPPORTED before any launch; TXL_ERR_CUDA if a launch fails.
 * Long memories (few query tiles, many keys) split the keys across CTAs; the
 * partial results then live in a library-owned device scratch buffer.  bf16
 * heads with d_head != 64 also use it: q, k, v, r and the biases are copied
 * into 64-wide zero-padded vectors there (rows the TMA unit can read), and
 * the output's d_head columns are copied back.  There is one such buffer per
 * (device, stream handle): calls on different streams never share one and may
 * run concurrently.  A buffer is allocated on first need and grown in stream
 * order (cudaFreeAsync / cudaMallocAsync on that stream, no host-side wait),
 * so the first call of a larger size on a stream must not be made during
 * stream capture (it returns TXL_ERR_UNSUPPORTED there); later captured calls
 * reuse the buffer.  Buffers are keyed by the stream handle's value: destroy a
 * stream only after its calls have finished if a new stream may reuse the
 * handle.  At most 256 (device, stream) pairs are served (then
 * TXL_ERR_UNSUPPORTED); txl_shutdown() releases the current device's.
 */
txl_status txl_rel_attn_fwd(const void *q, const void *k, const void *v, const void *r,
                            const float *u_bias, const float *v_bias,
                            int batch, int mem_len, int seg_len, int heads, int d_head,
                            txl_dtype dtype, void *out, void *stream);

/*
 * txl_rel_attn_fwd_plan -- how txl_rel_attn_fwd runs a call of this shape:
 * the number of key-range splits (the keys of each query block divided over
 * that many CTAs, merged by a combine launch) and the number of kernel
 * launches it makes, for 16-byte aligned operands.  No GPU work; the split
 * choice is the one the call itself makes on the current device (a cost
 * model of the kernel's schedule, measured on GB300).
 *
 * splits, launches : host int outputs (NULL => TXL_ERR_INVALID).  A call with
 * nothing to do reports 1 split and 0 launches.  Same dtype and d_head limits
 * as txl_rel_attn_fwd.
 */
txl_status txl_rel_attn_fwd_plan(int batch, int mem_len, int seg_len, int heads, int d_head, txl_dtype dtype,
                                 int *splits, int *launches);

/*
 * txl_rel_attn_fwd_lse -- txl_rel_attn_fwd that also stores, per query row,
 * the natural log of the softmax denominator (the log-sum-exp of the row's
 * visible scaled scores s_ij above):
 *     lse[(b*heads + h)*seg_len + i] = log sum_{j <= M+i} exp(s_ij)
 * so that P_ij = exp(s_ij - lse) recovers the weights without a second pass
 * over the keys.  txl_rel_attn_bwd takes out and lse back to skip its own
 * forward.
 *
 * lse : device float32 [batch][heads][seg_len], 4-byte aligned, must not
 *       overlap out or any input; required (NULL => TXL_ERR_INVALID unless
 *       there is nothing to do).
 * Only TXL_BF16 (else TXL_ERR_UNSUPPORTED).  Everything else, including the
 * result in out, as txl_rel_attn_fwd.
 */
txl_status txl_rel_attn_fwd_lse(const void *q, const void *k, const void *v, const void *r,
                                const float *u_bias, const float *v_bias, int batch, int mem_len,
                                int seg_len, int heads, int d_head, txl_dtype dtype, void *out,
                                float *lse, void *stream);

/*
 * txl_mem_update -- the per-layer memory rollover (Transformer-XL,
 * Section 3.2: a cache of the last M hidden states, possibly spanning several
 * segments, reused as extended context by the next segment).
 *
 * ext_ctx  : device, [M+L][batch][d_model] = [memory; current hidden states].
 * mem_next : device, at least [M][batch][d_model]; rows 0..M-1 receive the
 *            newest M rows of ext_ctx (rows L..M+L-1), oldest first -- i.e.
 *            the memory part of the next segment's extended context.  Must not
 *            overlap ext_ctx (use two buffers and swap them per segment).
 * Bit-exact copy of dtype elements.  mem_len == 0 or batch == 0 or
 * d_model == 0 => nothing to do.  Same error behaviour as above.
 */
txl_status txl_mem_update(void *mem_next, const void *ext_ctx, int batch, int mem_len,
                          int seg_len, int d_model, txl_dtype dtype, void *stream);

/*
 * txl_rel_attn_fwd_mem -- one layer's txl_rel_attn_fwd and txl_mem_update in
 * one call (Section 3.3's attention and Section 3.2's cache update of the
 * same layer, which do not depend on each other).  Where it pays, the
 * attention launch does the rollover copy as well (bf16, d_head = 64, the
 * tensor-memory path, 16-byte aligned ext_ctx + seg_len rows and mem_next,
 * M*batch*d_model*2 a multiple of 16, and a copy small against the
 * attention's own work); otherwise the rollover runs as its own launch right
 * after, on the same stream.  Results are exactly those of the two calls.
 *
 * Arguments as txl_rel_attn_fwd, plus mem_next, ext_ctx and d_model as
 * txl_mem_update (same batch, mem_len, seg_len and dtype).  mem_next must not
 * overlap ext_ctx or any buffer of the attention; ext_ctx must not overlap
 * out.  With nothing to attend (batch, seg_len or heads 0) only the rollover
 * runs; with nothing to roll (mem_len or d_model 0) mem_next and ext_ctx are
 * unused.  Same error behaviour as the two calls.
 */
txl_status txl_rel_attn_fwd_mem(const void *q, const void *k, const void *v, const void *r,
                                const float *u_bias, const float *v_bias, int batch, int mem_len,
                                int seg_len, int heads, int d_head, txl_dtype dtype, void *out,
                                void *mem_next, const void *ext_ctx, int d_model, void *stream);

/*
 * txl_rel_attn_fwd_mem_cells -- several independent txl_rel_attn_fwd_mem
 * calls of one shape (e.g. the layer calls of one step of a layer-by-segment
 * wavefront: different layers, different segments, none waiting for
 * another's result).  Call c takes q[c], k[c], v[c], r[c], u_bias[c],
 * v_bias[c], out[c], mem_next[c] and ext_ctx[c], each as
 * txl_rel_attn_fwd_mem takes it; batch, mem_len, seg_len, heads, d_head,
 * dtype and d_model are shared.  The results are exactly those of the calls
 * one after another.  With bf16 and d_head = 64, unsplit calls with TMA-
 * addressable operands share launches (up to 8 calls a launch, their work
 * items in one persistent schedule, each call's rollover inside where it
 * fuses); other shapes run call by call.
 *
 * cells           : number of calls, >= 0 (0: nothing).
 * q .. ext_ctx    : host arrays of `cells` device pointers.  u_bias, v_bias
 *                   may be NULL (no bias in any call) or hold NULL entries;
 *                   mem_next and ext_ctx may be NULL when there is nothing to
 *                   roll (batch, mem_len or d_model 0); the others are
 *                   required when there is attention work.
 * Errors: every call's txl_rel_attn_fwd_mem checks, plus TXL_ERR_INVALID
 * when one call's out or mem_next overlaps any buffer of another call.
 * Nothing is launched when an argument is rejected.
 */
txl_status txl_rel_attn_fwd_mem_cells(int cells, const void *const *q, const void *const *k,
                                      const void *const *v, const void *const *r,
                                      const float *const *u_bias, const float *const *v_bias, int batch,
                                      int mem_len, int seg_len, int heads, int d_head, txl_dtype dtype,
                                      void *const *out, void *const *mem_next, const void *const *ext_ctx,
                                      int d_model, void *stream);

/*
 * txl_rel_attn_fwd_ring -- txl_rel_attn_fwd with k and v stored as a ring.
 * The extended context [memory; segment] of Section 3.2 slides forward by L
 * rows per segment; kept in a ring of M+L rows, a segment adds only its L new
 * rows (txl_ring_append) instead of moving the M memory rows.  The paper has
 * no counterpart to this storage order; the result is exactly that of
 * txl_rel_attn_fwd on the unrolled context.
 *
 * k, v     : device, [M+L][batch][heads][d_head]; the context's key j (j = 0
 *            is the oldest memory row, j = M+L-1 the segment's last row) is
 *            stored at row (kv_start + j) mod (M+L).
 * kv_start : 0 <= kv_start < M+L (0 gives txl_rel_attn_fwd's layout).
 * Everything else as txl_rel_attn_fwd.  With bf16 and d_head = 64 the rows
 * are read by TMA when kv_start and M+L are multiples of 8, by thread loads
 * otherwise (same result, slower).
 */
txl_status txl_rel_attn_fwd_ring(const void *q, const void *k, const void *v, const void *r,
                                 const float *u_bias, const float *v_bias, int batch, int mem_len,
                                 int seg_len, int heads, int d_head, int kv_start, txl_dtype dtype,
                                 void *out, void *stream);

/*
 * txl_rel_attn_fwd_padded -- txl_rel_attn_fwd on head vectors stored with
 * d_pad >= d_head elements each (zeros past d_head), the layout
 * txl_project_heads and txl_rel_table write.  q, k, v, r, out are
 * [..][heads][d_pad]; u_bias, v_bias [heads][d_pad] (or NULL).  The result
 * equals txl_rel_attn_fwd on the first d_head elements (scale 1/sqrt(d_head));
 * out's padding columns come out zero.  With bf16 and d_pad = 64 the rows are
 * read by TMA whatever d_head is (e.g. d_head 41 padded to 64).
 */
txl_status txl_rel_attn_fwd_padded(const void *q, const void *k, const void *v, const void *r,
                                   const float *u_bias, const float *v_bias, int batch, int mem_len,
                                   int seg_len, int heads, int d_head, int d_pad, txl_dtype dtype,
                                   void *out, void *stream);

/*
 * txl_project_heads -- the projections of Section 3.3's procedure
 * (q = h W_q^T, k = h~ W_kE^T, v = h~ W_v^T) into the attention's layout:
 *     y[rows][heads][d_pad] = x[rows][d_in] . W^T
 * with W in the paper's layout, [heads*d_head][d_in] (row h*d_head + d is
 * output column d of head h; also torch.nn.Linear's weight layout), and
 * padding columns d_head..d_pad-1 of every head exactly zero.  With
 * x = a T-major [positions][batch][d_model] buffer (rows = positions*batch)
 * the result is the T-major [positions][batch][heads][d_pad] layout.
 * bf16: the library's tcgen05 GEMM (fp32 accumulation, one rounding to
 * bf16), for d_in even and x, w 4-byte aligned (TMA operand loads when d_in
 * is a multiple of 8, x and w 16-byte aligned and d_pad divides 256; TMA
 * output stores when out is 16-byte aligned and heads*d_pad*2 a multiple of
 * 16); fp32 and other bf16 shapes: a CUDA-core kernel (fp32 accumulation).
 * x, w, out device, row-major, dtype elements; out must not overlap x or w.
 * d_pad >= d_head >= 1; d_in == 0 gives zeros.
 */
txl_status txl_project_heads(const void *x, const void *w, void *out, int rows, int d_in, int heads,
                             int d_head, int d_pad, txl_dtype dtype, void *stream);

/*
 * txl_project_qkv -- a layer's three projections of Section 3.3's procedure
 * from one extended context h~ = [memory; h] (x, [rows][d_in], rows =
 * positions x batch of a T-major buffer):
 *     k = x W_k^T and v = x W_v^T over all rows, and
 *     q = x[q_row0 ..] W_q^T over the last rows - q_row0 rows (the segment's
 *         own positions h: q_row0 = mem_len x batch),
 * each as txl_project_heads writes it ([..][heads][d_pad], padding zero).
 * w_q and q are both given or both NULL (then only k and v).  bf16 with
 * d_in a multiple of 8, every pointer 16-byte aligned, heads*d_pad*2 a
 * multiple of 16 and d_pad dividing 256: the three come from one launch of
 * the projection GEMM that reads x once for k and v (and for q too when
 * q_row0 is a multiple of 128; otherwise q's rows are a band of their own in
 * the same launch); other shapes are computed as by three txl_project_heads
 * calls.
 * Outputs must not overlap x, the weights or one another; 0 <= q_row0 <=
 * rows.  Results equal the separate txl_project_heads calls bit for bit.
 */
txl_status txl_project_qkv(const void *x, int rows, int d_in, const void *w_q, const void *w_k, const void *w_v,
                           void *q, void *k, void *v, int q_row0, int heads, int d_head, int d_pad, txl_dtype dtype,
                           void *stream);

/*
 * txl_project_qkv_cells -- txl_project_qkv for several layer calls of one
 * shape at once (cells c = 0 .. cells-1, e.g. the layer calls of a
 * recurrence that do not depend on each other): cell c projects x[c] with
 * w_q[c], w_k[c], w_v[c] into q[c], k[c], v[c] (rows, d_in, q_row0, heads,
 * d_head, d_pad shared).  x, w_*, q, k, v are host arrays of `cells` device
 * pointers (w_q and q both NULL, or both arrays with every entry set); no
 * output may overlap any input or any other output of any cell.  Where
 * txl_project_qkv would use one launch per cell, up to eight cells share a
 * launch; results equal the per-cell calls bit for bit.
 */
txl_status txl_project_qkv_cells(int cells, const void *const *x, const void *const *w_q, const void *const *w_k,
                                 const void *const *w_v, void *const *q, void *const *k, void *const *v, int rows,
                                 int d_in, int q_row0, int heads, int d_head, int d_pad, txl_dtype dtype,
                                 void *stream);

/*
 * txl_rel_table -- Appendix B's reversed projected table of one layer:
 * out[t][h][d] = sum_c R[klen-1-t][c] * W_kR[h*d_head + d][c] for t < klen,
 * R[p][2c] = sin(p * 10000^(-2c/d_model)), R[p][2c+1] = cos(the same angle)
 * (the sinusoid of the relative distance p, evaluated in fp32 on the device;
 * fp32 accumulation).  out [klen][heads][d_pad], padding zero; W_kR in the
 * paper's layout [heads*d_head][d_model].  Batch- and segment-independent:
 * once per layer.
 */
txl_status txl_rel_table(const void *w_r, void *out, int klen, int d_model, int heads, int d_head, int d_pad,
                         txl_dtype dtype, void *stream);

/*
 * txl_rel_attn_bwd -- gradients of one txl_rel_attn_fwd call for a given
 * output gradient dout (the chain rule through the masked softmax and the
 * four-term score of Section 3.3).  With P the softmax weights of query row
 * i, dA_ij = P_ij (dout_i.v_j - sum_l P_il dout_i.v_l) / sqrt(d_head) for the
 * visible keys j <= M+i and off = M+i-j:
 *     dq_i = sum_j dA_ij (k_j + r[T-1-off])    dk_j = sum_i dA_ij (q_i + u)
 *     dv_j = sum_i P_ij dout_i                 dr[T-1-off] += dA_ij (q_i + v)
 *     du   = sum_{b,i,j} dA_ij k_j             dw = sum_{b,i,j} dA_ij r[T-1-off]
 * (dr, du, dw summed over the batch).  Every input gets its gradient, the
 * memory rows 0..M-1 of k and v included: Section 3.2's stop-gradient acts
 * on the cached hidden states, while the keys and values projected from them
 * still carry gradient to the projections.
 *
 * q, k, v, r, dout : device, dtype, layouts as txl_rel_attn_fwd (dout like q).
 * u_bias, v_bias   : device float32 [heads][d_head] or NULL (zero bias).
 * out, lse         : the forward's output and row log-sum-exp as
 *                    txl_rel_attn_fwd_lse wrote them for these inputs (out
 *                    16-byte aligned, lse 4-byte aligned), or both NULL.
 *                    Given, they spare the backward its own forward pass;
 *                    the bf16 d_head = 64 path reads them, the others (which
 *                    recompute the scores in full) ignore them.  Exactly one
 *                    of them NULL => TXL_ERR_INVALID.
 * dq, dk, dv, dr   : device outputs, dtype, shaped like q, k, v, r.
 * du, dw           : device float32 [heads][d_head] outputs, or NULL (not
 *                    computed).  Outputs must not overlap each other, any
 *                    input or the workspace.
 * workspace        : device scratch of at least the bytes that
 *                    txl_rel_attn_bwd_workspace reports, 256-byte aligned,
 *                    owned by the caller.  bf16 with d_head = 64: P and dA
 *                    as bf16 plus dA in the table's frame (about 3 x 2 bytes
 *                    per (b, h, i, j) score entry); otherwise the score, P,
 *                    dP and dA of every head (about 3 x 4 + 3 x dtype bytes
 *                    per entry).
 * Limits: d_head <= 128 (else TXL_ERR_UNSUPPORTED).  Asynchronous on stream.
 * bf16: operands of the contractions in bf16 (q+u, q+v, P and dA rounded
 * once), fp32 accumulation, fp32 softmax; fp32: fp32 throughout.
 */
txl_status txl_rel_attn_bwd_workspace(int batch, int mem_len, int seg_len, int heads, int d_head,
                                      txl_dtype dtype, size_t *bytes);
txl_status txl_rel_attn_bwd(const void *q, const void *k, const void *v, const void *r, const float *u_bias,
                            const float *v_bias, const void *dout, const void *out, const float *lse, int batch,
                            int mem_len, int seg_len, int heads, int d_head, txl_dtype dtype, void *dq, void *dk,
                            void *dv, void *dr, float *du, float *dw, void *workspace, size_t workspace_bytes,
                            void *stream);

/*
 * txl_ring_append -- write n_rows new rows into a ring of ring_len rows at
 * rows (start + i) mod ring_len, i = 0 .. n_rows-1 (the oldest rows of the
 * ring, for a ring kept as above: start = the current kv_start, after which
 * the next kv_start is (start + n_rows) mod ring_len).  Serves both the
 * cached hidden states of Section 3.2 and projected k / v rings.
 *
 * ring : device, [ring_len][row_elems] dtype elements.
 * rows : device, [n_rows][row_elems]; must not overlap ring.
 * 0 <= n_rows <= ring_len, 0 <= start < ring_len (unless nothing to do),
 * row_elems >= 0; element-aligned pointers.  Bit-exact copy (one or two
 * contiguous runs).  Same error behaviour as txl_mem_update.
 */
txl_status txl_ring_append(void *ring, const void *rows, int ring_len, int n_rows, int row_elems,
                           int start, txl_dtype dtype, void *stream);

/*
 * txl_rel_attn_fwd_noalloc -- txl_rel_attn_fwd for callers that may not
 * allocate device memory.  (No counterpart in the paper: this is a deployment
 * variant of the same computation.)
 *
 * Some callers cannot call cudaMalloc: code inside a framework that owns all
 * device memory through its own pool or a fixed arena, hosts that forbid
 * allocation once initialised, or processes whose device memory is already
 * fully reserved.  txl_rel_attn_fwd may allocate its split-key scratch on
 * first use; this entry point allocates nothing.  Its scratch is one fixed
 * array of TXL_NOALLOC_SCRATCH_BYTES inside the library's device code, held
 * on every GPU that loads that code until the process exits.
 *
 * Same arguments, layouts, results and error rules as txl_rel_attn_fwd, plus:
 *   - a call whose key split needs more than TXL_NOALLOC_SCRATCH_BYTES
 *     (splits * batch * heads * seg_len * (2 * ceil16(d_head) + 4) + 256
 *     bytes) returns TXL_ERR_UNSUPPORTED before touching the GPU;
 *   - the first call on a device that splits its keys looks up the array's
 *     device address (cudaGetSymbolAddress, with that device current); make
 *     that first call before any stream capture.  Under CUDA's default lazy
 *     module loading the array is reserved on a device when the library's
 *     device code is first loaded there, which can be as late as that lookup:
 *     a caller that reserves the rest of device memory afterwards should make
 *     one such call first (a long-memory shape, e.g. B 1, H 4, D 64,
 *     L 128, M 1600);
 *   - the cached address belongs to the device's primary context: a device
 *     reset (cudaDeviceReset) while the library is loaded is not supported;
 *   - every call shares the one array, and each call writes every part of it
 *     that it reads back, so nothing carries over between calls; but calls
 *     whose kernels overlap on the GPU (different streams, or concurrent
 *     host threads) race on it and must be serialised by the caller.
 */
#define TXL_NOALLOC_SCRATCH_BYTES ((size_t)32 << 20)

txl_status txl_rel_attn_fwd_noalloc(const void *q, const void *k, const void *v, const void *r,
                                    const float *u_bias, const float *v_bias,
                                    int batch, int mem_len, int seg_len, int heads, int d_head,
                                    txl_dtype dtype, void *out, void *stream);

/*
 * txl_softmax_xent_fwd -- the output layer's cross entropy (Transformer-XL's
 * training objective, Section 4: the negative log-likelihood of the next
 * token), taken over the vocabulary in pieces: the rows x vocab logits are
 * never in memory.  For every row i < rows, with j < vocab:
 *     z_ij   = h_i . w_j + bias_j
 *     lse_i  = log sum_j exp(z_ij)
 *     loss_i = lse_i - z_{i,target_i}
 * A row whose target lies outside [0, vocab) (a negative padding label, say)
 * is empty: its loss is 0, whatever h_i holds, and its lse is still
 * computed.  A row whose every logit is -infinity has lse -infinity and
 * loss 0.  A bias entry of -infinity takes its token out of the vocabulary
 * (its row of w has to be finite all the same).  Logits are scaled by log2(e)
 * in float32: one below -2^127 counts as -infinity, so that the type's lowest
 * value masks as -infinity does (and a row of nothing else has lse -infinity
 * and loss 0, a target among them loss infinity).
 *
 * h         : device, dtype [rows][d_model] (any leading shape: a T-major
 *             [positions][batch][d_model] buffer has rows = positions*batch).
 * w         : device, dtype [vocab][d_model] (torch.nn.Linear's and
 *             torch.nn.Embedding's weight layout: a tied embedding fits).
 * bias      : device, float32 [vocab], or NULL (no bias).
 * target    : device, int64 [rows].
 * loss, lse : device outputs, float32 [rows].
 * workspace : device scratch of at least the bytes that
 *             txl_softmax_xent_workspace reports for backward = 0, 256-byte
 *             aligned, owned by the caller: calls that may overlap on the GPU
 *             need workspaces of their own.  Nothing is kept in it between
 *             calls.
 * Pointers are element-aligned (h, w: 2 or 4 bytes; float32: 4; int64: 8);
 * rows of w and h that the TMA unit can address (d_model a multiple of 8,
 * 16-byte aligned bases) are read in place with TXL_BF16, others are copied
 * piece by piece into the workspace first (not for a handful of rows with
 * d_model <= 1024 and w 16-byte aligned).
 * rows == 0: nothing to do.  d_model >= 1, vocab >= 1, else TXL_ERR_INVALID;
 * vocab and rows <= 2^30, d_model <= 2^24 and at most 2^40 elements in h and
 * in w, else TXL_ERR_UNSUPPORTED.  Asynchronous on
 * stream; no allocation; results do not depend on what else runs (no
 * atomics: the same call gives the same bits).  bf16: products of bf16
 * operands, accumulated and normalised in fp32.
 */
txl_status txl_softmax_xent_workspace(int rows, int d_model, int vocab, txl_dtype dtype, int backward, size_t *bytes);
txl_status txl_softmax_xent_fwd(const void *h, const void *w, const float *bias, const int64_t *target, int rows,
                                int d_model, int vocab, txl_dtype dtype, float *loss, float *lse, void *workspace,
                                size_t workspace_bytes, void *stream);

/*
 * txl_softmax_xent_bwd -- gradients of sum_i dloss_i loss_i of one
 * txl_softmax_xent_fwd call, from its lse:
 *     dz_ij = dloss_i (exp(z_ij - lse_i) - [j = target_i])
 *     dh_i  = sum_j dz_ij w_j,  dw_j = sum_i dz_ij h_i,  dbias_j = sum_i dz_ij
 * The logits are computed again, piece by piece.  Empty rows, rows of lse
 * -infinity and rows of dloss 0 have dh exactly 0 and add nothing to dw and
 * dbias, whatever h_i holds.
 *
 * lse       : device, float32 [rows], as the forward wrote it.
 * dloss     : device, float32 [rows].
 * dh, dw    : device outputs, dtype, shaped like h and w; either may be NULL
 *             (not computed: a frozen layer).
 * dbias     : device output, float32 [vocab], or NULL; it may be asked for
 *             with bias NULL as well.
 * workspace : as above, for backward = 1 (which also suffices for the
 *             forward).
 * rows == 0: dw and dbias are set to 0.  Outputs must not overlap each other,
 * any input or the workspace.  bf16: with more than 128 rows dz is rounded
 * once to bf16 for the two products, else it keeps at least 16 bits (fp32
 * accumulation over the whole vocabulary and all rows, one rounding of the
 * results); dbias sums the unrounded dz.
 */
txl_status txl_softmax_xent_bwd(const void *h, const void *w, const float *bias, const int64_t *target,
                                const float *lse, const float *dloss, int rows, int d_model, int vocab,
                                txl_dtype dtype, void *dh, void *dw, float *dbias, void *workspace,
                                size_t workspace_bytes, void *stream);

/*
 * txl_distill_fwd -- the output layer as a student of a teacher of which the
 * top_k largest logits per row were kept.  With temperature t,
 *     p_ik   = softmax over row i's valid entries of teacher_logits_ik / t
 *     lse_i  = log sum_j exp(z_ij / t)      (the whole vocabulary)
 *     loss_i = t^2 sum_k p_ik (log p_ik - (z_{i,idx_ik} / t - lse_i))
 * i.e. t^2 KL(teacher's kept entries, renormalised || student), the factor
 * t^2 keeping gradients of different temperatures alike.  An entry is valid
 * when 0 <= teacher_idx < vocab and its logit is not -infinity; a row
 * without a valid entry is empty (loss 0, as a padding row above).  An index
 * listed twice counts twice.  A teacher's logit of its type's lowest value is
 * a value like others: of weight 0 next to larger ones, and a row of nothing
 * else is uniform over its entries.  z, h, w, bias, loss, lse, workspace and
 * everything unsaid as txl_softmax_xent_fwd.
 *
 * teacher_idx    : device, int64 [rows][top_k], in any order.
 * teacher_logits : device, teacher_dtype [rows][top_k].
 * 1 <= top_k (else TXL_ERR_INVALID), top_k <= 256 (else
 * TXL_ERR_UNSUPPORTED); 2^-63 <= temperature <= 2^63 (its square is a normal
 * float32 number), else TXL_ERR_INVALID.
 */
txl_status txl_distill_workspace(int rows, int d_model, int vocab, int top_k, txl_dtype dtype, int backward,
                                 size_t *bytes);
txl_status txl_distill_fwd(const void *h, const void *w, const float *bias, const int64_t *teacher_idx,
                           const void *teacher_logits, txl_dtype teacher_dtype, float temperature, int rows,
                           int d_model, int vocab, int top_k, txl_dtype dtype, float *loss, float *lse,
                           void *workspace, size_t workspace_bytes, void *stream);

/*
 * txl_distill_bwd -- gradients of sum_i dloss_i loss_i of one
 * txl_distill_fwd call, from its lse (taken at the same temperature t):
 *     dz_ij = dloss_i t (exp(z_ij / t - lse_i) - sum_{k: idx_ik = j} p_ik)
 * and dh, dw, dbias as txl_softmax_xent_bwd, with its rules for empty rows,
 * absent outputs, rows == 0, the workspace and rounding.
 */
txl_status txl_distill_bwd(const void *h, const void *w, const float *bias, const int64_t *teacher_idx,
                           const void *teacher_logits, txl_dtype teacher_dtype, float temperature, const float *lse,
                           const float *dloss, int rows, int d_model, int vocab, int top_k, txl_dtype dtype,
                           void *dh, void *dw, float *dbias, void *workspace, size_t workspace_bytes, void *stream);

/*
 * txl_embed_fwd -- the token embedding: out_i = scale * table[token_i] for
 * every row i < rows (the scale is sqrt(d_model) where the table is tied to
 * the output layer), a row of zeros for a token outside [0, vocab) (a
 * negative padding token, say).
 *
 * tokens : device, int64 [rows] (any leading shape: a T-major
 *          [positions][batch] buffer has rows = positions*batch).
 * table  : device, dtype [vocab][d_model].
 * out    : device output, dtype [rows][d_model]; must not overlap an input.
 * Element-aligned pointers; rows that are multiples of 16 bytes at 16-byte
 * aligned bases move fastest.  rows == 0: nothing to do.  d_model >= 1, vocab
 * >= 1, else TXL_ERR_INVALID; vocab and rows <= 2^30, d_model <= 2^24 and at
 * most 2^40 elements in table and out, else TXL_ERR_UNSUPPORTED.
 * Asynchronous on stream; no allocation.
 */
txl_status txl_embed_fwd(const int64_t *tokens, const void *table, float scale, int rows, int d_model, int vocab,
                         txl_dtype dtype, void *out, void *stream);

/*
 * txl_embed_bwd -- the table's gradient of one txl_embed_fwd call:
 *     dtable_t = scale * sum_{i: token_i = t} dout_i
 * for every token t, 0 for a token that no row has; with accumulate != 0 the
 * sum is added to what dtable holds (the gradient of an output layer tied to
 * the table, as txl_softmax_xent_bwd wrote it) and rows of other tokens are
 * left as they are.  Rows of tokens outside [0, vocab) add nothing, whatever
 * dout holds there.  Sums are held in fp32, in an order that the tokens alone
 * determine (no atomics: the same call gives the same bits), and rounded once.
 *
 * dout      : device, dtype [rows][d_model].
 * dtable    : device output, dtype [vocab][d_model].
 * workspace : device scratch of at least the bytes that
 *             txl_embed_bwd_workspace reports, 256-byte aligned, owned by the
 *             caller: calls that may overlap on the GPU need workspaces of
 *             their own.  Nothing is kept in it between calls.
 * dtable and workspace must not overlap each other or an input.  rows == 0:
 * dtable is set to 0, or left as it is.  Sizes and everything unsaid as
 * txl_embed_fwd.
 */
txl_status txl_embed_bwd_workspace(int rows, int d_model, int vocab, txl_dtype dtype, size_t *bytes);
txl_status txl_embed_bwd(const int64_t *tokens, const void *dout, float scale, int rows, int d_model, int vocab,
                         txl_dtype dtype, int accumulate, void *dtable, void *workspace, size_t workspace_bytes,
                         void *stream);

/*
 * txl_layer_norm_fwd -- layer norm of a residual sum, per row of d = d_model
 * columns:
 *     s = x + residual,  mean = sum_d s / d,  var = sum_d (s - mean)^2 / d,
 *     rstd = 1 / sqrt(var + eps),  y = (s - mean) rstd gamma + beta
 * after a sub-layer (y = LN(x + f(x)), the paper's order), or before one, with
 * the sum kept for the next residual: where `sum` is given, s is rounded to
 * dtype, stored there, and normalised as stored.
 *
 * x, residual : device, dtype [rows][d_model]; residual may be NULL (s = x).
 * gamma, beta : device, float32 [d_model]; either may be NULL (1, 0).
 * y           : device output, dtype [rows][d_model].
 * sum         : device output, dtype [rows][d_model], or NULL.
 * mean, rstd  : device outputs, float32 [rows], for the backward; both or
 *               neither NULL (not stored).
 * Outputs must not overlap each other or any input.  Element-aligned
 * pointers; rows that are multiples of 16 bytes at 16-byte aligned bases
 * move fastest.  eps > 0 and finite.  rows == 0: nothing to do.  d_model >=
 * 1, else TXL_ERR_INVALID; d_model <= 8192, rows <= 2^30, else
 * TXL_ERR_UNSUPPORTED.  fp32 arithmetic, sums in an order as
 * txl_layer_norm_bwd's, one rounding of y.  Asynchronous on stream; no
 * allocation.
 */
txl_status txl_layer_norm_fwd(const void *x, const void *residual, const float *gamma, const float *beta, float eps,
                              int rows, int d_model, txl_dtype dtype, void *y, void *sum, float *mean, float *rstd,
                              void *stream);

/*
 * txl_layer_norm_bwd -- gradients of one txl_layer_norm_fwd call, from its
 * mean and rstd.  With xh = (s - mean) rstd and g = dy gamma,
 *     dx     = rstd (g - sum_d g / d - xh sum_d (g xh) / d) + dsum
 *     dgamma = sum_i dy_i xh_i,  dbeta = sum_i dy_i
 * dx is the gradient of s: of x and of the residual alike.
 *
 * dy       : device, dtype [rows][d_model].
 * x        : what was normalised: the forward's x, with its residual again in
 *            `residual`; or the sum it kept, with residual NULL.
 * dsum     : device, dtype [rows][d_model]: the gradient that reaches the kept
 *            sum by its other path, added to dx; or NULL.
 * dx       : device output, dtype [rows][d_model].
 * dgamma, dbeta : device outputs, float32 [d_model]; either may be NULL (not
 *            computed).
 * workspace : device scratch of at least the bytes that
 *            txl_layer_norm_bwd_workspace reports, 256-byte aligned, owned by
 *            the caller, as txl_embed_bwd's; unused (and may be NULL) without
 *            dgamma and dbeta.
 * rows == 0: dgamma and dbeta are set to 0.  fp32 arithmetic and sums, over
 * a row and over rows, in an order that the sizes, the dtype and the buffers'
 * alignment determine (the same call gives the same bits; at addresses of
 * another alignment the last ones may differ), one rounding of dx.  Outputs
 * must not overlap each other, any input or the workspace.  Sizes as
 * txl_layer_norm_fwd.
 */
txl_status txl_layer_norm_bwd_workspace(int rows, int d_model, txl_dtype dtype, size_t *bytes);
txl_status txl_layer_norm_bwd(const void *dy, const void *x, const void *residual, const void *dsum, const float *gamma,
                              const float *mean, const float *rstd, int rows, int d_model, txl_dtype dtype, void *dx,
                              float *dgamma, float *dbeta, void *workspace, size_t workspace_bytes, void *stream);

/*
 * One tensor of an optimiser step.  Element-aligned device pointers; tensors
 * at 16-byte boundaries move fastest.
 */
typedef struct {
    void *param;              /* param_dtype [size] */
    float *master;            /* [size]: the float32 weights of which a TXL_BF16 param is the rounded copy; or NULL
                                 (the step acts on param itself) */
    const void *grad;         /* grad_dtype [size] */
    void *exp_avg;            /* m: float32 [size], or e4m3 codes of m / scale (uint8 [size]) */
    void *exp_avg_sq;         /* v: float32 [size], or e4m3 codes of sqrt(v) / scale */
    float *exp_avg_scale;     /* NULL: float32 moments; else their scales, one per 256 elements, */
    float *exp_avg_sq_scale;  /* [ceil(size / 256)] each (both or neither) */
    int64_t size;             /* elements, 0 .. 2^40 */
    float weight_decay;       /* finite, >= 0 */
    txl_dtype param_dtype, grad_dtype;
} txl_adamw_tensor;

typedef struct {
    float lr;                 /* finite, >= 0 (unused with lr_device) */
    float eps;                /* finite, >= 2^-126 */
    double beta1, beta2;      /* 0 <= beta < 1 */
    int64_t step;             /* the step's number t >= 1 (unused with step_device) */
    const float *lr_device;   /* device float32 [1], or NULL: read when the kernel runs (captured steps), and
                                 used as it is */
    const int64_t *step_device;  /* device int64 [1], or NULL */
    const float *grad_scale;  /* device float32 [1], or NULL (1): a factor of all gradients */
    uint64_t seed;            /* of the 8-bit moments' rounding */
} txl_adamw_options;

/*
 * txl_grad_norm -- the norm of all the tensors' gradients taken as one
 * vector, and the factor that clips it:
 *     norm = sqrt(sum_k sum_i grad_ki^2),  clip = min(1, max_norm / norm)
 * A norm that is not finite (also: a square, or a part's sum of squares, past
 * the float32 range) has clip NaN, which makes a txl_adamw_step that takes it
 * as its grad_scale do nothing.
 *
 * t          : host array of `tensors` descriptions; grad, grad_dtype and size
 *              are used.
 * max_norm   : > 0.
 * norm, clip : device outputs, float32 [1]; either may be NULL.
 * workspace  : device scratch of at least the bytes that
 *              txl_grad_norm_workspace reports for these sizes, 256-byte
 *              aligned, owned by the caller, as txl_embed_bwd's.
 * Squares are rounded to fp32; their sums keep the bits of a double's, in an
 * order that the sizes determine.  Asynchronous on stream.
 */
txl_status txl_grad_norm_workspace(int tensors, const txl_adamw_tensor *t, size_t *bytes);
txl_status txl_grad_norm(int tensors, const txl_adamw_tensor *t, float max_norm, float *norm, float *clip,
                         void *workspace, size_t workspace_bytes, void *stream);

/*
 * txl_adamw_step -- one AdamW step over many tensors, in place.  With p the
 * master weights (or param where there are none), per element:
 *     g = grad * grad_scale
 *     m = beta1 m + (1 - beta1) g,  v = beta2 v + ((1 - beta2) g) g
 *     p = p - lr (weight_decay p + (m / (1 - beta1^step)) / (sqrt(v / (1 - beta2^step)) + eps))
 * in fp32; param is rounded to nearest from p.  Up to 384 tensors share a
 * launch.  A grad_scale that is not finite, or a step_device below 1, makes
 * the call leave everything as it is.
 *
 * 8-bit moments: x (m, or sqrt(v)) is stored as a code c and the scale of its
 * 256 elements (the tensor's elements 256 b .. 256 b + 255), x = c * scale,
 * with scale = max |x| (1 / 448) (a block whose largest is below 2^-100 is
 * stored as zeros).  y = x ((1 / max |x|) 448) is rounded to one of its two
 * neighbours among the e4m3 values, 2^(e-3) apart with e = max(floor(log2
 * |y|), -6): to floor(|y| / 2^(e-3) + u) such steps, at most 448, and for
 * sqrt(v) > 0 at least one (a denominator is not lost).  u is the low 16 bits
 * (for m; the high ones for sqrt(v)) over 2^16 of
 *     h = mix(mix(mix(mix(mix(seed lo) + seed hi) + k) + step) + i + (i >> 32) 0x9e3779b9)
 * in 32 bits, k the tensor's place in the call, i the element, where
 * mix(x): x = (x ^ x >> 16) 0x7feb352d, x = (x ^ x >> 15) 0x846ca68b,
 * x ^ x >> 16 (constants of C. Wellons, "Prospecting for Hash Functions",
 * 2018, public domain).  m, v, sqrt(v) and y are computed operation by
 * operation as written, each rounded to fp32, so that plain fp32 arithmetic
 * gives the same codes.  The update uses m and v before they become codes (0 where a finite
 * gradient's v is infinite, as with float32 moments).  A block whose m or
 * sqrt(v) is not finite, or 2^126 or more, has lost them: its scale becomes
 * NaN, and what the next step makes of it; use grad_scale.
 *
 * t : host array of `tensors` descriptions.  param, master, the moments and
 * their scales must overlap neither each other, in any tensor, nor a gradient
 * or an option's device value.  tensors == 0 or sizes of 0: nothing to do.
 * Asynchronous on stream; no allocation on the device.
 */
txl_status txl_adamw_step(int tensors, const txl_adamw_tensor *t, const txl_adamw_options *options, void *stream);

/*
 * txl_check -- synchronise `stream`, then report and clear the library's
 * device error word: TXL_ERR_TIMEOUT if an in-kernel bounded wait gave up
 * since the last check, TXL_ERR_CUDA if the stream reports an error, else
 * TXL_OK.
 */
txl_status txl_check(void *stream);

/*
 * txl_selftest_wait -- exercise the failure path of the kernels' bounded
 * waits without any fault: a one-warp kernel waits on an mbarrier that
 * nothing completes, through the same bounded wait the kernels use but
 * limited to limit_us microseconds (1 .. 1,000,000; else TXL_ERR_INVALID).
 * The wait runs out and records the device error word, so the next
 * txl_check(stream) returns TXL_ERR_TIMEOUT (and clears it); the context
 * stays usable.  No counterpart in the paper: a test hook of the library.
 */
txl_status txl_selftest_wait(unsigned int limit_us, void *stream);

/* Static description of a status code; never NULL. */
const char *txl_status_string(txl_status s);

/* Number of the most recent CUDA error seen by the library on this thread
 * (0 if none); pairs with TXL_ERR_CUDA. */
int txl_last_cuda_error(void);

/* Library version, major * 10000 + minor * 100 + patch. */
int txl_version(void);

/* Free the library-owned scratch buffers of the current device (every
 * stream's).  Waits for the device to finish its work first (this is not a
 * compute call).  Safe to call more than once; later calls re-allocate on
 * demand. */
void txl_shutdown(void);

#ifdef __cplusplus
}
#endif

#endif /* TXL_H_ */
