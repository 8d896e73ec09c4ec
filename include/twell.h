/*
 * twell.h — C ABI of the TwELL activation-sparse feed-forward layer (sm_103a).
 *
 * The layer is the ReLU (or ReLU-gated) transformer feed-forward block of
 * "Sparser, Faster, Lighter Transformer Language Models" (Cetin, Peluchetti,
 * Castillo, Naruse, Murakami, Jones, 2026; gist.science summary, Resumo Técnico
 * §2 Metodologia). L1-regularised training leaves more than 99 % of the hidden
 * activations at zero; the post-ReLU hidden matrix h is packed into TwELL
 * (Tile-wise ELLPACK) straight from the up-projection's epilogue, and the
 * down-projection and the backward run only over the stored entries.
 *
 * TwELL layout (one tile = T consecutive token rows spanning all F hidden units):
 *   nnz_row[r]   number of active entries of row r
 *   K_tile[t]    max nnz_row over the rows of tile t (the tile's width)
 *   tile_off[t]  first slot of tile t; tile_off[0] = 0,
 *                tile_off[t+1] = tile_off[t] + rows(t) * K_tile[t],
 *                rows(t) = min(T, M - t*T)
 *   slot off[t] + i*K[t] + k of row i of tile t holds, for k < nnz, the k-th
 *   active column in ascending order (idx, int32) and h there (val, bf16 bits);
 *   for k >= nnz it holds idx = -1, val = +0.
 * Active set: h != 0 for the ReLU layer and for twell_pack (-0 counts as zero,
 * NaN as nonzero); pre_gate > 0 for the gated layer.
 *
 * Conventions for every entry point:
 *   - Pointers named in the argument list are DEVICE pointers unless marked
 *     "host". bf16 tensors are passed as uint16_t bit arrays; all matrices are
 *     row-major and densely packed (row stride = column count) unless a leading
 *     dimension is given. Weights are [F, d]: one row per hidden unit.
 *   - The caller owns and allocates every buffer. The library never allocates
 *     memory, frees or synchronises (twell_check is the one call that
 *     synchronises); each call only enqueues work on `stream` (a cudaStream_t
 *     passed as void*, NULL = the legacy default stream) and returns. Buffers
 *     must stay alive until that work has finished. twell_ffn_bwd forks part
 *     of its work onto a library stream and joins it back through events: one
 *     stream and two events per host thread and device, created by the first
 *     call that is not being stream-captured and kept until the process ends
 *     (cudaDeviceReset invalidates them; later backward calls on that thread
 *     and device then return TWELL_ERR_CUDA).
 *   - Host-side argument errors are returned at once and nothing is enqueued.
 *     Errors found on the device (capacity, bounded-wait timeout) are written
 *     to `*status`, a caller-owned device int32 that the caller sets to 0
 *     before the first call; the first nonzero code sticks and later kernels of
 *     the same call skip their work. Read it after synchronising the stream, or
 *     with twell_check().
 *   - Alignment: every device pointer of a bf16 matrix must be 16-byte aligned
 *     and d, F must be multiples of 8 (128-bit loads, TMA strides).
 *   - All calls are deterministic: the same inputs give the same bits.
 */
#ifndef TWELL_H
#define TWELL_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum twell_status {
    TWELL_OK = 0,
    TWELL_ERR_INVALID_ARG = 1, /* null pointer, non-positive size, misaligned pointer, bad d/F */
    TWELL_ERR_UNSUPPORTED = 2, /* shape or mode this build does not implement */
    TWELL_ERR_WORKSPACE = 3,   /* ws_bytes smaller than twell_workspace_bytes() */
    TWELL_ERR_CAPACITY = 4,    /* device: TwELL needs more slots than cap_slots */
    TWELL_ERR_TIMEOUT = 5,     /* device: a bounded wait inside a kernel expired */
    TWELL_ERR_CUDA = 6         /* a CUDA runtime call or launch failed */
} twell_status;

/* Host struct describing one TwELL held in device memory (layout above).
 * M, F, T, n_tiles = ceil(M/T) and cap_slots are set by the caller; the five
 * device arrays are caller-allocated: nnz_row[M], K_tile[n_tiles],
 * tile_off[n_tiles+1], idx[cap_slots], val[cap_slots]. */
typedef struct twell_buf {
    int32_t M, F, T, n_tiles;
    int64_t cap_slots;
    int32_t* nnz_row;
    int32_t* K_tile;
    int64_t* tile_off;
    int32_t* idx;
    uint16_t* val;
} twell_buf;

/* Element types of the tensors that take more than one. */
typedef enum twell_dtype { TWELL_BF16 = 0, TWELL_F32 = 1 } twell_dtype;

/* Operation codes for twell_workspace_bytes. */
enum { TWELL_OP_PACK = 0, TWELL_OP_SPMM_DOWN = 1, TWELL_OP_FFN_FWD = 2,
       TWELL_OP_FFN_BWD = 3, TWELL_OP_GATED_FWD = 4, TWELL_OP_HYBRID_FWD = 5 };

/* Human-readable name of a status code (static string, never NULL). */
const char* twell_status_string(int status);

/* Worst-case slot count of a TwELL of an M x F matrix with tile height T:
 * M*F (every entry active). Returns -1 for non-positive sizes. */
int64_t twell_buf_slots_bound(int M, int F, int T);

/* Device workspace, in bytes, that `op` needs for these sizes. cap_slots is the
 * TwELL capacity (used by TWELL_OP_FFN_BWD and TWELL_OP_GATED_FWD). 0 means
 * none is needed. */
size_t twell_workspace_bytes(int op, int M, int d, int F, int T, int64_t cap_slots);

/*
 * twell_fwd_workspace_bytes — workspace of the ReLU forward (twell_up_pack /
 * twell_ffn_fwd without a gate) whose up-projection epilogue stages at most
 * stage_cap nonzeros per (row, 256-column block): the capacity the method
 * predicts for N_nz (Resumo Técnico §2, "Formato Híbrido para Treinamento").
 * stage_cap is 256, 64 or 32 (the capacities the epilogue is compiled for);
 * 256 never overflows and equals twell_workspace_bytes(TWELL_OP_FFN_FWD, ...).
 * The forward uses the largest of them its ws_bytes allows; a block with more
 * nonzeros than that makes the call report TWELL_ERR_CAPACITY. Returns 0 for
 * invalid arguments.
 */
size_t twell_fwd_workspace_bytes(int M, int d, int F, int T, int64_t cap_slots, int stage_cap);

/* Number of streaming multiprocessors the library sizes its grids for. */
int twell_device_sm_count(void);

/*
 * twell_pack — TwELL of a dense hidden matrix (the "Formato de Dados TwELL"
 * paragraph of Resumo Técnico §2).
 *   h      [M, ldh] bf16, entries (r, j < F) are read; ldh >= F, ldh % 8 == 0
 *   out    host struct with out->M == M, out->F == F, out->T == T
 * Writes nnz_row, K_tile, tile_off always; writes the slots only if
 * tile_off[n_tiles] <= cap_slots, else sets *status = TWELL_ERR_CAPACITY.
 */
twell_status twell_pack(const uint16_t* h, int M, int F, int ldh, int T,
                        const twell_buf* out, int32_t* status, void* stream);

/*
 * twell_up_pack — rows a1-a3 of the forward alone: the tcgen05 up (or gate)
 * projection whose epilogue packs h into h_out, without the down-projection.
 * Same arguments, workspace and error behaviour as twell_ffn_fwd minus W_down
 * and y; in gated mode h_out's val holds h = bf16(relu(g) * u) on return.
 * twell_ffn_fwd is exactly twell_up_pack followed by twell_spmm_down.
 */
twell_status twell_up_pack(const uint16_t* x, const uint16_t* W_up, const uint16_t* W_gate,
                           const float* b, int M, int d, int F, int T, const twell_buf* h_out,
                           void* ws, size_t ws_bytes, int32_t* status, void* stream);

/*
 * twell_spmm_down — y = h W_down over the stored entries of a TwELL (Resumo
 * Técnico §2, "Kernels de Inferência": iterate only over the active neurons).
 *   h       host struct of a valid TwELL (F rows of W_down are indexed)
 *   W_down  [F, d] bf16
 *   y       [M, d] bf16 output; fp32 accumulation, one rounding to bf16
 */
twell_status twell_spmm_down(const twell_buf* h, const uint16_t* W_down, int d,
                             uint16_t* y, int32_t* status, void* stream);

/*
 * twell_spmm_down_tc — the same product y = h W_down on the tensor cores
 * (Resumo Técnico §2, "Kernels de Inferência": only the active neurons are
 * visited and the tensor cores do the multiplication). For each group of 128
 * consecutive tokens, U is the ascending union of their active units; then
 * y[group] = h[group, U] W_down[U, :] runs as one tcgen05 GEMM with K = |U|
 * (A built in shared memory from the TwELL, B the gathered rows of W_down).
 * Same arguments, result and error behaviour as twell_spmm_down, plus:
 *   ws        device workspace of at least
 *             twell_spmm_down_tc_workspace_bytes(h->M, h->F, h->cap_slots)
 *             bytes, 256-byte aligned; contents are scratch
 * h->F must be a multiple of 8 and at most 65536, and the device must offer
 * the kernel's shared memory (about 227 KB per block; else
 * TWELL_ERR_UNSUPPORTED). y equals twell_spmm_down's up to fp32 summation
 * order. Launches two kernels: the groups' unions and entry buckets, then the
 * GEMM.
 */
size_t twell_spmm_down_tc_workspace_bytes(int M, int F, int64_t cap_slots);
twell_status twell_spmm_down_tc(const twell_buf* h, const uint16_t* W_down, int d, uint16_t* y,
                                void* ws, size_t ws_bytes, int32_t* status, void* stream);

/*
 * twell_ffn_fwd — the layer's forward pass.
 *   ReLU  (W_gate == NULL): h = relu(x W_up^T + b), packed into TwELL inside the
 *          tcgen05 up-projection's epilogue (Resumo Técnico §2: TwELL materialised
 *          in the epilogue of the dense matmul), then y = h W_down.
 *   Gated (W_gate != NULL): the gate GEMM x W_gate^T + b gives the active set and
 *          is packed the same way; then for each active (r, j):
 *          u = x[r] . W_up[j], h = bf16(relu(g) * u), y[r] += h W_down[j] (the
 *          sparse up+down inference kernels of the same section).
 *   x [M, d] bf16; W_up, W_gate, W_down [F, d] bf16; b [F] fp32 (added to the
 *   ReLU pre-activation, or to the gate); y [M, d] bf16.
 *   h_out: TwELL of h (M, F, T as given), its val holding h.
 *   ws: device workspace of at least twell_workspace_bytes(TWELL_OP_FFN_FWD or
 *   TWELL_OP_GATED_FWD, M, d, F, T, h_out->cap_slots) bytes, 256-byte aligned;
 *   contents need no init.
 * Capacity overflow of h_out: nnz/K/off are written, slots and y are not, and
 * *status = TWELL_ERR_CAPACITY.
 */
twell_status twell_ffn_fwd(const uint16_t* x, const uint16_t* W_up, const uint16_t* W_gate,
                           const float* b, const uint16_t* W_down, int M, int d, int F, int T,
                           const twell_buf* h_out, uint16_t* y, void* ws, size_t ws_bytes,
                           int32_t* status, void* stream);

/*
 * Hybrid format (Resumo Técnico §2, "Formato Híbrido para Treinamento"): rows
 * are partitioned dynamically; a row with more than C nonzeros is an overflow
 * row and goes to a dense backup matrix, every other row stays in the TwELL.
 * Overflow rows are empty rows of the TwELL (nnz 0), so every TwELL entry point
 * applies to the TwELL part unchanged.
 *   C         ELL capacity per row, >= 0
 *   cap_rows  rows the dense block can hold, >= 0
 *   n_rows    [1] int32 device, written: number of overflow rows
 *   rows      [cap_rows] int32 device, written: overflow row ids, ascending
 *   dense     [cap_rows, F] bf16 device, written: row i is the hidden row of
 *             rows[i] (all F columns, zeros included)
 * More than cap_rows overflow rows: *status = TWELL_ERR_CAPACITY and the first
 * cap_rows are kept. All arrays are caller-owned.
 */
typedef struct {
    int32_t C;
    int32_t cap_rows;
    int32_t* n_rows;
    int32_t* rows;
    uint16_t* dense;
} twell_overflow;

/*
 * twell_hybrid_up_pack — ReLU up-projection (as twell_up_pack) packed into the
 * hybrid format: h_out holds the rows with nnz <= ov->C, ov the others.
 *   x [M, d] bf16; W_up [F, d] bf16; b [F] fp32; ws: at least
 *   twell_workspace_bytes(TWELL_OP_HYBRID_FWD, M, d, F, T, 0) bytes,
 *   256-byte aligned.
 */
twell_status twell_hybrid_up_pack(const uint16_t* x, const uint16_t* W_up, const float* b, int M, int d, int F,
                                  int T, const twell_buf* h_out, const twell_overflow* ov, void* ws,
                                  size_t ws_bytes, int32_t* status, void* stream);

/*
 * twell_hybrid_spmm_down — y = h W_down on the hybrid format: the TwELL rows by
 * the sparse down-projection (twell_spmm_down), the overflow rows by the
 * tcgen05 dense GEMM on ov->dense, its output rows placed by ov->rows.
 *   W_down [F, d] bf16 (rows gathered by the TwELL part); W_downT [d, F] bf16,
 *   the same matrix transposed (the dense GEMM's K-major operand); y [M, d]
 *   bf16, every row written.
 */
twell_status twell_hybrid_spmm_down(const twell_buf* h, const twell_overflow* ov, const uint16_t* W_down,
                                    const uint16_t* W_downT, int d, uint16_t* y, int32_t* status, void* stream);

/* twell_hybrid_ffn_fwd — twell_hybrid_up_pack followed by twell_hybrid_spmm_down. */
twell_status twell_hybrid_ffn_fwd(const uint16_t* x, const uint16_t* W_up, const float* b, const uint16_t* W_down,
                                  const uint16_t* W_downT, int M, int d, int F, int T, const twell_buf* h_out,
                                  const twell_overflow* ov, uint16_t* y, void* ws, size_t ws_bytes,
                                  int32_t* status, void* stream);

/*
 * twell_hybrid_ffn_bwd — the backward of twell_ffn_bwd (same loss, outputs,
 * layouts and determinism) for a layer whose forward ran on the hybrid format
 * (Resumo Técnico §2, "Formato Híbrido para Treinamento"): the TwELL rows of h
 * through the sparse kernels, the dense overflow rows of ov through tcgen05
 * GEMMs (dpre of those rows masked by their h, dx rows, and their shares of
 * dW_up, dW_down and db added to the sparse part's).
 *   W_upT [d, F] bf16: W_up transposed (K-major operand of the dense dx).
 *   ws: at least twell_hybrid_bwd_workspace_bytes(M, d, F, T, h->cap_slots,
 *   ov->cap_rows) bytes, 256-byte aligned. Limits as twell_ffn_bwd.
 * The overflow rows' dpre enters the GEMMs as the sum of two bf16 parts
 * (~2^-17 relative), accumulated in fp32.
 */
size_t twell_hybrid_bwd_workspace_bytes(int M, int d, int F, int T, int64_t cap_slots, int cap_rows);
twell_status twell_hybrid_ffn_bwd(const uint16_t* x, const uint16_t* W_up, const uint16_t* W_down,
                                  const uint16_t* W_upT, const twell_buf* h, const twell_overflow* ov,
                                  const uint16_t* dy, int d, float l1_coef, uint16_t* dx, float* dW_up,
                                  float* dW_down, float* db, void* ws, size_t ws_bytes, int32_t* status,
                                  void* stream);

/*
 * twell_ffn_bwd — backward of L = <dy, y> + l1_coef * sum |h| for the ReLU
 * layer (Resumo Técnico §2, "Técnicas de Treinamento": L1 on the ReLU
 * activations), restricted to the stored entries of h:
 *   dpre[r,j] = (dy[r] . W_down[j] + l1_coef) on active (r, j), 0 elsewhere
 *   dx        = dpre W_up                       [M, d] bf16
 *   dW_up     = dpre^T x                        [F, d] fp32 (every row written)
 *   dW_down   = h^T dy                          [F, d] fp32 (every row written)
 *   db        = column sums of dpre             [F]    fp32
 *   x, dy [M, d] bf16; W_up, W_down [F, d] bf16; M and F are h->M and h->F.
 *   h: the forward's TwELL; ws: at least twell_workspace_bytes(TWELL_OP_FFN_BWD,
 *   M, d, F, T, h->cap_slots) bytes, 256-byte aligned (it grows with d: the
 *   dot products of dpre are summed over column slices of 1024, one fp32 per
 *   stored slot and slice). Limit of this build: h->cap_slots < 2^31 (else
 *   TWELL_ERR_UNSUPPORTED).
 * The reduction order of every sum is fixed (no floating-point atomics).
 * The column lists' index-only kernels run on the library's side stream while
 * the SDDMM runs on `stream`; the call's work is complete when `stream`'s is.
 */
twell_status twell_ffn_bwd(const uint16_t* x, const uint16_t* W_up, const uint16_t* W_down,
                           const twell_buf* h, const uint16_t* dy, int d, float l1_coef,
                           uint16_t* dx, float* dW_up, float* dW_down, float* db,
                           void* ws, size_t ws_bytes, int32_t* status, void* stream);

/*
 * twell_dense_ffn_fwd — the same ReLU layer computed densely with the same
 * tcgen05 GEMM (a baseline for the sparse path, not part of the method):
 *   h_dense = bf16(relu(x W_up^T + b))   [M, F] bf16 (written; the dense
 *                                        backward's mask)
 *   y       = h_dense W_down             [M, d] bf16
 * Every argument has the layout of twell_ffn_fwd's; W_down [F, d] is read as
 * the MN-major operand of the second GEMM (no transposed copy). All pointers
 * 16-byte aligned; d % 8 == 0, F % 8 == 0. Runs on CTA pairs (TWELL_ERR_CUDA
 * if a cluster of two cannot be launched).
 */
twell_status twell_dense_ffn_fwd(const uint16_t* x, const uint16_t* W_up, const float* b,
                                 const uint16_t* W_down, int M, int d, int F,
                                 uint16_t* h_dense, uint16_t* y, int32_t* status, void* stream);

/*
 * twell_dense_ffn_bwd — backward of the dense baseline layer, the loss and
 * gradients of twell_ffn_bwd (L = <dy, y> + l1_coef * sum |h|) computed with
 * dense tcgen05 GEMMs (a baseline, not part of the method):
 *   dpre    = bf16((dy W_down^T + l1_coef) * 1[h_dense != 0])  [M, F] (workspace)
 *   db      = sum over rows of the fp32 values before that rounding
 *   dx      = dpre W_up          [M, d] bf16
 *   dW_up   = dpre^T x           [F, d] fp32
 *   dW_down = h_dense^T dy       [F, d] fp32
 * dpre is a bf16 GEMM operand, as in a bf16 training step. The token axis is
 * the inner dimension of the two weight-gradient GEMMs: x, dy, dpre and
 * h_dense are read as MN-major operands, so nothing is transposed.
 *   h_dense: the forward's [M, F] bf16 hidden matrix (twell_dense_ffn_fwd).
 *   ws: at least twell_dense_bwd_workspace_bytes(M, d, F) bytes, 256-byte
 *   aligned (dpre and per-128-row column sums of it).
 * All pointers 16-byte aligned; d % 8 == 0, F % 8 == 0. Fixed summation order
 * (no atomics). Runs on CTA pairs (TWELL_ERR_CUDA if a cluster of two cannot
 * be launched).
 */
size_t twell_dense_bwd_workspace_bytes(int M, int d, int F);
twell_status twell_dense_ffn_bwd(const uint16_t* x, const uint16_t* W_up, const uint16_t* W_down,
                                 const uint16_t* h_dense, const uint16_t* dy, int M, int d, int F,
                                 float l1_coef, uint16_t* dx, float* dW_up, float* dW_down, float* db,
                                 void* ws, size_t ws_bytes, int32_t* status, void* stream);

/*
 * twell_ffn_fwd_static_ws — twell_ffn_fwd for callers that cannot allocate
 * device memory. The paper has no counterpart; this is a convenience of this
 * library. It is meant for code that has no allocator to call (a plugin inside
 * a host framework that owns all device memory) or must not call one (a
 * latency-critical decode loop, where cudaMalloc/cudaFree synchronise the
 * device). Same arguments and results as twell_ffn_fwd, without ws/ws_bytes:
 * the workspace is a library-owned device array of TWELL_STATIC_WS_BYTES that
 * every GPU which loads the library keeps until the process exits.
 *   - Returns TWELL_ERR_WORKSPACE, with nothing enqueued, when the problem
 *     needs more workspace than the array holds: gated, when
 *     twell_workspace_bytes(TWELL_OP_GATED_FWD, M, d, F, T, h_out->cap_slots)
 *     > TWELL_STATIC_WS_BYTES; ReLU, when even the smallest epilogue staging
 *     (twell_fwd_workspace_bytes(M, d, F, T, h_out->cap_slots, 32)) does not
 *     fit. A ReLU call that fits runs with the largest staging capacity (256,
 *     64 or 32 entries per row and 256-column block) the array holds, and a
 *     block with more active units than that reports TWELL_ERR_CAPACITY in
 *     *status. Decode shapes such as M <= 64, d_model = 4096, d_ff = 14336
 *     fit in both modes, and so does the ReLU layer at M = 4096, d_model =
 *     2048, d_ff = 8192 (32-entry staging).
 *   - The first call on a device looks up the array's device address on that
 *     device (cudaGetSymbolAddress) and keeps it for the life of the process;
 *     make that first call before any stream capture. The kept address is
 *     that of the device's current context: after cudaDeviceReset on a device,
 *     do not call this entry point on it again.
 *   - All calls on a device share the one array, which keeps the last call's
 *     contents: calls whose work overlaps on the GPU (different streams, or
 *     different host threads, without ordering between them) race on it and
 *     corrupt each other's results. Serialise them, e.g. on one stream.
 *   - The allocation-free guarantee covers this call only; the caller still
 *     owns x, the weights, b, y, h_out's arrays and status.
 */
#define TWELL_STATIC_WS_BYTES (32u * 1024u * 1024u)
twell_status twell_ffn_fwd_static_ws(const uint16_t* x, const uint16_t* W_up, const uint16_t* W_gate,
                                     const float* b, const uint16_t* W_down, int M, int d, int F, int T,
                                     const twell_buf* h_out, uint16_t* y, int32_t* status, void* stream);

/*
 * Layer norm around the feed-forward layer. Rows of d elements; row strides
 * (ld*) in elements, >= d, of any alignment (rows that all start on 16-byte
 * boundaries are read in 16-byte pieces, others in pairs or single elements). x_type is the type of the residual stream
 * (x, res, sum, dres, dx), y_type that of y and dy, w_type that of w and b; each
 * TWELL_BF16 or TWELL_F32. w or b may be NULL (1 and 0). N >= 0, d >= 1. Limit of
 * this build: d <= 2^29 (TWELL_ERR_UNSUPPORTED).
 * Statistics and sums are fp32; outputs are rounded once. Outputs must not
 * overlap inputs (the call rejects equal pointers).
 *
 * twell_layernorm_fwd
 *   s    = x + res, rounded to x_type and written to sum (res and sum both NULL: s = x)
 *   mean = mean of the row of s, rstd = 1 / sqrt(variance + eps) (biased variance)
 *   y    = (s - mean) rstd w + b
 *   mean, rstd [N] fp32 (the backward's inputs); both may be NULL.
 */
twell_status twell_layernorm_fwd(const void* x, int64_t ldx, const void* res, int64_t ldres, const void* w,
                                 const void* b, int64_t N, int d, float eps, int x_type, int y_type, int w_type,
                                 void* sum, int64_t ldsum, void* y, int64_t ldy, float* mean, float* rstd,
                                 void* stream);

/*
 * twell_layernorm_bwd — with hat = (x - mean) rstd and v = w dy:
 *   dx = rstd (v - mean(v) - hat mean(v hat)) + dres   (dres NULL: 0)
 *   dw = sum over rows of dy hat, db = sum over rows of dy   [d] fp32
 *   x: the forward's normalised rows (its sum, if there was a residual); mean,
 *   rstd: the forward's. dw and db may both be NULL. The rows are summed in a
 *   fixed order (no atomics).
 *   ws: at least twell_layernorm_bwd_workspace_bytes(N, d) bytes, 256-byte aligned.
 */
size_t twell_layernorm_bwd_workspace_bytes(int64_t N, int d);
twell_status twell_layernorm_bwd(const void* dy, int64_t lddy, const void* x, int64_t ldx, const void* w,
                                 const float* mean, const float* rstd, const void* dres, int64_t lddres, int64_t N,
                                 int d, int x_type, int y_type, int w_type, void* dx, int64_t lddx, float* dw,
                                 float* db, void* ws, size_t ws_bytes, void* stream);

/*
 * Softmax cross entropy of a linear head over a vocabulary of V words:
 *   z = x W^T, lse_r = log sum_j exp z_rj, nll_r = lse_r - z_r,target(r),
 *   loss = sum of nll over the scored rows, or with mean != 0 their mean.
 * Rows whose target is ignore_index are not scored: their nll, lse and dx are 0
 * and they take no part in dW, whatever x holds there. No scored row: loss 0,
 * zero gradients. A target outside [0, V) that is not ignore_index sets
 * *status = TWELL_ERR_INVALID_ARG and the outputs are then unspecified.
 *   x [N, d] bf16, W [V, d] bf16 (one row per word), target [N] int64;
 *   nll, lse [N] fp32, loss [1] fp32. N >= 0, V >= 1, d % 8 == 0. Limit of this
 *   build: N, d, V <= 2^30 (TWELL_ERR_UNSUPPORTED).
 * A logit is an fp32 sum: the tensor cores', which drop what does not fit towards
 * zero, over 512 of d at a time, joined with rounding.
 * The logits are never stored: twell_xent_fwd keeps a maximum and a sum for
 * every (row, 128 words), and the scored rows of x copied together.
 *
 * twell_xent_fwd_bwd also gives the gradients of grad_scale * loss:
 *   dz_rj = g (exp(z_rj - lse_r) - [j = target(r)]), g = grad_scale (/ scored rows)
 *   dx = dz W [N, d] bf16; dW = dz^T x [V, d], bf16 or fp32 (dw_type); with
 *   accumulate != 0 (fp32 only) dW += dz^T x.
 * dz enters the products as a bf16 operand (like any operand of the tensor
 * cores); sums are fp32. The rows are worked through chunk_rows at a time (0: all
 * at once); a chunk keeps 2 bytes per (row, word) in the workspace, and a bf16
 * dW over several chunks 4 bytes per (word, d).
 *   ws: at least twell_xent_fwd_workspace_bytes(N, d, V), or
 *   twell_xent_bwd_workspace_bytes(N, d, V, chunk_rows, dw_type), 256-byte
 *   aligned. Runs on CTA pairs (TWELL_ERR_CUDA if a cluster of two cannot be
 *   launched).
 */
size_t twell_xent_fwd_workspace_bytes(int N, int d, int V);
size_t twell_xent_bwd_workspace_bytes(int N, int d, int V, int chunk_rows, int dw_type);
twell_status twell_xent_fwd(const uint16_t* x, const uint16_t* W, const int64_t* target, int N, int d, int V,
                            int64_t ignore_index, int mean, float* nll, float* lse, float* loss, void* ws,
                            size_t ws_bytes, int32_t* status, void* stream);
twell_status twell_xent_fwd_bwd(const uint16_t* x, const uint16_t* W, const int64_t* target, int N, int d, int V,
                                int64_t ignore_index, int mean, float grad_scale, int chunk_rows, float* nll,
                                float* lse, float* loss, uint16_t* dx, void* dW, int dw_type, int accumulate,
                                void* ws, size_t ws_bytes, int32_t* status, void* stream);

/*
 * twell_grad_clip — L2 norm over many tensors, and the tensors scaled so that it
 * is at most max_norm:
 *   norm = sqrt(sum of g^2 over all elements), c = min(1, max_norm / norm),
 *   out = c g, rounded once to the tensor's type.
 * out[i] may be in[i] (then nothing is written while c = 1) or a tensor that
 * overlaps no input. max_norm >= 0; c = 1 where norm <= max_norm (both 0 included).
 * INFINITY gives the norm alone (in place; copies otherwise), whatever the norm is.
 * With a finite bound a NaN norm makes every element NaN, and an infinite element
 * makes the finite ones 0. The norm is a 64-bit sum: finite elements whose norm
 * passes fp32's range are scaled as others are, and *norm is infinite.
 *   list: host struct of host arrays (read during the call): n tensors, device
 *   addresses, element counts (>= 0) and twell_dtype codes; tensors are
 *   contiguous and aligned to their element size. norm [1] fp32 device.
 *   ws: at least twell_grad_clip_workspace_bytes() bytes, 256-byte aligned.
 *   Limit of this build: 32768 tensors (TWELL_ERR_UNSUPPORTED).
 */
typedef struct twell_tensor_list {
    int32_t n;
    const void* const* in;
    void* const* out;
    const int64_t* numel;
    const int32_t* type;
} twell_tensor_list;
size_t twell_grad_clip_workspace_bytes(void);
twell_status twell_grad_clip(const twell_tensor_list* list, float max_norm, float* norm, void* ws, size_t ws_bytes,
                             void* stream);

/*
 * Linear layer with bias, activation and residual, and its backward:
 *   pre = x W^T + bias, y = act(pre) + res
 *   dpre = dy act'(pre), dx = dpre W, dW = dpre^T x, dbias = column sums of dpre
 * x [M, K] bf16; W bf16, [N, K] (w_kn 0) or [K, N] (w_kn 1: x W), densely packed;
 * bias [N] fp32 or NULL; act a twell_activation; res [M, N] of y's type or NULL;
 * y [M, N] bf16 or fp32 (y_type); pre [M, N] bf16 or NULL (kept for the backward).
 * Row strides (ld*) in elements. x: a multiple of 8, <= 2^30, 16-byte aligned; y, res, pre,
 * dy, dx: any that is at least the width, of any alignment (16-byte boundaries are
 * fastest). M >= 0, N >= 1, K % 8 == 0; with w_kn N % 8 == 0. Limit of this build:
 * M, N, K <= 2^30 (TWELL_ERR_UNSUPPORTED). y may be res, with the same row stride;
 * otherwise outputs and ws must not overlap inputs or one another (the calls reject
 * equal pointers, and y = res with another stride).
 * Sums are fp32, the tensor cores', which drop what does not fit towards zero, over at
 * most 512 of depth for fp32 results and 16384 for bf16 ones, joined with rounding;
 * outputs are rounded once.
 *
 * twell_linear_bwd: dy [M, N] bf16; pre as the forward kept it (NULL if act is
 * TWELL_ACT_NONE). dx [M, K] bf16; dW in W's layout, bf16 or fp32 (dw_type), with
 * accumulate != 0 (fp32 only) added to what is there; dbias [N] fp32. Each of the
 * three may be NULL, not all; a gradient's bits do not depend on which others are
 * asked for. With an activation dpre enters the products rounded
 * to bf16, like any operand of the tensor cores; dbias sums it in fp32.
 *   ws: at least twell_linear_bwd_workspace_bytes(M, N, K) bytes, 256-byte aligned.
 * M = 0: dW and dbias are 0 (dW unchanged with accumulate).
 * Large batches run on CTA pairs (TWELL_ERR_CUDA if a cluster of two cannot be
 * launched).
 */
enum twell_activation { TWELL_ACT_NONE = 0, TWELL_ACT_RELU = 1, TWELL_ACT_SILU = 2, TWELL_ACT_GELU = 3,
                        TWELL_ACT_GELU_TANH = 4 };
twell_status twell_linear_fwd(const uint16_t* x, int64_t ldx, const uint16_t* W, int w_kn, const float* bias, int act,
                              const void* res, int64_t ldres, int M, int N, int K, uint16_t* pre, int64_t ldpre,
                              void* y, int64_t ldy, int y_type, int32_t* status, void* stream);
size_t twell_linear_bwd_workspace_bytes(int M, int N, int K);
twell_status twell_linear_bwd(const uint16_t* dy, int64_t lddy, const uint16_t* x, int64_t ldx, const uint16_t* W,
                              int w_kn, int act, const uint16_t* pre, int64_t ldpre, int M, int N, int K, uint16_t* dx,
                              int64_t lddx, void* dW, int dw_type, int accumulate, float* dbias, void* ws,
                              size_t ws_bytes, int32_t* status, void* stream);

/*
 * The gated feed-forward layer computed densely, forward and backward. With act =
 * TWELL_ACT_RELU it is the layer that twell_ffn_fwd serves sparsely with W_gate.
 *   g = x W_gate^T + b, u = x W_up^T, h = act(g) u, y = h W_down + res
 *   L = <dy, y> + l1_coef sum |h|:
 *   dh = dy W_down^T + l1_coef sign(act(g) u), dg = dh u act'(g), du = dh act(g)
 *   dx = dg W_gate + du W_up, dW_gate = dg^T x, dW_up = du^T x, dW_down = h^T dy,
 *   db = column sums of dg
 * x, y, res, dy, dx [M, d] bf16; W_* [F, d] bf16; b, db [F] fp32 or NULL; g, u, h
 * [M, F] bf16; res may be NULL, or y itself. The forward writes h, and g and u unless
 * both are NULL (only a backward reads them); h is formed from the unrounded g and u,
 * y from h as stored. Everything is densely packed; d, F multiples of 8, M >= 0.
 * Apart from res, outputs and ws must not overlap inputs or one another (the calls
 * reject equal pointers).
 * Limit of this build: M, d, F <= 2^30 (TWELL_ERR_UNSUPPORTED).
 * Backward: dg and du enter the products rounded to bf16, db sums dg in fp32. dW_*
 * bf16 or fp32 (dw_type), with accumulate != 0 (fp32 only) added to what is there; the
 * three may all be NULL, and so may dx and db, but not everything; a gradient's bits
 * do not depend on which others are asked for.
 *   ws: at least twell_dense_gated_bwd_workspace_bytes(M, d, F) bytes, 256-byte aligned.
 * M = 0: dW_* and db are 0 (dW_* unchanged with accumulate). Large batches run on CTA
 * pairs (TWELL_ERR_CUDA if a cluster of two cannot be launched).
 */
twell_status twell_dense_gated_ffn_fwd(const uint16_t* x, const uint16_t* W_gate, const uint16_t* W_up, const float* b,
                                       const uint16_t* W_down, int act, const uint16_t* res, int M, int d, int F,
                                       uint16_t* g, uint16_t* u, uint16_t* h, uint16_t* y, int32_t* status,
                                       void* stream);
size_t twell_dense_gated_bwd_workspace_bytes(int M, int d, int F);
twell_status twell_dense_gated_ffn_bwd(const uint16_t* x, const uint16_t* W_gate, const uint16_t* W_up,
                                       const uint16_t* W_down, int act, const uint16_t* g, const uint16_t* u,
                                       const uint16_t* h, const uint16_t* dy, float l1_coef, int M, int d, int F,
                                       uint16_t* dx, void* dW_gate, void* dW_up, void* dW_down, int dw_type,
                                       int accumulate, float* db, void* ws, size_t ws_bytes, int32_t* status,
                                       void* stream);

/*
 * twell_adamw — one step of Adam with decoupled weight decay over many tensors:
 *   c = norm > max_norm ? max_norm / norm : 1,  g' = c g
 *   m = beta1 m + (1 - beta1) g',  v = beta2 v + (1 - beta2) g'^2
 *   param -= lr (m / (1 - beta1^t) / (sqrt(v / (1 - beta2^t)) + eps) + weight_decay param)
 * lr [1] fp32 and step [1] int32 (t, 1 for the first step) are read on the device, so
 * that a captured call follows them; norm [1] fp32 as twell_grad_clip writes it (with
 * an infinite bound), or NULL: c = 1. Gradients are read only. With a norm that is not
 * finite, or a step below 1, the call changes nothing, and *norm, which the caller
 * holds, is the only sign of it. That drops the step of finite gradients whose norm
 * passes fp32's range (2^128) too; twell_grad_clip with a finite bound scales those,
 * after which norm = NULL takes the step. beta1, beta2 in [0, 1), eps >= 2^-126, weight_decay >= 0.
 * The list is a host struct of host arrays (read during the call): n tensors, device
 * addresses, element counts (>= 0). param and grad bf16 or fp32 (twell_dtype codes);
 * copy (the array or any entry may be NULL): a bf16 copy of an fp32 param. Tensors are
 * contiguous and aligned to their element size; no tensor overlaps another.
 * state_bits 32: m, v [numel] fp32. state_bits 8: m, v [numel] uint8 codes and m_scale,
 * v_scale [ceil(numel / 256)] fp32, each the power of two that TWELL_ADAMW_BLOCK
 * consecutive elements share. A code is s eeee fff (m) or eeeee fff (v):
 *   scale 2^(e - 2^E) (1 + f / 8), or scale 2^(1 - 2^E) f / 8 for e = 0   (E = 4, 5)
 * All zeros, codes and scales, are the states before the first step. Codes are rounded
 * up or down so that their mean is the value, and so is a bf16 param; a v above 0 never
 * becomes 0. The random bits are a function of (seed, step, tensor's place in the list,
 * element) alone. A block with a value that is not finite, or above 15/16 2^127, has a NaN scale.
 * Limits of this build: 32768 tensors (TWELL_ERR_UNSUPPORTED).
 *
 * twell_adamw_values — the values that 8-bit states stand for, to the out tensors of
 * two lists (bf16, where every one is exact while it is in range, or fp32) with the
 * list's element counts: to save, inspect or convert them.
 */
#define TWELL_ADAMW_BLOCK 256
typedef struct twell_adamw_list {
    int32_t n;
    int32_t state_bits;
    void* const* param;
    const void* const* grad;
    void* const* m;
    void* const* v;
    float* const* m_scale; /* state_bits 8 only, else ignored */
    float* const* v_scale;
    void* const* copy;
    const int64_t* numel;
    const int32_t* param_type;
    const int32_t* grad_type;
} twell_adamw_list;
twell_status twell_adamw(const twell_adamw_list* list, const float* lr, const int32_t* step, double beta1, double beta2,
                         double eps, double weight_decay, const float* norm, float max_norm, uint64_t seed,
                         void* stream);
twell_status twell_adamw_values(const twell_adamw_list* list, const twell_tensor_list* m_out,
                                const twell_tensor_list* v_out, void* stream);

/*
 * twell_set_kernel_timer — measurement hook. While set, every launch of the
 * kernel at call site `site` is bracketed by cudaEventRecord(ev_begin) and
 * cudaEventRecord(ev_end) on the launch's stream; ev_begin/ev_end are
 * caller-created cudaEvent_t handles passed as void*. site = 0 (or NULL
 * events) turns the hook off. Process-wide setting, not thread-safe: set it
 * from the thread that launches. Sites:
 *   1 up-projection GEMM (twell_up_pack / twell_ffn_fwd)
 *   2 sparse down-projection (twell_spmm_down / twell_ffn_fwd)
 *   3 backward SDDMM            4 backward dx
 *   5 backward column lists: the kernels that read only the TwELL indices
 *     (on the library's side stream, concurrently with the SDDMM)
 *   6 backward weight gradients
 *   7 gated decode tail (M <= 64: layout, gated up products and, in
 *     twell_ffn_fwd, the down-projection, in one launch)
 *   8 dense GEMM of the hybrid format's overflow rows (twell_hybrid_spmm_down)
 *   9 union down-projection on the tensor cores (twell_spmm_down_tc, both kernels)
 *  10 its first kernel alone (the groups' unions and entry buckets)
 */
enum { TWELL_SITE_NONE = 0, TWELL_SITE_UP_GEMM = 1, TWELL_SITE_SPMM_DOWN = 2, TWELL_SITE_SDDMM = 3,
       TWELL_SITE_DX = 4, TWELL_SITE_CSC = 5, TWELL_SITE_WGRAD = 6, TWELL_SITE_DECODE_TAIL = 7,
       TWELL_SITE_OVERFLOW_GEMM = 8, TWELL_SITE_SPMM_UNION = 9, TWELL_SITE_UNION_BUILD = 10 };
twell_status twell_set_kernel_timer(int site, void* ev_begin, void* ev_end);

/*
 * twell_wait_selftest — diagnostic of the library's bounded waits: runs a
 * wait that nothing will complete, with the same helpers the kernels use
 * (which = 0: an mbarrier no thread arrives on; which = 1: the decode tail's
 * grid barrier with a target the grid cannot reach). After its limit (about
 * one second) the wait gives up and writes TWELL_ERR_TIMEOUT to *status
 * (first error sticks); the CUDA context stays usable.
 *   scratch: one int32 of device memory (zeroed by the call).
 * Asynchronous on `stream`; TWELL_ERR_INVALID_ARG for another `which` or null
 * pointers.
 */
twell_status twell_wait_selftest(int which, int32_t* scratch, int32_t* status, void* stream);

/* Number of kernels this library has launched in this process (host-side
 * counter, all devices). Lets a caller count the library's launches in a
 * timed region. */
int64_t twell_kernel_launches(void);

/*
 * twell_check — synchronises `stream`, copies *status (device) to
 * *host_status (host) and returns TWELL_OK, or TWELL_ERR_CUDA if the stream
 * reported an error. This is the one entry point that synchronises.
 */
twell_status twell_check(const int32_t* status, void* stream, int32_t* host_status);

#ifdef __cplusplus
}
#endif

#endif /* TWELL_H */
