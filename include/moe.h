/*
 * moe.h -- C ABI of the MI355X (gfx950) forward pass of one Mixture-of-Experts layer.
 *
 * One layer call computes, for T tokens x[t] (hidden size d), E routed experts
 * (SwiGLU, FFN size f) and top-k routing:
 *
 *   l[t,e]   = x[t] . Wg[e] + bias[e]                      gate GEMM + bias
 *   S_t      = the k largest l[t,.]  (ties: lower e)         top-k
 *   w[t,j]   = softmax over the k selected logits            renormalised weights
 *   out[t]   = sum_j w[t,j] * W2_e ( SiLU(W1_e x[t]) * (W3_e x[t]) ),  e = S_t[j]
 *
 * Sources: the gating network and its routing steps (top-k, per-expert counts,
 * weight normalisation, scatter into per-expert buffers) follow MegaScale-Infer,
 * "3.2 Big-Picture Architecture" and "Supporting Implementation Details / Fused
 * Kernels"; the per-expert assignment order (token, then top-k position) follows
 * MegaFlux appendix A.2; tile-aligned token blocks follow MegaFlux section 3.1;
 * the SwiGLU expert (gate, up and down matrices) follows Piper section III-A.
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 * - All pointers are DEVICE pointers unless stated otherwise; `dims` is a HOST
 *   pointer. The caller owns every buffer; the library never allocates device
 *   memory and keeps no pointer after the call returns.
 * - Every call is asynchronous on `stream` (a hipStream_t; NULL = the null
 *   stream). Buffers must stay valid until the stream has passed the call.
 * - Arguments are validated on the host before anything is enqueued. On an
 *   invalid argument nothing is launched and a nonzero moe_status_t comes back.
 *   Faults during execution surface at the caller's next synchronisation.
 * - Layouts are row-major; "[a][b]" lists dimensions outermost first. Weights
 *   use the linear-layer layout [out][in] per expert.
 * - dtype MOE_DTYPE_BF16: x, Wg, W1, W3, W2, the intermediate h, y_sorted and
 *   out are bf16 (fp32 accumulation, round-to-nearest-even stores).
 *   dtype MOE_DTYPE_F32: all of them are fp32. bias, logits and topk_w are fp32
 *   in both cases; indices and counts are int32.
 * - Assignment a = t*k + j (token t, slot j). Sorted position p orders the
 *   assignments by expert, then by a.
 * - Shape limits: T >= 0 (T = 0 is a no-op), d >= 1, f >= 1, 1 <= k <= E <= 1024,
 *   T*k < 2^31, T*E < 2^31. The GPU path needs d % 64 == 0 and f % 64 == 0,
 *   and x (T*d), h (T*k*f) and one expert matrix (d*f) each under 4 GiB
 *   (MOE_ERR_UNSUPPORTED otherwise; moe_route alone accepts d % 8 == 0).
 *   Device pointers to bf16/fp32 tensors must be 16-byte aligned.
 * - Non-finite inputs give unspecified results.
 * - Thread safety: calls are independent except for the stage-timing state,
 *   which is process-wide.
 */
#ifndef MOE_H_
#define MOE_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  MOE_DTYPE_F32 = 0,
  MOE_DTYPE_BF16 = 1
} moe_dtype_t;

typedef enum {
  MOE_OK = 0,
  MOE_ERR_INVALID = 1,      /* null pointer, bad shape, misaligned pointer */
  MOE_ERR_UNSUPPORTED = 2,  /* valid shape the GPU path does not run (see limits) */
  MOE_ERR_WORKSPACE = 3,    /* ws_bytes below what the call needs */
  MOE_ERR_HIP = 4,          /* a HIP launch or runtime call failed */
  MOE_ERR_SCRATCH = 5       /* moe_layer_forward_noalloc: the shape needs more than its static scratch */
} moe_status_t;

typedef struct {
  int64_t T;     /* tokens */
  int64_t d;     /* hidden size */
  int64_t f;     /* expert FFN size */
  int32_t E;     /* routed experts */
  int32_t k;     /* experts per token */
  int32_t dtype; /* moe_dtype_t */
} moe_dims_t;

/* Library version (major*10000 + minor*100 + patch). */
int moe_version(void);

/* Static text for a status code; never NULL. */
const char* moe_status_string(int status);

/* Workspace bytes that make every call below succeed for `dims` (the maximum
 * over the calls; moe_layer_forward with every optional output NULL needs the
 * most). 0 if dims is invalid. The workspace must be 256-byte aligned. */
size_t moe_workspace_bytes(const moe_dims_t* dims);

/* Rows per m-block (the tile-aligned token blocks of at most beta rows that
 * the grouped FFN's tiles cover; MegaFlux section 3.1) that moe_grouped_ffn and
 * moe_layer_forward use for `dims`: 128 when the batch has few rows per active
 * expert (96 or fewer on average, decode batches) or the data is fp32, else 256.
 * The MOE_GEMM_REGIME environment switch overrides the choice. 0 if dims is
 * invalid. Host-only query: no device work. */
int moe_ffn_block_rows(const moe_dims_t* dims);

/* Whether the gate GEMM (MegaScale-Infer, Fused Kernels, step 1) of `dims`
 * runs on the fp32 matrix cores (1) or the vector ALUs (0); -1 if dims is
 * invalid. Both give the same logits, bit for bit. The matrix cores take bf16
 * batches with d a multiple of 64, E >= 32 and at least 256 tiles of 32 tokens
 * x 32 experts; the MOE_GATE_CFG environment switch overrides ("mfma" forces
 * them where they can run, a VALU tile name forces the VALU). Host-only query:
 * no device work. */
int moe_gate_on_matrix_cores(const moe_dims_t* dims);

/* Gate GEMM + bias, top-k selection and renormalised weights
 * (MegaScale-Infer, Fused Kernels, steps 1 and 3).
 *   x      [T][d]   tokens
 *   wg     [E][d]   gate weight
 *   bias   [E] fp32 per-expert gate-logit bias, or NULL for none
 *   logits [T][E] fp32 output, or NULL (then kept in ws)
 *   topk_idx [T][k] int32 output: slot j = expert with the j-th largest logit
 *   topk_w   [T][k] fp32 output: exp(l_j - l_0) / sum_i exp(l_i - l_0)
 * Logits are bit-reproducible: each is the fp32 sum of the products
 * x[t,i]*Wg[e,i] in a fixed order -- 64 lane classes i mod 64, each summed in
 * increasing i from +0.0, then a butterfly over offsets 32,16,8,4,2,1, then
 * one add of bias[e] -- with fp32 products rounded before each add. */
int moe_route(const moe_dims_t* dims, const void* x, const void* wg, const float* bias,
              float* logits, int32_t* topk_idx, float* topk_w,
              void* ws, size_t ws_bytes, void* stream);

/* Dispatch: per-expert histogram, exclusive scan and stable permutation
 * (MegaScale-Infer, Fused Kernels, steps 2 and 4; MegaFlux appendix A.2).
 *   topk_idx [T][k] int32 input, every entry in [0, E)
 *   counts   [E]    rows per expert
 *   offsets  [E+1]  exclusive prefix sum; offsets[E] = T*k
 *   perm     [T*k]  perm[p] = a
 *   inv_perm [T*k]  inv_perm[a] = p
 * Out-of-range expert ids in topk_idx give unspecified (in-bounds) output. */
int moe_permute(const moe_dims_t* dims, const int32_t* topk_idx, int32_t* counts,
                int32_t* offsets, int32_t* perm, int32_t* inv_perm,
                void* ws, size_t ws_bytes, void* stream);

/* Grouped SwiGLU expert FFN over the sorted rows (Piper, section III-A;
 * MegaFlux, sections 2.1 and 3.1): for each sorted row p of expert e,
 * with t = perm[p] / k,
 *   h[p]        = SiLU(W1_e x[t]) * (W3_e x[t])      (h rounded to dtype, kept in ws)
 *   y_sorted[p] = W2_e h[p]
 *   x [T][d]; w1, w3 [E][f][d]; w2 [E][d][f]; y_sorted [T*k][d] output.
 * perm, counts, offsets as produced by moe_permute. */
int moe_grouped_ffn(const moe_dims_t* dims, const void* x, const int32_t* perm,
                    const int32_t* counts, const int32_t* offsets,
                    const void* w1, const void* w3, const void* w2, void* y_sorted,
                    void* ws, size_t ws_bytes, void* stream);

/* Weighted combine (MegaFlux section 2.1, the separate final top-k sum):
 *   out[t] = sum_{j ascending} topk_w[t][j] * y_sorted[inv_perm[t*k+j]]
 * accumulated in fp32, stored in dtype. out [T][d]. */
int moe_combine(const moe_dims_t* dims, const void* y_sorted, const int32_t* inv_perm,
                const float* topk_w, void* out, void* stream);

/* The whole layer: route -> permute -> grouped FFN -> combine, all on `stream`,
 * with no host synchronisation. The sequence of steps follows the pages: the
 * gating network picks each token's experts and its routing steps (top-k,
 * per-expert counts, weight normalisation, scatter into per-expert order) run
 * before the experts (MegaScale-Infer, "3.2 Big-Picture Architecture" item 2
 * and "Supporting Implementation Details / Fused Kernels"); each expert's rows
 * go through FC1 then FC2 in tile-aligned token blocks, and the final top-k
 * sum is a step of its own (MegaFlux, sections 2.1 and 3.1); the expert is the
 * SwiGLU FFN of Piper, section III-A.
 *   x [T][d]; wg [E][d]; bias [E] fp32 or NULL; w1, w3 [E][f][d]; w2 [E][d][f];
 *   out [T][d] output (dtype of x).
 * logits, topk_idx, topk_w, counts, offsets, perm and inv_perm are optional
 * outputs with the layouts of moe_route and moe_permute (NULL = kept in ws).
 * ws: device workspace of at least moe_workspace_bytes(dims) bytes, 256-byte
 * aligned, owned by the caller; its contents need not be initialised and are
 * scratch after the call (moe_layer_plan_layout says where the tile plan is).
 * Errors: MOE_ERR_INVALID (null or misaligned pointer, bad dims),
 * MOE_ERR_UNSUPPORTED (shape limits above), MOE_ERR_WORKSPACE, MOE_ERR_HIP. */
int moe_layer_forward(const moe_dims_t* dims, const void* x, const void* wg, const float* bias,
                      const void* w1, const void* w3, const void* w2, void* out,
                      float* logits, int32_t* topk_idx, float* topk_w,
                      int32_t* counts, int32_t* offsets, int32_t* perm, int32_t* inv_perm,
                      void* ws, size_t ws_bytes, void* stream);

/* moe_layer_forward for callers that cannot allocate device memory (code under
 * HIP graph capture, tight serving loops, harnesses that forbid allocation):
 * the same launches, arguments (minus ws and ws_bytes), outputs and bits as
 * moe_layer_forward, with the workspace taken from a static device array of
 * MOE_NOALLOC_SCRATCH_BYTES that the library holds on every GPU it runs on
 * until the process ends. The call allocates nothing: no hipMalloc or
 * allocating library routine. Shapes whose workspace
 * (moe_workspace_bytes) exceeds that size are refused with MOE_ERR_SCRATCH
 * before anything is enqueued; 128 MiB covers a Mixtral-8x22B-shaped layer
 * of up to about 700 tokens. Every call on one GPU shares that
 * GPU's array, so calls that overlap on one GPU (on different streams, or
 * from different threads) race and give undefined results; serialise them.
 * The first call on a device looks up the array's address there. */
#define MOE_NOALLOC_SCRATCH_BYTES ((size_t)128 << 20)
int moe_layer_forward_noalloc(const moe_dims_t* dims, const void* x, const void* wg, const float* bias,
                              const void* w1, const void* w3, const void* w2, void* out, float* logits,
                              int32_t* topk_idx, float* topk_w, int32_t* counts, int32_t* offsets, int32_t* perm,
                              int32_t* inv_perm, void* stream);

/* Shared (always-active) experts: a layer whose tokens each also pass through
 * n_shared SwiGLU experts of the same sizes outside the routing (Piper, Table III
 * notation; DeepSeek-V3: 256 routed + 1 shared, Piper Table I, note b):
 *   out[t] = sum_j w[t,j] * FFN_{S_t[j]}(x[t]) + sum_{s ascending} FFN^shared_s(x[t])
 * with weight 1 for the shared experts (not part of the renormalised softmax).
 *   sw1, sw3 [n_shared][f][d], sw2 [n_shared][d][f]: shared expert weights.
 * The routed and shared rows run in one grouped FFN (shared rows after the
 * T*k routed ones). Other arguments and outputs as moe_layer_forward (the
 * routing outputs cover the routed experts only). 1 <= n_shared and
 * E + n_shared <= 1024, else MOE_ERR_INVALID. */
size_t moe_workspace_bytes_shared(const moe_dims_t* dims, int n_shared);
int moe_layer_forward_shared(const moe_dims_t* dims, int n_shared, const void* x, const void* wg,
                             const float* bias, const void* w1, const void* w3, const void* w2,
                             const void* sw1, const void* sw3, const void* sw2, void* out,
                             float* logits, int32_t* topk_idx, float* topk_w,
                             int32_t* counts, int32_t* offsets, int32_t* perm, int32_t* inv_perm,
                             void* ws, size_t ws_bytes, void* stream);

/* The same layer in one persistent launch. Workgroups take tiles from
 * device-side sequences: route tiles (one token: its logits, top-k and
 * weights), then, once the workgroup that stored the last route tile has run
 * the dispatch and written the tile plan, FC1 tiles, FC2 tiles and blocks of
 * 512 output vectors for the combine (a batch of at most 16 logits, T*E <=
 * 16, is routed and dispatched by every workgroup for itself, with no wait);
 * an FC2 tile starts once every FC1 tile of its
 * block of rows is stored, the combine once every FC2 tile is, tracked by
 * readiness counters in the workspace instead of kernel boundaries
 * (MegaScale-Infer, "Fused Kernels": the small routing steps fused; MegaFlux,
 * section 2.1: MegaMoE's tiled FC1/FC2 in one persistent kernel). Route and
 * dispatch run inside the launch when E <= 64 and T*k <= 65536 (else as
 * separate launches before it; the MOE_FUSED_FRONT=0 environment switch
 * forces that). The tiles are those of moe_layer_forward: the same rows per
 * block, FC2 tile width and the same split of K (of every tile when a
 * launch has fewer tiles than compute units, of FC2's last partial round of
 * tiles at prefill sizes; the workgroup that stores a split tile's last part
 * sums the parts in the same order), so the outputs and
 * routing arrays are bitwise equal. bf16 only (MOE_ERR_UNSUPPORTED
 * otherwise); other arguments, limits and the workspace size
 * (moe_workspace_bytes) as moe_layer_forward. */
int moe_layer_forward_fused(const moe_dims_t* dims, const void* x, const void* wg, const float* bias,
                            const void* w1, const void* w3, const void* w2, void* out, float* logits,
                            int32_t* topk_idx, float* topk_w, int32_t* counts, int32_t* offsets, int32_t* perm,
                            int32_t* inv_perm, void* ws, size_t ws_bytes, void* stream);
/* Readiness of the fused launch. Its waits need every workgroup of the grid
 * resident at once (persistent workgroups, MegaFlux section 2.1);
 * moe_layer_forward_fused checks the occupancy on the host and returns
 * MOE_ERR_UNSUPPORTED, enqueueing nothing, when the grid cannot all be
 * resident. Each wait is still bounded: a workgroup that polled a readiness
 * counter too long (another kernel holding CUs, for instance) gives up, sets
 * an error word in the workspace and carries on, so the launch always ends but
 * its outputs are then wrong. moe_fused_status waits for `stream` and copies
 * that word of the last moe_layer_forward_fused call on `ws` (same dims) to
 * *flags (host pointer): 0 = every wait was met, so the outputs are valid;
 * nonzero = some wait gave up, discard the outputs (bit 0: a wait for FC1 or
 * FC2 tiles; bit 1: a wait for the tile plan, after which that workgroup left
 * the launch). The word is cleared at the start of every fused call. T == 0
 * gives *flags = 0. Errors as for the workspace checks of moe_layer_forward;
 * MOE_ERR_HIP if the copy fails. */
int moe_fused_status(const moe_dims_t* dims, const void* ws, size_t ws_bytes, int32_t* flags, void* stream);

/* Where the tile plan of a layer call sits in its workspace (host-only query,
 * no device work). After moe_layer_forward, _packed, _fused or (with the same
 * n_shared) _shared on `ws`, bytes [mblocks_offset, + 16 * count) of ws hold
 * the m-blocks the grouped FFN's tiles covered -- tile-aligned token blocks of
 * at most moe_ffn_block_rows rows, at most one partial block per expert
 * (MegaFlux, section 3.1) -- and the int32 at count_offset holds count
 * (<= *max_mblocks), and the int32 after it is 1 if some expert's rows span
 * more than one m-block, else 0 (the grouped FFN's 256-row launches then take
 * their tiles from per-XCD queues). Each m-block is four int32: expert, first sorted row,
 * rows, and (first m-block of its tile group << 4) | group size (the runs of
 * up to 8 m-blocks of one expert the GEMM walks together). n_shared = 0 for
 * layers without shared experts. MOE_ERR_INVALID for bad dims, a null
 * output pointer or n_shared out of range. */
int moe_layer_plan_layout(const moe_dims_t* dims, int n_shared, size_t* mblocks_offset, size_t* count_offset,
                          int64_t* max_mblocks);

/* Expert weights re-laid in the order the grouped FFN streams them (no
 * arithmetic: a permutation of each expert matrix's bf16 values). The expert
 * FFN's FC1/FC2 tiles (MegaFlux, section 2.1) read a column block of weight
 * rows one 64-wide K step at a time, 128 bytes from each of hundreds of rows;
 * in this order every 64-row group of a matrix is K/64 contiguous 8 KiB
 * blocks, one per K step, each already in the order the loads place it in
 * LDS, which HBM streams faster. Meant for weights that are packed once and
 * read by many calls (decode); the packing is not part of a layer call.
 *   moe_pack_weights: w1p, w3p [E][f][d] and w2p [E][d][f] (device buffers the
 *     caller owns, the sizes of w1, w3, w2, 16-byte aligned, not overlapping
 *     the inputs) receive the stage-order copies of w1, w3, w2; asynchronous
 *     on `stream`. bf16 only (MOE_ERR_UNSUPPORTED otherwise); d and f
 *     multiples of 64 as for the layer.
 *   moe_layer_forward_packed: moe_layer_forward reading the packed weights
 *     in place of w1, w3, w2; same arguments, limits, workspace and outputs,
 *     and bitwise the same result (the tiles load the same values into LDS).
 * Element (e, n, k) of a packed tensor of row length K (d for w1p, w3p; f for
 * w2p) sits at 16-byte unit (((e*N/64 + n/64) * K/64 + k/64) * 64 + n%64) * 8
 * + ((k%64)/8 ^ ((n%64)/2)%8), element k%8 of the unit. */
int moe_pack_weights(const moe_dims_t* dims, const void* w1, const void* w3, const void* w2, void* w1p,
                     void* w3p, void* w2p, void* stream);
/* moe_pack_weights for weights held in the other orientation, input-major:
 * w1t, w3t [E][d][f] and w2t [E][f][d], i.e. each expert's gate and up
 * matrices as d x f and its down matrix as f x d, as Piper section III-A
 * writes them (w1t[e][i][j] = w1[e][j][i], and so on). The outputs are the
 * same stage-order tensors w1p, w3p [E][f][d], w2p [E][d][f], bitwise equal to
 * what moe_pack_weights gives for the [out][in] tensors, so the caller never
 * transposes. Same limits, ownership and errors as moe_pack_weights (plus
 * MOE_ERR_UNSUPPORTED when E * d/64 * f/64 >= 2^31); the inputs are
 * 16-byte aligned device buffers that do not overlap the outputs. */
int moe_pack_weights_transposed(const moe_dims_t* dims, const void* w1t, const void* w3t, const void* w2t,
                                void* w1p, void* w3p, void* w2p, void* stream);
int moe_layer_forward_packed(const moe_dims_t* dims, const void* x, const void* wg, const float* bias,
                             const void* w1p, const void* w3p, const void* w2p, void* out, float* logits,
                             int32_t* topk_idx, float* topk_w, int32_t* counts, int32_t* offsets,
                             int32_t* perm, int32_t* inv_perm, void* ws, size_t ws_bytes, void* stream);
/* moe_layer_forward_fused reading packed weights (moe_pack_weights): the one
 * persistent launch of moe_layer_forward_fused with the weight loads of
 * moe_layer_forward_packed; bitwise the same outputs as both. Arguments,
 * limits, workspace, errors and moe_fused_status as moe_layer_forward_fused. */
int moe_layer_forward_fused_packed(const moe_dims_t* dims, const void* x, const void* wg, const float* bias,
                                   const void* w1p, const void* w3p, const void* w2p, void* out, float* logits,
                                   int32_t* topk_idx, float* topk_w, int32_t* counts, int32_t* offsets,
                                   int32_t* perm, int32_t* inv_perm, void* ws, size_t ws_bytes, void* stream);

/* ---- backward pass ----
 * Gradients of the layer for a scalar loss whose gradient with respect to
 * `out` is `dout`. The pages name the parts (MegaFlux, section 2.1: token
 * blocks stream through DGrad and WGrad, and the final top-k sum is a step of
 * its own; section 3.2 and Figure 2); the formulas are the chain rule of the
 * forward: per assignment (t, j) of expert e with weight w,
 *   dtopk_w[t][j] = dout_t . y,   dW2_e += (w dout_t) h^T,
 *   dg = (W2_e^T w dout_t) * u * SiLU'(g),  du = (W2_e^T w dout_t) * SiLU(g),
 *   dW1_e += dg x_t^T,  dW3_e += du x_t^T,  dx_t += W1_e^T dg + W3_e^T du,
 * then the softmax over the k selected logits,
 *   dlogits[t][e_j] = w_j (dtopk_w[t][j] - sum_i w_i dtopk_w[t][i]) (0 elsewhere),
 * and the gate: dbias = column sums of dlogits, dwg = dlogits^T x,
 * dx += dlogits wg. The selection itself is piecewise constant and gets no
 * gradient.
 *
 * Inputs: the forward's inputs (bf16 only: dims->dtype must be MOE_DTYPE_BF16)
 * and its routing outputs topk_idx, topk_w, counts, offsets, perm, inv_perm
 * (exactly as moe_layer_forward or moe_route + moe_permute return them), and
 * dout [T][d] bf16. Outputs (device, caller-allocated): dx [T][d] bf16;
 * dwg [E][d], dbias [E], dw1 [E][f][d], dw3 [E][f][d], dw2 [E][d][f] fp32
 * (every entry written, zero for experts that received no rows); optional
 * (NULL to skip) dlogits [T][E] and dtopk_w [T][k] fp32.
 * FC1 is recomputed (moe_layer_forward keeps only h; moe_layer_forward_train
 * and moe_layer_backward_saved below keep g and u instead); W1, W3 and W2
 * are read as stored (the DGrad products take them through transposing LDS
 * loads, no copies). Accumulation is fp32 throughout;
 * dg, du, h and w*dout enter the matrix products as bf16. Every reduction
 * has a fixed order: results are deterministic.
 * Limits: d and f multiples of 256, else MOE_ERR_UNSUPPORTED; pointers
 * 16-byte aligned (4 for the int32 / fp32 routing arrays); ws at least
 * moe_backward_workspace_bytes(dims), 256-byte aligned. T == 0 writes zero
 * weight gradients. Asynchronous on `stream`. */
size_t moe_backward_workspace_bytes(const moe_dims_t* dims);
int moe_layer_backward(const moe_dims_t* dims, const void* x, const void* wg, const void* w1, const void* w3,
                       const void* w2, const int32_t* topk_idx, const float* topk_w, const int32_t* counts,
                       const int32_t* offsets, const int32_t* perm, const int32_t* inv_perm, const void* dout,
                       void* dx, float* dwg, float* dbias, float* dw1, float* dw3, float* dw2,
                       float* dlogits, float* dtopk_w, void* ws, size_t ws_bytes, void* stream);

/* ---- training pair: FC1's g | u kept from the forward for the backward ----
 * The backward above recomputes FC1 (g = x W1_e^T, u = x W3_e^T per sorted
 * row) because the forward keeps only h. MegaFlux (section 2.1) runs the
 * backward as its own DGrad and WGrad streams and is silent on what the
 * forward saves; this pair trades [T*k][2f] bf16 of memory for that
 * recompute (4 d f FLOP per sorted row).
 *
 * moe_layer_forward_train: moe_layer_forward (same arguments, routing outputs,
 * optional NULLs and workspace, moe_workspace_bytes) plus the output
 * gu [T*k][2f] bf16 (device, caller-allocated, 16-byte aligned; required when
 * T > 0): row p holds g then u of sorted row p (the order of perm), rounded to
 * bf16. FC1 runs over 256-row tiles of the same plan as the backward's
 * recompute, so gu is bit for bit what moe_layer_backward computes internally;
 * the same launch forms h = SiLU(g) u from the fp32 sums, as moe_layer_forward
 * does, so `out` has the plain forward's arithmetic (it can differ from
 * moe_layer_forward's in the last bf16 bit where that call sums a tile's K
 * range in parts, and is held to the same 2e-2 bar against the fp64
 * definition). bf16 only; d and f multiples of 256;
 * no shared experts; errors as moe_layer_backward's limits
 * (MOE_ERR_UNSUPPORTED) and moe_layer_forward's arguments.
 *
 * moe_layer_backward_saved: moe_layer_backward with `gu` (as written by
 * moe_layer_forward_train for the same x, W1, W3 and routing arrays) read
 * instead of recomputed; every output is bit for bit moe_layer_backward's.
 * Same workspace (moe_backward_workspace_bytes), limits and errors; gu must be
 * 16-byte aligned when T > 0 (MOE_ERR_INVALID otherwise). */
int moe_layer_forward_train(const moe_dims_t* dims, const void* x, const void* wg, const float* bias,
                            const void* w1, const void* w3, const void* w2, void* out, float* logits,
                            int32_t* topk_idx, float* topk_w, int32_t* counts, int32_t* offsets,
                            int32_t* perm, int32_t* inv_perm, void* gu, void* ws, size_t ws_bytes, void* stream);
int moe_layer_backward_saved(const moe_dims_t* dims, const void* x, const void* wg, const void* w1,
                             const void* w3, const void* w2, const int32_t* topk_idx, const float* topk_w,
                             const int32_t* counts, const int32_t* offsets, const int32_t* perm,
                             const int32_t* inv_perm, const void* dout, const void* gu, void* dx, float* dwg,
                             float* dbias, float* dw1, float* dw3, float* dw2, float* dlogits, float* dtopk_w,
                             void* ws, size_t ws_bytes, void* stream);

/* moe_layer_backward with its options in one call: `gu` NULL recomputes FC1
 * (moe_layer_backward), non-NULL reads it (moe_layer_backward_saved; 16-byte
 * aligned); `wgrad_dtype` MOE_DTYPE_F32 writes dw1, dw3, dw2 as fp32 (as those
 * two calls do), MOE_DTYPE_BF16 as bf16 [same shapes], each element the
 * round-to-nearest-even bf16 of the fp32 value the fp32 form writes. The bf16
 * form halves the bytes the weight-gradient products write (3 E d f values
 * per call), which bound them when experts receive ~100 rows (the DeepSeek
 * shape). dx, dwg, dbias, dlogits, dtopk_w are as in moe_layer_backward and
 * bitwise the same. Workspace, limits and errors as moe_layer_backward;
 * MOE_ERR_INVALID for another wgrad_dtype or a misaligned gu. */
int moe_layer_backward_ex(const moe_dims_t* dims, const void* x, const void* wg, const void* w1, const void* w3,
                          const void* w2, const int32_t* topk_idx, const float* topk_w, const int32_t* counts,
                          const int32_t* offsets, const int32_t* perm, const int32_t* inv_perm, const void* dout,
                          const void* gu, int wgrad_dtype, void* dx, float* dwg, float* dbias, void* dw1,
                          void* dw3, void* dw2, float* dlogits, float* dtopk_w, void* ws, size_t ws_bytes,
                          void* stream);

/* ---- scored router: selection from scores, its losses and gradients ----
 * The router of layers whose experts are chosen by softmax or sigmoid scores
 * with a balance bias, optionally inside groups of experts. For the logits l
 * of one token (fp32, as moe_route computes them):
 *   s_e = sigmoid(l_e), or exp(l_e) / sum_i exp(l_i) over all E experts;
 *   c_e = s_e + balance_bias[e]     the key: chooses, does not weigh;
 *   an expert is out of the token's choice when its logit or its bias is -inf
 *   or NaN (+inf counts as the largest finite logit); NaN in such places
 *   reaches no output;
 *   with groups > 1, the E / groups consecutive experts of a group have the
 *   group key max c, or the sum of their two largest c (the one, if only one
 *   is in the choice); the topk_groups groups with the largest keys are kept
 *   (ties: lower group; a group with no expert in the choice comes last), and
 *   the other groups' experts are out of the choice;
 *   the k experts with the largest c are chosen, slot by slot (ties: larger
 *   logit, then lower expert). Keys are compared as doubles;
 *   topk_w[j] = scale * s_j, with renormalise divided by the sum of the chosen s.
 *   Scores (with renormalise, their quotients by the largest chosen one) below
 *   2^-126 have that absolute precision and may come as 0; a weight of 0 passes
 *   no gradient.
 * Where fewer than k experts are in the choice, the slots left take the
 * experts out of it in ascending order with weight 0 (so every index is valid
 * for moe_permute); a row with none gets experts 0 .. k-1 and weights 0.
 * Limits: as moe_dims_t (only T, E and k are used), groups <= 64 dividing E,
 * topk_groups * E / groups >= k, scale finite, else MOE_ERR_INVALID. */
typedef enum {
  MOE_SCORE_SOFTMAX = 0,
  MOE_SCORE_SIGMOID = 1
} moe_score_t;
typedef enum {
  MOE_GROUP_MAX = 0,  /* group key: its largest key */
  MOE_GROUP_TOP2 = 1  /* group key: the sum of its two largest keys */
} moe_group_rule_t;
typedef struct {
  int32_t score;       /* moe_score_t */
  int32_t groups;      /* groups of consecutive experts; 1 = no groups */
  int32_t topk_groups; /* groups kept per token */
  int32_t group_rule;  /* moe_group_rule_t */
  int32_t renormalise; /* 1: weights divided by their sum */
  float scale;         /* factor of the weights */
} moe_route_opts_t;

/* Selection from logits. logits [T][E] fp32; balance_bias [E] fp32 or NULL;
 * outputs topk_idx [T][k] int32, topk_w [T][k] fp32. `opts` is a HOST pointer. */
int moe_route_select(const moe_dims_t* dims, const moe_route_opts_t* opts, const float* logits,
                     const float* balance_bias, int32_t* topk_idx, float* topk_w, void* stream);

/* Gate GEMM + bias (moe_route's logits, bit for bit), then the selection.
 * x [T][d], wg [E][d], bias [E] fp32 or NULL (added to the logits), logits
 * [T][E] fp32 output (required: the backward reads it). d % 8 == 0. */
int moe_route_scored(const moe_dims_t* dims, const moe_route_opts_t* opts, const void* x, const void* wg,
                     const float* bias, const float* balance_bias, float* logits, int32_t* topk_idx, float* topk_w,
                     void* stream);

/* Balance losses over n_seq packed sequences: rows seq_offsets[s] ..
 * seq_offsets[s+1]-1 (device int32 [n_seq+1], not decreasing, clamped to
 * [0, T]; NULL with n_seq = 1: all T rows). Rows outside every sequence count
 * in neither loss. With n_s rows, f[s][e] = how often sequence s chose expert
 * e, shares q = s_e / sum_i s_i of each row and the sequences that have rows:
 *   losses[0] = mean over them of E / (k n_s^2) sum_e f[s][e] sum_t q[t][e]
 *   losses[1] = mean over their rows of (log sum_e exp l[t][e])^2
 * (a row with every logit -inf adds nothing; no rows: both 0). Only
 * opts->score is used. topk_idx [T][k] (entries outside [0, E) are not
 * counted). Outputs losses [2] fp32, load [n_seq][E] int32 = f (the loads a
 * caller adjusts balance_bias by). Fixed summation order. ws: at least
 * moe_balance_workspace_bytes (0 for invalid arguments), 256-byte aligned.
 * n_seq <= 65535 (MOE_ERR_UNSUPPORTED beyond). */
size_t moe_balance_workspace_bytes(const moe_dims_t* dims, int32_t n_seq);
int moe_balance_loss(const moe_dims_t* dims, const moe_route_opts_t* opts, const float* logits,
                     const int32_t* topk_idx, const int32_t* seq_offsets, int32_t n_seq, float* losses, int32_t* load,
                     void* ws, size_t ws_bytes, void* stream);

/* Gradient of selection and losses with respect to the logits; the choice
 * itself is piecewise constant. dlogits [T][E] fp32 = the gradient of
 *   sum_t sum_j dtopk_w[t][j] topk_w[t][j] + dlosses[0] losses[0] + dlosses[1] losses[1]
 * (the loads f are constants), every element written. dtopk_w [T][k] NULL: without the first term (topk_idx and
 * topk_w may then be NULL too); dlosses (device fp32 [2]) NULL: without the
 * others (load, seq_offsets and n_seq are then not looked at), else load
 * [n_seq][E] as moe_balance_loss returned it for the same seq_offsets.
 * topk_idx and topk_w as moe_route_select returned them for these logits and
 * options: a slot of weight 0 passes no gradient, an entry outside [0, E) is
 * skipped, repeated entries add up. Values of dtopk_w and dlosses that are not
 * finite go where the formula sends them; a finite dlosses[1] whose product with
 * a row's log-sum-exp passes fp32's range counts as the largest value there is.
 * Experts whose logit is -inf or NaN get 0;
 * shares below 2^-126 have that absolute precision. */
int moe_route_select_backward(const moe_dims_t* dims, const moe_route_opts_t* opts, const float* logits,
                              const int32_t* topk_idx, const float* topk_w, const float* dtopk_w,
                              const float* dlosses, const int32_t* load, const int32_t* seq_offsets, int32_t n_seq,
                              float* dlogits, void* stream);

/* Gradients of the gate GEMM for a dense logit gradient:
 *   dx = dx_in + dlogits Wg (bf16, one rounding), dwg = dlogits^T x, dbias = column sums (fp32)
 * x [T][d], wg [E][d], dx_in [T][d] or NULL, dx [T][d] bf16 (may be dx_in, and
 * overlaps nothing else);
 * dlogits [T][E], dwg [E][d], dbias [E] fp32. bf16 only, d % 8 == 0, T <=
 * 4194176, d <= 2^24 and (T/128 + 1)(d/128 + 1) < 2^23 (MOE_ERR_UNSUPPORTED otherwise). T = 0 writes zero dwg and
 * dbias. dwg's sums are fp32, of exact products; fixed summation order. dx's sum
 * is fp32 too, but takes dlogits to 16 bits: up to 2^-16 of each term is lost
 * before it, which shows behind the bf16 rounding where terms cancel by more than
 * some 2^8. In both, bits of dlogits below 2^-133 are rounded to that.
 * Infinities and NaN, of x and wg as of dlogits, go where the formula sends them.
 * ws: at least moe_gate_backward_workspace_bytes(dims), 256-byte aligned. */
size_t moe_gate_backward_workspace_bytes(const moe_dims_t* dims);
int moe_gate_backward(const moe_dims_t* dims, const void* x, const void* wg, const float* dlogits, const void* dx_in,
                      void* dx, float* dwg, float* dbias, void* ws, size_t ws_bytes, void* stream);

/* The experts' part of moe_layer_backward_ex, for routers whose gradient is
 * taken elsewhere (moe_route_select_backward, moe_gate_backward): the same
 * arguments without the gate's; dx [T][d] bf16 is the experts' part alone and
 * dtopk_w [T][k] fp32 (required) the gradient of the weights. Expert weight
 * gradients and dtopk_w are bitwise moe_layer_backward_ex's. Workspace, limits
 * and errors as there. */
int moe_experts_backward(const moe_dims_t* dims, const void* x, const void* w1, const void* w3, const void* w2,
                         const int32_t* topk_idx, const float* topk_w, const int32_t* counts, const int32_t* offsets,
                         const int32_t* perm, const int32_t* inv_perm, const void* dout, const void* gu,
                         int wgrad_dtype, void* dx, void* dw1, void* dw3, void* dw2, float* dtopk_w, void* ws,
                         size_t ws_bytes, void* stream);

/* ---- dropout beside the combine ----
 * The combine with dropout on the layer's output, added to a residual:
 *   out[t][c] = residual[t][c] + keep(t, c) S sum_j topk_w[t][j] y_sorted[inv_perm[t*k+j]][c]
 * keep is drawn from a counter-based generator and never stored: element
 * i = t*d + c takes 16-bit number i % 8 (low half of word 0, its high half, low
 * half of word 1, ..) of Philox4x32 with ten rounds, key = seed (low word
 * first), counter = {i / 8 (64 bits), offset (64 bits)}, and is kept when it is
 * at least thr = round(65536 p), ties to even; S = 65536 / (65536 - thr). p = 0
 * keeps all, p = 1 drops all (out = residual). p outside [0, 1] or NaN:
 * MOE_ERR_INVALID. rng: DEVICE pointer to {seed, offset}, 8-byte aligned, read
 * when the kernel runs: a captured graph draws anew when its owner updates it
 * between replays. Two calls with the same seed and offset draw the same.
 * A dropped element is the residual alone, whatever its value.
 *   moe_combine_dropout: arguments as moe_combine, and residual [T][d] (the
 *     dtype; NULL = 0; out may be residual). Sum, scaling and residual in fp32,
 *     one rounding.
 *   moe_dropout_backward: dy = keep S dout [T][d], the gradient of the combined
 *     sum, which moe_experts_backward or moe_layer_backward takes as its dout
 *     (residual's gradient is dout itself); dy may be dout.
 * d % 8 == 0 (MOE_ERR_UNSUPPORTED otherwise); bf16 and fp32. */
int moe_combine_dropout(const moe_dims_t* dims, double p, const uint64_t* rng, const void* y_sorted,
                        const int32_t* inv_perm, const float* topk_w, const void* residual, void* out, void* stream);
int moe_dropout_backward(const moe_dims_t* dims, double p, const uint64_t* rng, const void* dout, void* dy,
                         void* stream);

/* ---- around the layer: the norm in front of it ----
 * y = norm(s), s = x + residual: the row s is summed in fp32 and rounded to the
 * dtype, and what is normalised is that rounded row. With d columns:
 *   MOE_NORM_RMS:    rstd = (mean s^2 + eps)^(-1/2),            y = s rstd weight
 *   MOE_NORM_LAYER:  rstd = (mean (s - mean s)^2 + eps)^(-1/2), y = (s - mean s) rstd weight + bias
 * Statistics in fp32, from the differences to the mean (taken as a number and the
 * rest that its rounding lost); a row whose sums pass fp32's range is summed at a
 * smaller scale. y is rounded once. Infinities and NaN in a row go where the
 * formula sends them.
 *   x, residual (NULL = 0), sum (NULL: not written; may be x or residual), y [T][d]
 *   dtype; y may be x or residual (and is not sum);
 *   weight, bias [d] of opts->param_dtype, or NULL (1 and 0); bias NULL for RMS;
 *   mean, rstd [T] fp32 outputs, or NULL (mean NULL for RMS).
 * d % 8 == 0 and d <= 16384 (MOE_ERR_UNSUPPORTED otherwise); eps in [2^-100, 2^100],
 * else MOE_ERR_INVALID. dims are the layer's and must be valid as a whole, T * k and
 * T * E below 2^31 among it; the norm itself uses T, d and dtype. `opts` is a HOST
 * pointer. Tensors of x's shape, weight and bias 16-byte aligned. */
typedef enum {
  MOE_NORM_RMS = 0,
  MOE_NORM_LAYER = 1
} moe_norm_kind_t;
typedef struct {
  int32_t kind;        /* moe_norm_kind_t */
  int32_t param_dtype; /* moe_dtype_t of weight and bias */
  float eps;
} moe_norm_opts_t;
int moe_norm_forward(const moe_dims_t* dims, const moe_norm_opts_t* opts, const void* x, const void* residual,
                     const void* weight, const void* bias, void* sum, void* y, float* mean, float* rstd,
                     void* stream);

/* Its gradients. With h = (s - mean) rstd (RMS: s rstd) and g = dy weight:
 *   dx = rstd (g - mean g - h mean(g h)) + dx_in   (RMS: without mean g)
 *   dweight = sum_t dy h,  dbias = sum_t dy
 * dx is the gradient of s, hence of x and of residual alike. The mean handed in is
 * rounded: what that puts the h of a row off by, their mean, is taken back in rows whose
 * mean lies more than 8 / rstd from zero; in others it is at most 2^-21.
 *   dy, s [T][d] (s: the row that was normalised: x, or the forward's sum);
 *   weight as in the forward; mean (layer norm), rstd [T] as the forward gave them;
 *   dx_in [T][d] (the gradient that reaches s by other ways) or NULL;
 *   dx [T][d] (may be dy, s or dx_in); dweight, dbias [d] fp32, each NULL to leave
 *   it out (dbias NULL for RMS).
 * fp32 throughout, dx rounded once; sums over rows in a fixed order. T = 0 writes
 * zero dweight and dbias. Limits as the forward's; dweight and dbias 16-byte
 * aligned. ws: at least moe_norm_backward_workspace_bytes (0 for invalid dims),
 * 256-byte aligned; not looked at where neither dweight nor dbias is asked for. */
size_t moe_norm_backward_workspace_bytes(const moe_dims_t* dims, const moe_norm_opts_t* opts);
int moe_norm_backward(const moe_dims_t* dims, const moe_norm_opts_t* opts, const void* dy, const void* s,
                      const void* weight, const float* mean, const float* rstd, const void* dx_in, void* dx,
                      float* dweight, float* dbias, void* ws, size_t ws_bytes, void* stream);

/* ---- behind the backward: the gradients' norm and the update ----
 * Both take a list of tensors, a HOST array that is read during the call only (a
 * captured graph holds its contents). At most 2^36 elements to a gradient, 2^34 to
 * a parameter, and 2^20 tensors (MOE_ERR_UNSUPPORTED beyond); tensors of 0 elements
 * are passed over.
 * Buffers need their element's alignment; where all of a tensor's are 16-byte
 * aligned (8-bit codes: 8-byte) the loads are wide. */
typedef struct {
  const void* grad; /* DEVICE [n] */
  int64_t n;
  int64_t dtype;    /* moe_dtype_t */
} moe_grad_t;

/* out[0] = N = |grad_scale| (sum over all elements g^2)^(1/2), and the factor
 * that unscales and clips: out[1] = grad_scale min(1, max_norm / (N + 1e-6)), or
 * NaN where N (formed in double) is not finite. Squares are summed in double in a
 * fixed order.
 * out [2] fp32 (DEVICE). grad_scale finite, max_norm >= 0 (infinity: no clipping),
 * else MOE_ERR_INVALID. ws: at least moe_grad_norm_workspace_bytes (0 for an
 * invalid list), 256-byte aligned. An empty list gives N = 0. */
size_t moe_grad_norm_workspace_bytes(const moe_grad_t* grads, int32_t count);
int moe_grad_norm(const moe_grad_t* grads, int32_t count, double grad_scale, double max_norm, float* out, void* ws,
                  size_t ws_bytes, void* stream);

/* AdamW (decoupled weight decay) over a list of tensors, in place. With step t:
 *   x  = gscale g
 *   m' = beta1 m + (1 - beta1) x,   v' = beta2 v + (1 - beta2) x^2
 *   w' = w - lr / (1 - beta1^t) m' / (sqrt(v' / (1 - beta2^t)) + eps) - lr weight_decay w
 * in fp32; w is master where there is one, else param. param bf16 is rounded to
 * nearest even, or with `stochastic` (without master) up or down at random so that
 * its mean is w'. A gscale that is not finite leaves everything as it was.
 *
 * state_bits 32: m, v [n] fp32. state_bits 8: m, v [n] uint8 and m_scale, v_scale
 * [ceil(n / 128)] uint8, one for each 128 elements of the tensor. A scale byte E is
 * a biased fp32 exponent; code c of m stands for (-1)^(c >> 7) a 2^(E - 15), a the
 * fp32 value whose bits are (c & 127) << 20, and code c of v for the ROOT of the
 * second moment, a 2^(E - 15) with bits c << 19: four exponent bits, three (m, with
 * a sign) or four fraction bits, gradual underflow. E = 255: NaN. All zero bytes
 * are the state before the first step. m' and sqrt(v') are formed in fp32 and then
 * rounded at random: E is the least exponent whose top code holds the largest of the
 * 128 (255 where one is not finite or lies above 254's top code; their codes are 0 then),
 * and a value is rounded
 * away from zero where the part of a code step that it drops (to 2^-20 of a step)
 * and u / 2^16 reach 1, u the element's 16-bit number; a root above 0 takes code 1
 * at least. So m and the root keep their means from step to step; v is the root's square
 * and stands high by the variance of its rounding, at most 1/32 of the mean of |x^2 - v|
 * (1 to 2 % for normally distributed x and beta2 from 0.95 to 0.999), an element's v
 * scattering by some 20 % around that.
 *
 * Numbers: elements are counted through the list, each tensor beginning at a
 * multiple of 128; element i takes number i % 8 (low half of word 0, its high half,
 * low half of word 1, ..) of Philox4x32 with ten rounds, key = seed, counter =
 * {i / 8, offset} (as moe_combine_dropout's). rng: DEVICE {seed, offset}, 8-byte
 * aligned, needed with state_bits 8 and with stochastic; states and weights of an
 * element share its number.
 *
 * lr_step: DEVICE {lr, step} (two doubles, step a whole number from 1), read when
 * the kernels run, so that a captured graph follows its owner's schedule; NULL:
 * opts->lr and opts->step. gscale: DEVICE fp32 [1] or NULL (1).
 * grads[i] belongs to tensors[i] and has its n. No buffer may overlap another
 * (one that is written and appears twice: MOE_ERR_INVALID). beta1, beta2 in
 * [0, 1), eps in [2^-100, 2^100], lr and weight_decay finite, step >= 1 (unless
 * lr_step), else MOE_ERR_INVALID. `opts`, `tensors` and `grads` are HOST pointers. */
typedef struct {
  void* param;      /* [n] */
  float* master;    /* [n] fp32, or NULL; bf16 parameters only */
  void* m;          /* [n] */
  void* v;          /* [n] */
  uint8_t* m_scale; /* 8-bit states; else not looked at */
  uint8_t* v_scale;
  int64_t n;
  int64_t dtype;    /* moe_dtype_t of param */
} moe_adam_tensor_t;
typedef struct {
  double lr, beta1, beta2, eps, weight_decay;
  int64_t step;
  int32_t state_bits; /* 32 or 8 */
  int32_t stochastic; /* 0 or 1 */
} moe_adam_opts_t;
int moe_adam_step(const moe_adam_opts_t* opts, const moe_adam_tensor_t* tensors, const moe_grad_t* grads,
                  int32_t count, const double* lr_step, const float* gscale, const uint64_t* rng, void* stream);

/* What 8-bit states stand for: m_out[i] [n] = m and r_out[i] [n] = sqrt(v) of
 * tensors[i] (HOST arrays of DEVICE pointers), of out_dtype (bf16 holds every
 * code's value from 2^-126 on; smaller ones are rounded). param, master are not
 * looked at. An output that appears twice: MOE_ERR_INVALID; none may overlap the
 * states. */
int moe_adam_state_values(const moe_adam_tensor_t* tensors, int32_t count, void* const* m_out, void* const* r_out,
                          int out_dtype, void* stream);

/* ---- stage timing (instrumentation; process-wide, not thread-safe) ----
 * While enabled, every kernel the library launches is bracketed by HIP events
 * recorded on the stream it is launched on. Stages: */
enum {
  MOE_STAGE_GATE = 0,     /* gate logits */
  MOE_STAGE_TOPK = 1,     /* top-k + weights */
  MOE_STAGE_HIST = 2,     /* dispatch histogram */
  MOE_STAGE_SCAN = 3,     /* dispatch scan */
  MOE_STAGE_SCATTER = 4,  /* dispatch permutation */
  MOE_STAGE_PLAN = 5,     /* tile plan */
  MOE_STAGE_FC1 = 6,      /* grouped FC1 + SiLU*mul */
  MOE_STAGE_FC2 = 7,      /* grouped FC2 */
  MOE_STAGE_COMBINE = 8,  /* weighted combine */
  MOE_STAGE_DISPATCH = 9, /* single-workgroup histogram + scan + scatter (+ tile plan) */
  MOE_STAGE_BWD_WT = 10,      /* reserved (the backward reads the weights as stored) */
  MOE_STAGE_BWD_FC1 = 11,     /* backward: FC1 recompute (g | u) */
  MOE_STAGE_BWD_DH = 12,      /* backward: DGrad of FC2 (q = dout W2) */
  MOE_STAGE_BWD_SWIGLU = 13,  /* backward: dg | du and dtopk_w */
  MOE_STAGE_BWD_ROUTE = 14,   /* backward: softmax over the selected logits */
  MOE_STAGE_BWD_DX = 15,      /* backward: DGrad of FC1 */
  MOE_STAGE_BWD_DXSUM = 16,   /* backward: per-token dx sum (+ gate part) */
  MOE_STAGE_BWD_ACT_T = 17,   /* backward: activation transposes for WGrad */
  MOE_STAGE_BWD_WG2 = 18,     /* backward: WGrad of W2 */
  MOE_STAGE_BWD_WG13 = 19,    /* backward: WGrad of W1 and W3 */
  MOE_STAGE_BWD_GATE = 20,    /* backward: gate weight and bias gradients */
  MOE_STAGE_FFN_FUSED = 21,   /* FC1 + FC2 + combine in one launch (moe_layer_forward_fused) */
  MOE_STAGE_SELECT = 22,       /* scored selection */
  MOE_STAGE_BALANCE = 23,      /* balance losses */
  MOE_STAGE_SELECT_BWD = 24,   /* scored selection's and losses' backward */
  MOE_STAGE_GATE_BWD = 25,     /* dense gate gradients */
  MOE_STAGE_COMBINE_DROP = 26, /* combine with dropout */
  MOE_STAGE_DROP_BWD = 27,     /* dropout backward */
  MOE_STAGE_NORM = 28,         /* norm */
  MOE_STAGE_NORM_BWD = 29,     /* norm backward */
  MOE_STAGE_GRAD_NORM = 30,    /* 2-norm of the gradients */
  MOE_STAGE_ADAM = 31,         /* AdamW update; values of its states */
  MOE_NUM_STAGES = 32
};
/* Start recording; `capacity` = launches per stage to keep (host memory only);
 * `stage_mask` = bit s set records stage s (0 = every stage). Discards
 * earlier records. */
int moe_timing_enable(int capacity, unsigned stage_mask);
/* Stop recording (records are kept until the next enable). */
int moe_timing_disable(void);
/* Synchronises on the recorded events of `stage` and returns the summed
 * kernel time in ms and the number of launches recorded. */
int moe_timing_read(int stage, double* total_ms, int* launches);

/* ---- measurement probes (diagnostic; not part of the layer) ----
 * Kernels that measure what the GPU sustains, so that achieved fractions can be
 * reported against measured ceilings next to the datasheet peaks. Asynchronous
 * on `stream`; the caller times them (e.g. with events on that stream). */
/* Compute units; the probes launch one workgroup of 8 waves on each. */
int moe_probe_cus(void);
/* Streams `bytes` (a multiple of 16, 16-byte aligned device buffer `src`)
 * through LDS: each workgroup reads a contiguous slice of bytes / CUs (rounded
 * down to 16 bytes; at most 2 GiB) with 16-byte buffer loads, three 32 KiB
 * steps in flight. sink [CUs] int32 receives one loaded byte per workgroup.
 * MOE_ERR_INVALID for a null or misaligned pointer or a bad size,
 * MOE_ERR_UNSUPPORTED if a slice would be empty or too large. */
int moe_probe_hbm_read(const void* src, size_t bytes, int32_t* sink, void* stream);
/* `iters` rounds of 32 bf16 16x16x32 MFMAs (eight independent accumulator
 * chains) in each of 8 waves per CU, register operands with varied bits only:
 * FLOP = 2*16*16*32 * 32 * 8 * iters * CUs. sink [8 * CUs] fp32 receives each
 * wave's accumulator sum. MOE_ERR_INVALID for a null sink or iters < 1. */
int moe_probe_mfma(int iters, float* sink, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* MOE_H_ */
