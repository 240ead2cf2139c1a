/*
 * sdm.h -- C ABI of the Sparse Delta Memory (SDM) hot path on MI355X (gfx950).
 *
 * The operations follow "Sparse Delta Memory：中文精读笔记" (close-reading notes
 * on arXiv 2607.07386v1), cited below as [SDM], and the product-key
 * addressing of "Fast-weight Product Key Memory：中文精读笔记" §2.2, cited as
 * [FwPKM].
 *
 * Common conventions
 *   - Every tensor pointer is a DEVICE pointer owned by the caller. Tensors are
 *     row-major and contiguous; shapes are given in the comments. Sizes are
 *     int64_t. The library never frees or retains caller memory.
 *   - `stream` is a hipStream_t passed as void* (NULL = the null stream). All
 *     compute calls are asynchronous and ordered on that stream; results are
 *     visible after the caller synchronises it.
 *   - Every call validates its arguments on the host before any launch. On
 *     failure it returns a non-zero sdm_status, writes nothing and launches
 *     nothing; sdm_last_error() then describes the failure (thread-local).
 *     A failed launch returns SDM_ERR_HIP. Faults inside a kernel surface at
 *     the caller's next synchronisation. No C++ exception crosses the ABI.
 *   - Pointers to device tensors must be 16-byte aligned (SDM_ERR_ALIGN).
 *   - Empty work (B, H or T equal to 0) is valid, launches nothing and accepts
 *     NULL tensor pointers (empty tensors need not have storage).
 */
#ifndef SDM_H
#define SDM_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define SDM_ABI_VERSION 7

typedef enum sdm_status {
    SDM_OK = 0,
    SDM_ERR_NULL = 1,         /* a required pointer is NULL                      */
    SDM_ERR_SHAPE = 2,        /* a size is negative or sizes are inconsistent    */
    SDM_ERR_DTYPE = 3,        /* unknown dtype or delta form                     */
    SDM_ERR_ALIGN = 4,        /* a device pointer is not 16-byte aligned         */
    SDM_ERR_UNSUPPORTED = 5,  /* valid but outside the sizes the kernels cover   */
    SDM_ERR_HIP = 6,          /* a HIP launch failed                             */
    SDM_ERR_WORKSPACE = 7     /* workspace missing or too small                  */
} sdm_status;

/* SDM_E4M3 (8-bit floats of 4 exponent and 3 mantissa bits, largest value 448)
 * is an output type of sdm_residual_norm and sdm_residual_layer_norm only. */
typedef enum sdm_dtype { SDM_F32 = 0, SDM_BF16 = 1, SDM_E4M3 = 2 } sdm_dtype;

/* The two write rules the notes keep side by side ([SDM] §2.4-§2.5):
 *   SDM_DELTA_EQ4:  M[i] <- a M[i] + b w_i (v - a M[i])         (Eq. (4), per slot)
 *   SDM_DELTA_FIG2: vhat = sum_j w_j a M[j];  M[i] <- a M[i] + b w_i (v - vhat)
 *                   (shared residual read off Fig. 2; equals the gated delta
 *                   rule Eq. (2) when every slot is selected).            */
typedef enum sdm_delta_form { SDM_DELTA_EQ4 = 0, SDM_DELTA_FIG2 = 1 } sdm_delta_form;

/* SDM_ABI_VERSION of the loaded library. */
int sdm_abi_version(void);

/* Static text for a status code. */
const char* sdm_status_string(int status);

/* Detail of the last failing call on the calling thread ("" if none). */
const char* sdm_last_error(void);

/*
 * sdm_address -- product-key addressing of both branches ([SDM] §2.3, §2.2
 * notation; [FwPKM] §2.2).
 *
 * For each (b, h, t) and each branch (write with k = W, read with k = R):
 *   half-scores  s_j[a] = <q[.., j, :], subkeys[h, j, a, :]>, j in {0, 1}, a < n_sub
 *                (MFMA contraction, fp32 accumulation);
 *   per half     keep the k_h = min(k, n_sub) best, ordered (score desc, index asc);
 *   combine      slot (a, b) -> row a*n_sub + b with score fp32(s_0[a] + s_1[b]);
 *                the k best candidate slots, ordered (score desc, slot asc);
 *   weights      softmax over the k selected slot scores.
 *
 *   q_w, q_r             [B, H, T, 2, dh]   q_dtype (half 0 then half 1)
 *   subkeys_w, subkeys_r [H, 2, n_sub, dh]  k_dtype == q_dtype (may alias)
 *   idx_w, wt_w          [B, H, T, W]       int32 slots, fp32 weights (out)
 *   idx_r, wt_r          [B, H, T, R]       (out)
 *   score_w, score_r     [B, H, T, W|R]     optional (NULL): fp32 slot scores
 *
 * Supported: q_dtype in {SDM_F32, SDM_BF16}; n_sub a multiple of 16 up to 512;
 * dh a multiple of 8 (fp32) or 32 (bf16) up to 256; 1 <= W, R <= min(64, n_sub^2);
 * B * T < 2^32 tokens per call.
 */
int sdm_address(const void* q_w, const void* q_r, int q_dtype,
                const void* subkeys_w, const void* subkeys_r, int k_dtype,
                int64_t B, int64_t H, int64_t T, int64_t n_sub, int64_t dh,
                int64_t W, int64_t R,
                int32_t* idx_w, float* wt_w, int32_t* idx_r, float* wt_r,
                float* score_w, float* score_r, void* stream);

/*
 * sdm_debug_half_scores -- test hook: only the half-score contraction of
 * sdm_address (same kernel code), for one branch.
 *   q [B, H, T, 2, dh], subkeys [H, 2, n_sub, dh], half [B, H, T, 2, n_sub] fp32 (out).
 * Same support as sdm_address.
 */
int sdm_debug_half_scores(const void* q, int q_dtype, const void* subkeys, int k_dtype,
                          int64_t B, int64_t H, int64_t T, int64_t n_sub, int64_t dh,
                          float* half, void* stream);

/*
 * sdm_address_idw -- sdm_address with FwPKM's inverse-distance subkey score
 * ([FwPKM] §2.2, FwPKM's default scoring) in place of the dot product:
 *   half-scores  s_j[a] = -log(1e-3 + ||q[.., j, :] - subkeys[h, j, a, :]||^2)
 * (computed as ||q||^2 + ||K_a||^2 - 2 <q, K_a>, the inner product on MFMA with
 * fp32 accumulation). Per-half top-k, the outer sum, the selection and the
 * softmax are those of sdm_address, so the weights of the selected slots are
 * the normalised products 1 / ((1e-3 + d_0)(1e-3 + d_1)) of the two halves'
 * squared distances. Arguments, layouts, errors and support as sdm_address.
 */
int sdm_address_idw(const void* q_w, const void* q_r, int q_dtype,
                    const void* subkeys_w, const void* subkeys_r, int k_dtype,
                    int64_t B, int64_t H, int64_t T, int64_t n_sub, int64_t dh,
                    int64_t W, int64_t R,
                    int32_t* idx_w, float* wt_w, int32_t* idx_r, float* wt_r,
                    float* score_w, float* score_r, void* stream);

/*
 * sdm_debug_half_scores_idw -- test hook: the inverse-distance half-scores of
 * sdm_address_idw alone (same kernel code), for one branch. Arguments as
 * sdm_debug_half_scores.
 */
int sdm_debug_half_scores_idw(const void* q, int q_dtype, const void* subkeys, int k_dtype,
                              int64_t B, int64_t H, int64_t T, int64_t n_sub, int64_t dh,
                              float* half, void* stream);

/*
 * sdm_state_init -- per-sequence initial table from the (learned) initial
 * state M0 ([SDM] §2.6): M[b] = M0 for every b.
 *   M0 [H, N, dv] fp32, M [B, H, N, dv] (out) in m_dtype: SDM_F32 (a copy) or
 *   SDM_BF16 (each element rounded to nearest-even bfloat16). dv must be a
 *   multiple of 4.
 */
int sdm_state_init(const float* M0, void* M, int m_dtype, int64_t B, int64_t H, int64_t N,
                   int64_t dv, void* stream);

/*
 * sdm_scan_workspace_bytes -- device workspace sdm_scan_forward needs for these
 * sizes (0 when there is no work, -1 when the sizes are invalid).
 */
int64_t sdm_scan_workspace_bytes(int64_t B, int64_t H, int64_t T, int64_t W, int64_t R,
                                 int64_t dv);

/*
 * sdm_scan_forward -- the sparse gated delta recurrence with its sparse read,
 * sequential in t for each (b, h) ([SDM] §2.4 Eq. (3)-(5), §2.5 Fig. 2):
 *   for t = 0 .. T-1:
 *     for i in idx_w[b,h,t,:]:  Mt = alpha[b,h,t] * M[b,h,i,:]              (Eq. 3)
 *                               M[b,h,i,:] = Mt + beta * wt_w_i * (v - P_i)
 *                               P_i = Mt (EQ4)  or  sum_j wt_w_j * alpha * M[b,h,j,:] (FIG2)
 *     y[b,h,t,:] = sum_i wt_r_i * M[b,h,idx_r_i,:]   (after this token's writes, Eq. 5)
 *   Rows that no token selects for writing are never touched (bit-identical).
 *
 *   idx_w, wt_w  [B, H, T, W]   int32 / fp32     idx_r, wt_r [B, H, T, R]
 *   alpha, beta  [B, H, T]      fp32 gates
 *   v            [B, H, T, dv]  v_dtype (SDM_F32 or SDM_BF16)
 *   M            [B, H, N, dv]  m_dtype, in: state before token 0, out: after token T-1
 *   y            [B, H, T, dv]  fp32 (out)
 *   m_dtype      SDM_F32, or SDM_BF16: the table is stored in bfloat16 (the
 *                2-byte state elements the notes' per-layer state size implies,
 *                [SDM] §4.5 Table 3 with §2.8's element count); each update is
 *                computed in fp32 from the widened row and stored rounded to
 *                nearest even, halving the bytes of every row access
 *   workspace    device buffer of >= sdm_scan_workspace_bytes(B,H,T,W,R,dv) bytes,
 *                16-byte aligned; its contents on entry do not matter.
 *
 * The state is in/out, so a sequence split over several calls gives the same
 * result as one call. Preconditions: indices in [0, N) and the W write indices
 * of one token distinct (sdm_address guarantees both). Entries that break the
 * first are skipped (memory-safe, result unspecified); the second gives an
 * unspecified result. Weights are used as given.
 * Supported: 1 <= W, R <= 256, N <= 2^18, dv a multiple of 4 (of 8 for a bf16
 * table), N * dv * 4 < 2^31.
 */
int sdm_scan_forward(const int32_t* idx_w, const float* wt_w, int64_t W,
                     const int32_t* idx_r, const float* wt_r, int64_t R,
                     const float* alpha, const float* beta,
                     const void* v, int v_dtype,
                     void* M, int m_dtype, float* y,
                     int64_t B, int64_t H, int64_t T, int64_t N, int64_t dv,
                     int form, void* workspace, int64_t workspace_bytes, void* stream);

/*
 * sdm_scan_gated_workspace_bytes -- device workspace sdm_scan_forward_gated
 * needs: sdm_scan_workspace_bytes rounded up to 256, plus B*H*T*dv*4 bytes for
 * y in the calls that keep it themselves (0 when there is no work, -1 when the
 * sizes are invalid).
 */
int64_t sdm_scan_gated_workspace_bytes(int64_t B, int64_t H, int64_t T, int64_t W, int64_t R,
                                       int64_t dv);

/*
 * sdm_scan_forward_gated -- sdm_scan_forward followed by the head's output step
 * of the SDM layer ([SDM] §2.4: the read, then RMS-Norm and the output gate;
 * the same step as sdm_output_gate):
 *   o[b,h,t,i] = y[b,h,t,i] / sqrt(mean_j y[b,h,t,j]^2 + eps) * gamma[h,i] * sigmoid(g[b,h,t,i])
 * Arguments as sdm_scan_forward and sdm_output_gate, except:
 *   y          [B, H, T, dv] fp32 (out), or NULL: then y is not returned
 *   gamma      [H, dv] fp32; g [B, H, T, dv] g_dtype (SDM_F32 or SDM_BF16);
 *   eps >= 0;  o [B, H, T, dv] fp32 (out), not aliasing y
 *   workspace  >= sdm_scan_gated_workspace_bytes(B,H,T,W,R,dv) bytes, 16-byte aligned
 * The table M and y are bit-identical to sdm_scan_forward's, and o to
 * sdm_output_gate applied to that y. Where the scan splits the table rows into
 * partitions whose partial sums of y a last pass adds (long calls: the usual
 * case), that pass also normalises and gates each row while it holds it in
 * registers (d_v <= 1024), so y is stored only if requested and never read
 * back; otherwise y is stored (to `y`, or the workspace) and the output step
 * runs after the scan. Same support as sdm_scan_forward, and B*H*T < 2^32.
 */
int sdm_scan_forward_gated(const int32_t* idx_w, const float* wt_w, int64_t W,
                           const int32_t* idx_r, const float* wt_r, int64_t R,
                           const float* alpha, const float* beta,
                           const void* v, int v_dtype,
                           void* M, int m_dtype, float* y,
                           const float* gamma, const void* g, int g_dtype, float eps, float* o,
                           int64_t B, int64_t H, int64_t T, int64_t N, int64_t dv,
                           int form, void* workspace, int64_t workspace_bytes, void* stream);

/*
 * sdm_scan_forward_noalloc -- sdm_scan_forward without a workspace argument, for
 * callers that cannot allocate device memory (code under HIP graph capture,
 * tight serving loops, harnesses that forbid hipMalloc). Arguments, layouts,
 * results and support as sdm_scan_forward (the table and y are bit-identical
 * to it), except:
 *   - the scan's scratch (plan records, partial sums, counters) is one array of
 *     64 MiB per GPU inside the library, held from the first call on that GPU
 *     until the process ends; the call allocates and frees nothing;
 *   - calls of more tokens than that scratch holds at once are run as several
 *     launch chunks in order (the same result: the state carries over exactly);
 *     a call whose streams need more than 64 MiB for even one token per launch
 *     (B*H in the thousands) returns SDM_ERR_UNSUPPORTED;
 *   - every call on a GPU uses that GPU's one array, so calls that overlap in
 *     time on one GPU (on different streams or from different threads) race and
 *     give unspecified results; calls on one stream are ordered and safe;
 *   - `stream` selects the GPU (its device), else the current device.
 */
int sdm_scan_forward_noalloc(const int32_t* idx_w, const float* wt_w, int64_t W,
                             const int32_t* idx_r, const float* wt_r, int64_t R,
                             const float* alpha, const float* beta,
                             const void* v, int v_dtype,
                             void* M, int m_dtype, float* y,
                             int64_t B, int64_t H, int64_t T, int64_t N, int64_t dv,
                             int form, void* stream);

/*
 * Training: the forward with pre-images, then the backward that undoes it.
 * ([SDM] §2.9 Appendix A, backward memory: the forward writes the table in
 * place; the backward walks the tokens in reverse and restores each written
 * row from its stored pre-image, so the memory is O(N*dv + T*W*dv) instead of
 * one table per step.)
 */

/*
 * sdm_scan_snapshot_bytes -- bytes of the pre-image buffer for these sizes:
 * B*H*T*W*dv*4 (-1 when the sizes are invalid).
 */
int64_t sdm_scan_snapshot_bytes(int64_t B, int64_t H, int64_t T, int64_t W, int64_t dv);

/*
 * sdm_scan_forward_save -- sdm_scan_forward on an fp32 table (same arguments
 * but m_dtype; M bit-identical to it, y equal up to the order in which the read
 * rows are added) that also
 * stores, for every write, the row as it was before this token's decay:
 *   snap [B, H, T, W, dv] fp32 (out): snap[b,h,t,p,:] = M_{t-1}[b,h,idx_w[b,h,t,p],:]
 * The workspace is the one sdm_scan_workspace_bytes gives. Same support as
 * sdm_scan_forward.
 */
int sdm_scan_forward_save(const int32_t* idx_w, const float* wt_w, int64_t W,
                          const int32_t* idx_r, const float* wt_r, int64_t R,
                          const float* alpha, const float* beta,
                          const void* v, int v_dtype,
                          float* M, float* y, float* snap,
                          int64_t B, int64_t H, int64_t T, int64_t N, int64_t dv,
                          int form, void* workspace, int64_t workspace_bytes, void* stream);

/*
 * sdm_scan_backward_workspace_bytes -- device workspace sdm_scan_backward needs
 * (per-slab partial sums of the weight and gate gradients, and the planner's
 * W + 2R source words per token and stream that let the reverse walk load a
 * token's rows several tokens early); 0 when there is no work, -1 when the
 * sizes are invalid.
 */
int64_t sdm_scan_backward_workspace_bytes(int64_t B, int64_t H, int64_t T, int64_t W, int64_t R,
                                          int64_t dv);

/*
 * sdm_scan_backward -- reverse-mode derivatives of one sdm_scan_forward_save
 * call, tokens T-1 .. 0, with the forward's writes undone in place.
 *   idx_w, wt_w, idx_r, wt_r, alpha, beta, v, form: as given to the forward call
 *   snap  [B, H, T, W, dv] fp32: the forward call's pre-images
 *   dy    [B, H, T, dv] fp32: dL/dy
 *   M     [B, H, N, dv] fp32, in: the state after the forward call;
 *         out: the state before it (bit-identical to what the forward got)
 *   dM    [B, H, N, dv] fp32, in: dL/dM after the call (zeros if the final state
 *         does not enter the loss); out: dL/dM before the call
 *   dv_out [B, H, T, dv], dalpha, dbeta [B, H, T], dwt_w [B, H, T, W],
 *   dwt_r [B, H, T, R]: fp32 gradients (out)
 *   workspace: >= sdm_scan_backward_workspace_bytes(B,H,T,W,R,dv) bytes, 16-byte aligned
 * A sequence split into forward calls is differentiated call by call, last
 * call first, passing M and dM along. Preconditions: those of the forward, and
 * also the R read indices of one token distinct (sdm_address guarantees it).
 * Supported: as sdm_scan_forward; W, R <= 256 with ceil(W/G) + ceil(R/G) <= 16
 * wavefronts for some slab width (G = 64 / (S / 4) rows per wavefront, S in
 * {4, 8, 16, 32} dividing dv).
 */
int sdm_scan_backward(const int32_t* idx_w, const float* wt_w, int64_t W,
                      const int32_t* idx_r, const float* wt_r, int64_t R,
                      const float* alpha, const float* beta,
                      const void* v, int v_dtype, const float* snap, const float* dy,
                      float* M, float* dM,
                      float* dv_out, float* dalpha, float* dbeta, float* dwt_w, float* dwt_r,
                      int64_t B, int64_t H, int64_t T, int64_t N, int64_t dv,
                      int form, void* workspace, int64_t workspace_bytes, void* stream);

/*
 * sdm_state_init_backward -- adjoint of sdm_state_init: the gradient of the
 * shared initial state, dM0[h] = sum over b of dM[b, h] (added in b order).
 *   dM [B, H, N, dv] fp32, dM0 [H, N, dv] fp32 (out). dv a multiple of 4.
 */
int sdm_state_init_backward(const float* dM, float* dM0, int64_t B, int64_t H, int64_t N,
                            int64_t dv, void* stream);

/*
 * The steps either side of the scan ([SDM] §2.4).
 *
 * sdm_gates -- the scan's per-head scalar gates from the layer input:
 *   alpha[b,h,t] = exp(-A[h] * softplus(<W_a[h,:], x[b,t,:]> + b_dt[h]))
 *   beta[b,h,t]  = sigmoid(<W_b[h,:], x[b,t,:]>)
 * The projections of all heads are one MFMA contraction over d with fp32
 * accumulation (bf16 or fp32 operands); softplus, exp and sigmoid in fp32.
 *   x [B, T, d] x_dtype; W_a, W_b [H, d] w_dtype == x_dtype; b_dt, A [H] fp32;
 *   alpha, beta [B, H, T] fp32 (out): the layout sdm_scan_forward reads.
 * Supported: d a multiple of 32 (bf16) or 8 (fp32) up to 2^20, H <= 4096,
 * B * T < 2^32 tokens per call.
 */
int sdm_gates(const void* x, int x_dtype, const void* W_a, const void* W_b, int w_dtype,
              const float* b_dt, const float* A, int64_t B, int64_t T, int64_t d, int64_t H,
              float* alpha, float* beta, void* stream);

/*
 * sdm_output_gate -- each head's output after the read: RMS-Norm of the row
 * y[b,h,t,:], then the elementwise output gate; the gate's activation is taken
 * to be the sigmoid ([FwPKM] §2.3's output gate; the SDM notes name the gate
 * without its activation):
 *   o[b,h,t,i] = y[b,h,t,i] / sqrt(mean_j y[b,h,t,j]^2 + eps) * gamma[h,i] * sigmoid(g[b,h,t,i])
 *   y, o [B, H, T, dv] fp32; g [B, H, T, dv] g_dtype (gate pre-activation);
 *   gamma [H, dv] fp32; eps >= 0. o may not alias y. dv a multiple of 4;
 *   B * H * T < 2^32 rows per call.
 * The head-mixing projection W_o that follows is a plain dense layer and is
 * not part of this library.
 */
int sdm_output_gate(const float* y, const float* gamma, const void* g, int g_dtype, float eps,
                    int64_t B, int64_t H, int64_t T, int64_t dv, float* o, void* stream);

/*
 * The dense gated recurrence: the layers that a stack puts beside its sparse
 * ones, with the scan's gates, v and y ([SDM] §2.1 Eq. (1) without its normalised
 * read, with the gates of §2.4: a state of dk rows, all of them decayed and written
 * by every token). A write adds beta k (x) v as it is; it is not the delta rule, which
 * first takes off what the state holds for k (Eq. (2)).
 */

/*
 * sdm_dense_scan_workspace_bytes -- device workspace sdm_dense_scan_forward
 * needs (0: none, as when there is no work, for short calls or many streams; -1:
 * sizes that the call refuses).
 */
int64_t sdm_dense_scan_workspace_bytes(int64_t B, int64_t H, int64_t T, int64_t dk, int64_t dv);

/*
 * sdm_dense_scan_forward -- for t = 0 .. T-1, for each (b, h):
 *     S_t = alpha_t S_{t-1} + beta_t k_t (x) v_t
 *     y_t = q_t S_t                                  (after this token's write)
 *   q, k         [B, H, T, dk]  in_dtype (SDM_F32 or SDM_BF16); a scale of the
 *                queries is the caller's
 *   v            [B, H, T, dv]  in_dtype
 *   alpha, beta  [B, H, T]      fp32 gates (as sdm_gates writes them; alpha = 0
 *                starts a new sequence, alpha = 1 with beta = 0 skips a token)
 *   S0           [B, H, dk, dv] fp32: the state before token 0, or NULL (zeros)
 *   S            [B, H, dk, dv] fp32 (out): the state after token T-1, or NULL
 *                (not wanted); may be S0 itself (decoding)
 *   y            [B, H, T, dv]  fp32 (out), the layout sdm_output_gate reads
 *   workspace    >= sdm_dense_scan_workspace_bytes bytes, 16-byte aligned (may be
 *                NULL where that is 0)
 * Products and sums are fp32 for both input types, states fp32. A sequence may
 * be split over several calls. Inputs and states must be finite, fp32 ones below 2^127 in
 * magnitude: tokens are worked in tiles, and a NaN or infinity may reach earlier tokens
 * of its tile. T = 0
 * passes the state on (S = S0).
 * Supported: dk, dv multiples of 8 up to 256; B*H*ceil(T/64)*8 < 2^31,
 * B*H*ceil(T/512)*ceil(max(dk,dv)/64) < 2^21, B*H*dk*dv < 2^34 - 2^10.
 */
int sdm_dense_scan_forward(const void* q, const void* k, const void* v, int in_dtype,
                           const float* alpha, const float* beta, const float* S0, float* S, float* y,
                           int64_t B, int64_t H, int64_t T, int64_t dk, int64_t dv,
                           void* workspace, int64_t workspace_bytes, void* stream);

/*
 * sdm_dense_scan_backward_workspace_bytes -- device workspace
 * sdm_dense_scan_backward needs: the states S and G at the bounds of segments
 * of at most 512 tokens, and a few numbers a token (0: no work, -1: sizes that the
 * call refuses).
 */
int64_t sdm_dense_scan_backward_workspace_bytes(int64_t B, int64_t H, int64_t T, int64_t dk, int64_t dv);

/*
 * sdm_dense_scan_backward -- the gradients of sdm_dense_scan_forward, with
 *   G_t = alpha_{t+1} G_{t+1} + q_t (x) dy_t, and dL/dS_T in place of alpha G past the end:
 *   dq_t = S_t dy_t    dk_t = beta_t G_t v_t    dv_t = beta_t G_t^T k_t    dbeta_t = k_t^T G_t v_t
 *   dlog_alpha_t = alpha_t dL/dalpha_t = <G_t, alpha_t S_{t-1}>
 * The decay's gradient is the one to ln alpha: it is finite for alpha = 0, and
 * with alpha = exp(-A softplus(z)) the gate's inputs follow as
 * dz = -A sigmoid(z) dlog_alpha, dA = -softplus(z) dlog_alpha. It is formed as a running
 * difference of q.dq and k.dk: its error is some 2^-20 of those and of the neighbouring
 * tokens' values, not of its own, so do not divide it by a tiny alpha.
 *   q, k, v, in_dtype, alpha, beta, S0: as given to the forward call
 *   dy [B, H, T, dv] fp32: dL/dy;  dS [B, H, dk, dv] fp32: dL/dS, or NULL (zeros)
 *   dq, dk_out [B, H, T, dk], dv_out [B, H, T, dv], dlog_alpha, dbeta [B, H, T]: fp32 (out)
 *   dS0 [B, H, dk, dv] fp32 (out): dL/dS0, or NULL (not wanted); may be dS itself
 *   workspace >= sdm_dense_scan_backward_workspace_bytes bytes, 16-byte aligned
 * The states are formed again from the inputs; nothing is kept from the forward
 * call. Split sequences are differentiated last call first, dS0 passed on as dS.
 * Same support and preconditions as the forward; T = 0 gives dS0 = dS.
 */
int sdm_dense_scan_backward(const void* q, const void* k, const void* v, int in_dtype,
                            const float* alpha, const float* beta, const float* dy,
                            const float* S0, const float* dS,
                            float* dq, float* dk_out, float* dv_out, float* dlog_alpha, float* dbeta, float* dS0,
                            int64_t B, int64_t H, int64_t T, int64_t dk, int64_t dv,
                            void* workspace, int64_t workspace_bytes, void* stream);

/*
 * sdm_residual_norm -- the residual stream's addition and RMS-Norm in front of a
 * layer, per row (token):
 *   h = x + res,   y = h / sqrt(mean_j h_j^2 + eps) * gamma
 *   x [rows, d] x_dtype;  res [rows, d], h [rows, d] (out) h_dtype, both or neither
 *   NULL (then h = x and nothing is stored; h_dtype still names a dtype);
 *   gamma [d] fp32; eps >= 0
 *   y [rows, d] (out) y_dtype: SDM_F32, SDM_BF16, or SDM_E4M3 with
 *   scale (out, fp32; else unused, may be NULL): with group = 0 one per row, [rows, 1]; else
 *   one per `group` columns, [rows, d / group]. scale = max |y| / 448 over its columns (0
 *   where all are 0, else at least 2^-126), and y holds the fp32 quotients y / scale, rounded
 *   to nearest even; where a y is NaN or infinite, so is the scale, and all of its y are NaN
 * The norm is that of the fp32 sum; h is stored rounded to its dtype. h may
 * be res, or x in x's dtype (in place); y may not alias x, res or h. The squares are
 * summed in fp32: their sum must stay below 2^128 (y is 0 beyond), and above 0 where
 * eps = 0 (a row of zeros gives NaN then).
 * Supported: 1 <= d <= 16384; group 0, or a power of two from 32 to 512 that
 * divides d; rows < 2^31. rows = 0 is empty work.
 */
int sdm_residual_norm(const void* x, int x_dtype, const void* res, void* h, int h_dtype, const float* gamma,
                      float eps, int64_t rows, int64_t d, void* y, int y_dtype, float* scale, int64_t group,
                      void* stream);

/*
 * sdm_residual_norm_backward_workspace_bytes -- device workspace
 * sdm_residual_norm_backward needs (0: no work, -1: invalid sizes).
 */
int64_t sdm_residual_norm_backward_workspace_bytes(int64_t rows, int64_t d);

/*
 * sdm_residual_norm_backward -- its gradients, from the stored h (x where there was no
 * residual), with r = 1 / sqrt(mean h^2 + eps) and n = h r:
 *   dx = dh + r (gamma dy - n mean_j(gamma dy n)),   dgamma = sum over rows of dy n
 *   dy [rows, d]: dL/dy; dh [rows, d]: what arrives at h from the layers behind, or
 *   NULL (nothing); dx [rows, d] (out): the gradient of x and of res alike; all three
 *   g_dtype; h [rows, d] h_dtype; gamma [d], dgamma [d] (out) fp32
 *   workspace >= sdm_residual_norm_backward_workspace_bytes bytes, 16-byte aligned
 * dx may be dy or dh, or h in h's dtype. The sums' order follows from the sizes alone.
 * Support as sdm_residual_norm; rows = 0 is empty work (dgamma is not written).
 */
int sdm_residual_norm_backward(const void* dy, const void* dh, int g_dtype, const void* h, int h_dtype,
                               const float* gamma, float eps, int64_t rows, int64_t d, void* dx, float* dgamma,
                               void* workspace, int64_t workspace_bytes, void* stream);

/*
 * sdm_balance_workspace_bytes -- device workspace sdm_balance_forward needs (-1:
 * invalid sizes).
 */
int64_t sdm_balance_workspace_bytes(int64_t B, int64_t H, int64_t T, int64_t K, int64_t N);

/*
 * sdm_balance_forward -- how evenly an addressing result uses the slots, per
 * head over the n tokens that the mask keeps:
 *   counts[h,i] = selections of slot i;   mass[h,i] = the sum of their weights
 *   loss[h] = N sum_i f_i P_i,  f_i = counts / (n K),  P_i = mass / n
 * (1 when the slots are chosen evenly with weights that sum to 1, N / K when
 * all tokens choose the same K; 0 when no token is kept).
 *   idx, wt  [B, H, T, K]  int32 slots, fp32 weights, as sdm_address writes them
 *            (W or R as K); |wt| <= 2
 *   mask     [B, T] bytes, non-zero: kept; or NULL (all are). Any alignment
 *   counts, mass [H, N]  int32 / fp32 (out);  tokens [1] int32 (out): n;  loss [H] fp32 (out)
 *   workspace >= sdm_balance_workspace_bytes bytes, 16-byte aligned
 * Selections outside [0, N) are left out; a kept weight that is NaN or beyond 2
 * in magnitude makes its head's mass and loss NaN. Masked tokens are not
 * looked at. Weights are added in fixed point (to 2^-40, or with more than 2^21
 * selections a head, n = B*T*K, to 2^-(61 - ceil(log2 n))), so results do not
 * depend on the order of the additions. Without tokens (B or T = 0) the outputs are zeros;
 * H = 0 is empty work (tokens is not written).
 * Supported: N <= 2^18, K <= 256, H <= 4096, B*T*K < 2^31.
 */
int sdm_balance_forward(const int32_t* idx, const float* wt, const uint8_t* mask,
                        int64_t B, int64_t H, int64_t T, int64_t K, int64_t N,
                        int32_t* counts, float* mass, int32_t* tokens, float* loss,
                        void* workspace, int64_t workspace_bytes, void* stream);

/*
 * sdm_balance_backward -- the loss's gradient to the weights (the counts are
 * constants): dwt[b,h,t,p] = dloss[h] N / n * f[idx] at kept tokens and slots in
 * range, 0 elsewhere. It adds to what sdm_scan_backward gives for the same weights.
 *   idx, mask as given, counts and tokens as written by the forward call;
 *   dloss [H] fp32: dL/dloss;  dwt [B, H, T, K] fp32 (out)
 */
int sdm_balance_backward(const int32_t* idx, const uint8_t* mask, const int32_t* counts, const int32_t* tokens,
                         const float* dloss, int64_t B, int64_t H, int64_t T, int64_t K, int64_t N, float* dwt,
                         void* stream);

/*
 * A selective state-space layer's operators: the layers of a state per channel that a stack puts
 * beside its sparse and dense ones. The convolution is also what a dense layer has on its q, k and v.
 *
 * Tensors said to be "by strides" are rows of consecutive channels at any address that their elements'
 * size divides; their strides (in elements, not negative) are an array in host memory, or NULL for a
 * contiguous tensor. Everything else follows the conventions above.
 *
 * start [B, T] bytes or NULL: non-zero where a sequence begins (packed sequences): a token sees nothing
 * in front of it. lengths [B] int32 or NULL: only the first lengths[b] tokens are there (padded
 * sequences; taken into [0, T]); the others are not looked at, outputs and gradients there are 0, and the last state
 * is the one behind the last token that is there. Both: any alignment that their elements allow.
 */

/* Activations behind the convolution. */
typedef enum sdm_act { SDM_ACT_NONE = 0, SDM_ACT_SILU = 1 } sdm_act;

/*
 * sdm_causal_conv_forward -- the short causal convolution over time of every channel:
 *     y_t = act(bias + sum_j w_j x_{t-K+1+j}),   j = 0 .. K-1
 *   x       [B, H, T, d]    dtype (SDM_F32 or SDM_BF16), by strides [3]: batch, head, token (heads out of a
 *                           projection [B, T, H, d] need no copy; H = 1 for a layer without heads)
 *   w       [H, d, K], bias [H, d] fp32 (bias may be NULL)
 *   S0      [B, H, K-1, d]  dtype: the K-1 inputs in front of token 0, oldest first, or NULL (zeros)
 *   S       [B, H, K-1, d]  dtype (out): those behind the last token, or NULL (not wanted); may be S0
 *                           (decoding), and may not overlap another input. Rows in front of the last
 *                           sequence's first token are 0
 *   y       [B, H, T, d]    dtype (out); may not overlap x, S0 or S
 * Products and sums are fp32. T = 0 passes the state on.
 * Supported: K from 2 to 8; H*d <= 2^23, B*ceil(T/8)*ceil(H*d/64) < 2^26.
 */
int sdm_causal_conv_forward(const void* x, int dtype, const int64_t* x_strides, const float* w, const float* bias,
                            int act, const void* S0, void* S, const uint8_t* start, const int32_t* lengths, void* y,
                            int64_t B, int64_t H, int64_t T, int64_t d, int64_t K, void* stream);

/*
 * sdm_causal_conv_backward_workspace_bytes -- device workspace sdm_causal_conv_backward needs (0: no work;
 * -1: sizes that the call refuses).
 */
int64_t sdm_causal_conv_backward_workspace_bytes(int64_t B, int64_t H, int64_t T, int64_t d, int64_t K);

/*
 * sdm_causal_conv_backward -- its gradients; nothing is kept from the forward call.
 *   dy [B, H, T, d] dtype: dL/dy;  x, w, bias, act, S0, start, lengths as given to the forward call
 *   dS [B, H, K-1, d] dtype: dL/dS, or NULL (zeros)
 *   dx [B, H, T, d] dtype (out), by strides [3] (so that it may be a part of a projection's gradient); its
 *   elements may not share an address, nor overlap an input
 *   dw [H, d, K], dbias [H, d] fp32 (out; dbias may be NULL), summed over all tokens in an order that
 *   follows from the sizes alone;  dS0 [B, H, K-1, d] dtype (out), or NULL; may be dS only where T = 0.
 *   Outputs may not overlap each other, nor, that apart, an input
 *   workspace >= sdm_causal_conv_backward_workspace_bytes bytes, 16-byte aligned
 * Same support as the forward. B = 0 is empty work (dw and dbias are not written).
 */
int sdm_causal_conv_backward(const void* dy, const void* x, int dtype, const int64_t* x_strides, const float* w,
                             const float* bias, int act, const void* S0, const void* dS, const uint8_t* start,
                             const int32_t* lengths, void* dx, const int64_t* dx_strides, float* dw, float* dbias,
                             void* dS0, int64_t B, int64_t H, int64_t T, int64_t d, int64_t K, void* workspace,
                             int64_t workspace_bytes, void* stream);

/*
 * sdm_selective_scan_workspace_bytes -- device workspace sdm_selective_scan_forward needs (0: none, as when there
 * is no work, for short calls or many streams of channels; -1: sizes that the call refuses). Fewer sequences or
 * tokens can need more than many (2048 channels, 16 states, 4096 tokens: 36 MB for 32 sequences, none for 48):
 * one workspace for calls of several sizes is as large as the largest of their answers.
 */
int64_t sdm_selective_scan_workspace_bytes(int64_t B, int64_t T, int64_t D, int64_t G, int64_t N);

/*
 * sdm_selective_scan_forward -- for every channel d (of group g = d / (D / G)) and state n:
 *     delta_t = softplus(dt_t + dt_bias)               (or dt_t + dt_bias, softplus = 0)
 *     h_t = exp(delta_t A) h_{t-1} + delta_t x_t B_t
 *     y_t = (sum_n C_t h_t + D x_t) z_t sigmoid(z_t)   (without the last factors where z is NULL)
 *   x, dt, z  [B, T, D]     in_dtype (SDM_F32 or SDM_BF16), by strides (z may be NULL)
 *   Bm, Cm    [B, T, G, N]  in_dtype, by strides
 *   strides   [12]: x's batch and token, dt's, z's, then Bm's batch, token and group, and Cm's
 *   A [D, N], Dskip [D] (or NULL), dt_bias [D] (or NULL) fp32
 *   S0        [B, D, N]     fp32: the state before token 0, or NULL (zeros)
 *   S         [B, D, N]     fp32 (out): the state behind the last token, or NULL; may be S0 (decoding), and may
 *                           not overlap another input
 *   y         [B, T, D]     in_dtype (out); may not overlap an input
 *   workspace >= sdm_selective_scan_workspace_bytes bytes, 16-byte aligned (may be NULL where that is 0)
 * Products, sums and states are fp32. Meant for delta A <= 0; inputs and states must be finite (a NaN or
 * infinity in one channel's x, dt, z or state stays in that channel). T = 0 passes the state on.
 * Supported: N <= 64, D <= 2^20 with G dividing it, B*G*ceil(D/G/64)*ceil(N/16) < 2^22, token
 * strides below 2^26.
 */
int sdm_selective_scan_forward(const void* x, const void* dt, const void* z, const void* Bm, const void* Cm,
                               int in_dtype, const int64_t* strides, const float* A, const float* Dskip,
                               const float* dt_bias, int softplus, const float* S0, float* S, const uint8_t* start,
                               const int32_t* lengths, void* y, int64_t B, int64_t T, int64_t D, int64_t G, int64_t N,
                               void* workspace, int64_t workspace_bytes, void* stream);

/*
 * sdm_selective_scan_backward_workspace_bytes -- device workspace sdm_selective_scan_backward needs: a state
 * every 8 tokens and rows of partial sums (0: no work; -1: sizes that the call refuses; calls of several sizes as
 * there).
 */
int64_t sdm_selective_scan_backward_workspace_bytes(int64_t B, int64_t T, int64_t D, int64_t G, int64_t N);

/*
 * sdm_selective_scan_backward -- its gradients; nothing is kept from the forward call.
 *   dy [B, T, D] in_dtype, by strides: dL/dy;  strides [14]: the forward call's, then dy's batch and token
 *   dS [B, D, N] fp32: dL/dS, or NULL (zeros); the other inputs as given to the forward call
 *   dx, ddt, dz [B, T, D] in_dtype (out; dz NULL where z is)
 *   dA [D, N], dB, dC [B, T, G, N], dD, ddt_bias [D], dS0 [B, D, N] fp32 (out; dD, ddt_bias and dS0 may be
 *   NULL; dS0 may be dS). Outputs may not overlap each other, nor, that apart, an input
 *   workspace >= sdm_selective_scan_backward_workspace_bytes bytes, 16-byte aligned
 * The order of all sums follows from the sizes alone. Same support as the forward, and
 * B*T*G*ceil(N/16) <= 2^27 - 8, G*ceil(D/G/64)*ceil(N/16) < 2^17.
 * B = 0 is empty work (dA, dD and ddt_bias are not written).
 */
int sdm_selective_scan_backward(const void* dy, const void* x, const void* dt, const void* z, const void* Bm,
                                const void* Cm, int in_dtype, const int64_t* strides, const float* A,
                                const float* Dskip, const float* dt_bias, int softplus, const float* S0,
                                const float* dS, const uint8_t* start, const int32_t* lengths, void* dx, void* ddt,
                                void* dz, float* dA, float* dB, float* dC, float* dD, float* ddt_bias, float* dS0,
                                int64_t B, int64_t T, int64_t D, int64_t G, int64_t N, void* workspace,
                                int64_t workspace_bytes, void* stream);

/*
 * sdm_residual_layer_norm -- sdm_residual_norm with the mean taken off and a bias, per row:
 *   h = x + res,   m = mean_j h_j,   y = (h - m) / sqrt(mean_j (h_j - m)^2 + eps) * gamma + bias
 *   bias [d] fp32, or NULL (zeros); everything else, e4m3 outputs with their scales among it, as there
 *   (y, h and scale may not overlap gamma, bias or each other)
 * The mean and the squares about it are summed in fp32, over the fp32 sums h.
 */
int sdm_residual_layer_norm(const void* x, int x_dtype, const void* res, void* h, int h_dtype, const float* gamma,
                            const float* bias, float eps, int64_t rows, int64_t d, void* y, int y_dtype, float* scale,
                            int64_t group, void* stream);

/*
 * sdm_residual_layer_norm_backward_workspace_bytes -- device workspace
 * sdm_residual_layer_norm_backward needs (0: no work, -1: invalid sizes).
 */
int64_t sdm_residual_layer_norm_backward_workspace_bytes(int64_t rows, int64_t d);

/*
 * sdm_residual_layer_norm_backward -- its gradients, from the stored h (x where there was no residual), with
 * r = 1 / sqrt(mean (h - m)^2 + eps) and n = (h - m) r:
 *   dx = dh + r (gamma dy - mean_j(gamma dy) - n mean_j(gamma dy n))
 *   dgamma = sum over rows of dy n,   dbias = sum over rows of dy (may be NULL)
 * Arguments, aliases and support as sdm_residual_norm_backward; dx, dgamma and dbias may not overlap each other
 * or gamma.
 */
int sdm_residual_layer_norm_backward(const void* dy, const void* dh, int g_dtype, const void* h, int h_dtype,
                                     const float* gamma, float eps, int64_t rows, int64_t d, void* dx, float* dgamma,
                                     float* dbias, void* workspace, int64_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* SDM_H */
