/*
 * moe_gb300.h -- C ABI of the routed ReLU^2 mixture-of-experts layer
 * (NemotronH-style MoE feed-forward block), hand-written CUDA for sm_103a.
 *
 * The layer, for hidden rows x[T, d]:
 *   (latent shapes)  x_e = bf16(x W_ld^T)                       [T, L]      else x_e = x
 *   router           z = x W_r^T (FP32), s = sigmoid(z) (FP32),
 *                    group-limited top-K on c = s + b, weights from s,
 *                    normalised, times routed_scaling_factor
 *   dispatch         per-expert counts, exclusive scan, routes sorted by
 *                    (expert, token, slot)
 *   experts          h = bf16(relu(bf16(x_e W_up,e^T))^2);  u = w * (h W_down,e^T)  (FP32)
 *   combine          y_r[t] = sum of t's routed rows in ascending expert id (FP32)
 *   shared + output  y_s = W_sd bf16(relu(bf16(W_su x))^2)  (FP32)
 *                    y = bf16(y_r + y_s)                       (no latent)
 *                    y = bf16(bf16(y_r) W_lu^T + y_s)          (latent)
 * Sources: page "Nemotron Is Not One Circuit: Mamba, Attention, and MoE
 * Routing" (sections "The Four Layer Kinds CKE Must Preserve", "The Router Is
 * A Deterministic Algorithm", "The C Kernel Contract"); page "M6.1 - Routed
 * Capacity: MoE Experts, Routers, and Token Dispatch" (sections 0x04A,
 * 0x05A-0x05F); page "NemotronH (Nemotron 3.5 Lightning, Bolt, Super VL)"
 * (section "Arithmetic"); page "Nemotron-3.5-Super 120B on an 8 GB GPU"
 * (section "The only number that matters", latent experts; section "The
 * engine, step by step", item 4, NVFP4 block scales).
 *
 * Conventions for every entry point:
 *  - Pointers are DEVICE pointers unless stated otherwise, allocated and owned
 *    by the caller; the library never allocates device memory, frees or
 *    synchronises (except moe_get_device_error and the _host convenience
 *    call).  Every call only enqueues work on `stream` (a cudaStream_t passed
 *    as void*; NULL = the legacy default stream) and returns.
 *    moe_layer_forward (and moe_block_forward) runs the latent down
 *    projection and the shared expert on a library-owned auxiliary stream
 *    (one per device, created with its events on the first call), forked
 *    from and joined back to `stream` by events, so the layer is still
 *    ordered as one operation on `stream`.  Calls from several host threads
 *    take turns enqueuing (a per-device lock is held while a call enqueues),
 *    and their auxiliary work runs one call after another on that one
 *    stream: correct, but two layers on different caller streams overlap
 *    only in their routed parts.
 *  - Row-major storage.  Weight matrices are stored [out, in] (the
 *    nn.Linear orientation, page "M6.1 ...", section 0x04A).
 *  - Every device pointer must be 16-byte aligned; every inner width
 *    (d_model, d_latent, d_expert, d_shared) a multiple of 64.
 *  - Argument and shape errors are returned before anything is enqueued.
 *    A failed launch returns MOE_ERR_CUDA.  Conditions only the device can see
 *    (an expert id out of range, a non-finite router score) set bits of the
 *    device error word held in the workspace; read it with
 *    moe_get_device_error.  Kernels never trap or assert.
 *  - Outputs are overwritten, never accumulated into.
 *  - Results are bit-identical from run to run for the same inputs and T
 *    (no floating-point atomics; every sum has a fixed order).
 */
#ifndef MOE_GB300_H
#define MOE_GB300_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef int32_t moe_status_t;
enum {
  MOE_OK = 0,
  MOE_ERR_INVALID_ARG = 1,  /* null/misaligned pointer, bad shape or parameter */
  MOE_ERR_UNSUPPORTED = 2,  /* valid but not built (e.g. a width not a multiple of 64) */
  MOE_ERR_WORKSPACE = 3,    /* workspace smaller than moe_workspace_bytes() */
  MOE_ERR_CUDA = 4,         /* a CUDA call or launch failed */
  MOE_ERR_DEVICE = 5        /* moe_get_device_error found a device-side error bit */
};

/* device error word bits (moe_get_device_error) */
enum {
  MOE_DEVERR_EXPERT_ID = 1,      /* an expert id outside [0, n_experts) reached dispatch */
  MOE_DEVERR_NONFINITE = 2,      /* a router score was NaN (ranked last, never chosen before a finite one) */
  MOE_DEVERR_SCHEDULE = 4,       /* a tile schedule disagreed with the dispatch offsets */
  MOE_DEVERR_TIMEOUT = 8,        /* a kernel's bounded wait expired; that kernel stopped early */
  MOE_DEVERR_RANGE = 16,         /* NVFP4 experts on the FP16 path (under 8 tokens, or above 64): a value
                                    beyond FP16's range (|v| > 65504) reached an FP16 operand (expert
                                    input row or h); the affected outputs are not finite.  The FP4
                                    tensor path (8..64 tokens) carries each row's magnitude in its
                                    FP32 row scale and has no such limit */
  MOE_DEVERR_PAGES = 32,         /* moe_paged_plan ran out of free pages, or a request out of its
                                    block-table row */
  MOE_DEVERR_CACHE = 64          /* a length, parent, page or slot of the paged-attention entry points
                                    was out of range (that entry was clamped or skipped) */
};

typedef int32_t moe_dtype_t;
enum { MOE_DT_F32 = 0, MOE_DT_BF16 = 1, MOE_DT_NVFP4 = 2 };

typedef struct moe_config {
  int32_t d_model;       /* d: hidden width */
  int32_t d_latent;      /* L: latent width the experts act on; 0 = experts act on d */
  int32_t n_experts;     /* E: routed experts, 1..1024 */
  int32_t top_k;         /* K: experts per token, 1..min(E, 32) */
  int32_t n_group;       /* G: equal contiguous expert groups (E % G == 0) */
  int32_t topk_group;    /* TG: groups kept per token, 1..G */
  int32_t d_expert;      /* I: routed expert intermediate width */
  int32_t d_shared;      /* S: shared expert intermediate width; 0 = no shared expert */
  int32_t norm_topk_prob;          /* 1: chosen weights normalised to sum 1 before scaling */
  float routed_scaling_factor;     /* multiplies the (normalised) chosen weights */
  moe_dtype_t act_dtype;           /* MOE_DT_BF16 or MOE_DT_F32 (activations, dense weights) */
  moe_dtype_t expert_dtype;        /* MOE_DT_BF16, MOE_DT_F32 (with F32 activations) or MOE_DT_NVFP4 */
} moe_config_t;

/* Weights of one layer (device pointers, row-major [out, in]).  de = L if L>0 else d.
 * Dense tensors use act_dtype; routed experts use expert_dtype.               */
typedef struct moe_weights {
  const float* w_router;      /* [E, d]  FP32 router matrix                                  */
  const float* router_bias;   /* [E]     FP32 selection bias, or NULL (choice only)          */
  const void* w_lat_down;     /* [L, d]  latent down (latent shapes only)                    */
  const void* w_lat_up;       /* [d, L]  latent up   (latent shapes only)                    */
  const void* w_up;           /* [E, I, de] expert up   (BF16/F32) or NVFP4 packed [E, I, de/2] u8   */
  const void* w_down;         /* [E, de, I] expert down (BF16/F32) or NVFP4 packed [E, de, I/2] u8   */
  const uint8_t* w_up_sf;     /* NVFP4: E4M3 block scales [E, I, de/16], one per 16 K-elements       */
  const uint8_t* w_down_sf;   /* NVFP4: E4M3 block scales [E, de, I/16]                              */
  const float* w_up_gs;       /* NVFP4: FP32 per-tensor scale [E]                                    */
  const float* w_down_gs;     /* NVFP4: FP32 per-tensor scale [E]                                    */
  const void* w_sh_up;        /* [S, d] shared expert up   (S > 0)                                    */
  const void* w_sh_down;      /* [d, S] shared expert down (S > 0)                                    */
  /* optional: the expert down weights again, in the group-major layout of
   * moe_sparse_down_layout (NULL = not given).  When given, decode steps of
   * up to 16 tokens (BF16 experts; NVFP4 experts on their FP16 path)
   * compute the down projection by the ReLU^2-sparse kernel, which reads
   * only the 16-neuron groups of W_down with a live neuron.                 */
  const void* w_down_g;       /* BF16 [E, de * I] / NVFP4 values [E, de * I / 2] u8                   */
  const uint8_t* w_down_g_sf; /* NVFP4: E4M3 scales [E, de * I / 16]                                  */
} moe_weights_t;

/* Library version, e.g. 100 for 0.1.0.  Never fails. */
int32_t moe_version(void);

/* Short static description of a status code.  Never fails. */
const char* moe_status_string(moe_status_t s);

/* Validates a configuration without touching any pointer. */
moe_status_t moe_check_config(const moe_config_t* cfg);

/* Bytes of device workspace moe_layer_forward needs for T tokens (0 on an
 * invalid configuration).  The same workspace serves every step entry point;
 * its first 256 bytes hold the device error word and the expert schedule that
 * moe_dispatch leaves for moe_experts_up / moe_experts_down_combine.  The
 * error word is sticky: clear it once on a new workspace (zero the first 256
 * bytes, or moe_clear_device_error) before reading it. */
size_t moe_workspace_bytes(const moe_config_t* cfg, int32_t T);

/* Step 1: router (page "Nemotron Is Not One Circuit", sections "The Router Is
 * A Deterministic Algorithm" and "The C Kernel Contract"; page "NemotronH ...",
 * section "Arithmetic", router bullet).
 *   x        [T, d] act_dtype hidden rows (BF16 values enter FP32 exactly)
 *   logits   [T, E] FP32 out: z = x W_r^T, or NULL (kept in the workspace)
 *   scores   [T, E] FP32 out: s = sigmoid(z), or NULL
 *   topk_ids [T, K] int32 out: chosen experts, best biased score first,
 *            equal scores to the lower id
 *   topk_w   [T, K] FP32 out: s of the chosen experts, normalised (if
 *            configured) then times routed_scaling_factor                   */
moe_status_t moe_router(const moe_config_t* cfg, int32_t T, const void* x,
                        const float* w_router, const float* router_bias,
                        float* logits, float* scores, int32_t* topk_ids, float* topk_w,
                        void* ws, size_t ws_bytes, void* stream);

/* Step 2: dispatch (page "M6.1 ...", sections 0x05A "The Route Row Is The
 * Reversible Unit" and 0x05B).  Routes r = (token t, slot k) are laid out
 * expert-contiguously, sorted by (expert, token, slot); no atomics.
 *   topk_ids       [T, K] int32 in
 *   x_e            [T, de] act_dtype rows to pack (x, or the latent rows), or NULL
 *   counts         [E] int32 out: routes per expert
 *   offsets        [E+1] int32 out: exclusive prefix sum of counts
 *   route_token    [T*K] int32 out: token of each packed row
 *   route_slot     [T*K] int32 out: slot of each packed row
 *   token_slot_row [T, K] int32 out: packed row of route (t, k)
 *   x_packed       [T*K, de] out: x_packed[j] = x_e[route_token[j]], or NULL
 * Also leaves the expert schedule in the workspace header.                   */
moe_status_t moe_dispatch(const moe_config_t* cfg, int32_t T, const int32_t* topk_ids,
                          const void* x_e, int32_t* counts, int32_t* offsets,
                          int32_t* route_token, int32_t* route_slot, int32_t* token_slot_row,
                          void* x_packed, void* ws, size_t ws_bytes, void* stream);

/* Step 3: expert up projections with squared ReLU, no gate (page "NemotronH
 * ...", section "Arithmetic": bf16(relu(bf16(up x))^2)).
 *   x_e         [T, de] rows the experts read (gathered through route_token),
 *               ignored when x_packed is given
 *   x_packed    [T*K, de] packed rows from moe_dispatch, or NULL (above 64
 *               BF16 tokens, where the tensor-core kernel reads contiguous
 *               rows, x_e is then first gathered into the workspace)
 *   route_token, offsets: from moe_dispatch (same workspace)
 *   h           [T*K, I] out, packed order; BF16 (F32 for F32 layers)        */
moe_status_t moe_experts_up(const moe_config_t* cfg, int32_t T, const void* x_e,
                            const void* x_packed, const int32_t* route_token,
                            const int32_t* offsets, const moe_weights_t* w, void* h,
                            void* ws, size_t ws_bytes, void* stream);

/* Steps 4+5: expert down projections, times the routing weight, and the
 * combine: y_routed[t] = sum over t's routes in ascending expert id of
 * w_tk * (h_r W_down,e^T), all FP32 (page "NemotronH ...", section
 * "Arithmetic"; page "M6.1 ...", section 0x05B, weighted scatter-add).
 *   h              [T*K, I] from moe_experts_up
 *   route_token, route_slot, token_slot_row, offsets: from moe_dispatch
 *   topk_w         [T, K] FP32 from moe_router
 *   y_routed       [T, de] FP32 out                                         */
moe_status_t moe_experts_down_combine(const moe_config_t* cfg, int32_t T, const void* h,
                                      const int32_t* offsets, const int32_t* route_token,
                                      const int32_t* route_slot, const int32_t* token_slot_row,
                                      const float* topk_w, const moe_weights_t* w,
                                      float* y_routed, void* ws, size_t ws_bytes, void* stream);

/* Step 4 alone: the expert down projections times the routing weights, one
 * FP32 row per route in packed order, without the combine (page "NemotronH
 * ...", section "Arithmetic": the down projection accumulates in FP32; page
 * "M6.1 ...", section 0x05B, the gate-weighted routed rows).
 *   h, offsets, route_token, route_slot, topk_w: as for moe_experts_down_combine
 *   u   [T*K, de] FP32 out: u[r] = topk_w[t, k] * (h_r W_down,e^T) for packed
 *       row r of route (t, k) to expert e                                    */
moe_status_t moe_experts_down(const moe_config_t* cfg, int32_t T, const void* h, const int32_t* offsets,
                              const int32_t* route_token, const int32_t* route_slot, const float* topk_w,
                              const moe_weights_t* w, float* u, void* ws, size_t ws_bytes, void* stream);

/* Latent down projection of latent shapes: x_l = bf16(x W_ld^T), FP32
 * accumulation (page "Nemotron-3.5-Super 120B on an 8 GB GPU", section "The
 * only number that matters": experts work in a 1024-wide latent space).
 *   x [T, d] in, x_l [T, L] out (act_dtype).                                  */
moe_status_t moe_latent_down(const moe_config_t* cfg, int32_t T, const void* x,
                             const moe_weights_t* w, void* x_l,
                             void* ws, size_t ws_bytes, void* stream);

/* Shared expert and output (page "Nemotron Is Not One Circuit", section "The
 * Four Layer Kinds CKE Must Preserve": routed experts + shared expert).
 *   x        [T, d] hidden rows
 *   y_routed [T, de] FP32 combined routed output, or NULL (treated as zero)
 *   y        [T, d] act_dtype out: bf16(y_routed + y_s), or for latent shapes
 *            bf16(bf16(y_routed) W_lu^T + y_s); y_s = 0 when S == 0        */
moe_status_t moe_shared(const moe_config_t* cfg, int32_t T, const void* x,
                        const moe_weights_t* w, const float* y_routed, void* y,
                        void* ws, size_t ws_bytes, void* stream);

/* The whole layer, every step above on `stream`, intermediates in `ws`.
 *   x [T, d] in; y [T, d] out (act_dtype).
 *   topk_ids_out [T,K] / topk_w_out [T,K] / logits_out [T,E] / scores_out [T,E]:
 *   optional copies of the router's results (NULL = not written).
 * Clears the device error word first.  NVFP4 experts: see
 * moe_set_nvfp4_act_terms for how the activations enter their products.     */
moe_status_t moe_layer_forward(const moe_config_t* cfg, int32_t T, const void* x,
                               const moe_weights_t* w, void* y,
                               int32_t* topk_ids_out, float* topk_w_out,
                               float* logits_out, float* scores_out,
                               void* ws, size_t ws_bytes, void* stream);

/* ReLU^2-sparse down projection for decode (page "Nemotron-3.5-Super 120B on
 * an 8 GB GPU", section "The engine, step by step", item 4 "Skip the zeros",
 * and section "What didn't work": 16-neuron groups, not single neurons).
 * The down weights are re-laid once, a pure permutation of their values (and,
 * NVFP4, of their bytes and scales), so that each group of 16 neurons
 * 16g .. 16g+15 of an expert holds all de outputs' weights for those neurons
 * contiguously.  Within a group, 16-output tile o is one 512-byte block
 * (BF16) in which lane l = 4r + t (r = l / 4, t = l % 4) holds 16 bytes:
 * W[16o + r][16g + 4t .. +3] then W[16o + r + 8][16g + 4t .. +3].  NVFP4:
 * 64-output quad q of a group is one 512-byte value block, lane l holding
 * for tiles j = 0..3 of the quad the 2 bytes of W[64q + 16j + r][16g + 4t ..
 * +3] then the 2 bytes of row + 8 (low nibble = even neuron, as in w_down),
 * and one 64-byte scale block, bytes 8r + 2j and 8r + 2j + 1 holding the
 * group's E4M3 scales of rows 64q + 16j + r and 64q + 16j + r + 8.
 * A decode step that is given w_down_g finds, per expert, the groups with a
 * nonzero h value in any of the expert's rows and reads only those groups'
 * weights; dead groups only contribute zeros, so the result is that of the
 * dense product up to the order of its FP32 sum.  Needs BF16 activations,
 * I % 16 == 0, I / 16 <= 1024 and de % 32 == 0 (BF16) or de % 64 == 0
 * (NVFP4); else MOE_ERR_UNSUPPORTED.
 * moe_sparse_down_bytes: sizes of w_down_g (*values) and w_down_g_sf
 * (*scales, 0 for BF16).  moe_sparse_down_layout: writes both from w->w_down
 * (and w->w_down_sf) on `stream` (caller-owned, 16-byte aligned buffers).  */
moe_status_t moe_sparse_down_bytes(const moe_config_t* cfg, size_t* values, size_t* scales);
moe_status_t moe_sparse_down_layout(const moe_config_t* cfg, const moe_weights_t* w, void* w_down_g,
                                    uint8_t* w_down_g_sf, void* stream);

/* The MoE block of a decoder layer: RMSNorm, the layer, the residual add
 * (page "Nemotron Is Not One Circuit: Mamba, Attention, and MoE Routing",
 * section "The Four Layer Kinds CKE Must Preserve": an MoE layer is RMSNorm,
 * router, group-limited top-k, routed ReLU^2 experts + shared expert,
 * residual).  Chains of blocks need no host work between them, so several
 * can be captured in one CUDA graph (page "NemotronH (Nemotron 3.5 Lightning,
 * Bolt, Super VL)", section "Speculation": verify blocks of 1-16 rows).
 *   x        [T, d] act_dtype residual stream in
 *   norm_w   [d] FP32 RMSNorm weight gamma;  norm_eps >= 0
 *   out      [T, d] act_dtype: out = act(x + layer(xn)), the layer's FP32
 *            output and the residual added before the one rounding.  out may
 *            be x itself (in place); any other overlap with x is rejected.
 *   xn = act(gamma * (x * r)), r = 1 / sqrt(mean(x^2) + eps) per row, all in
 *            FP32 with one rounding: the rows the router, the latent down
 *            projection, the shared expert and (without a latent) the experts
 *            read.  x_norm_out [T, d]: an optional copy (NULL: kept in the
 *            workspace, MOE_WS_X_NORM); it must not overlap x or out.
 *   topk_ids_out / topk_w_out / logits_out / scores_out: as moe_layer_forward.
 * The RMSNorm kernel also clears the workspace header (no separate memset). */
moe_status_t moe_block_forward(const moe_config_t* cfg, int32_t T, const void* x,
                               const float* norm_w, float norm_eps,
                               const moe_weights_t* w, void* out, void* x_norm_out,
                               int32_t* topk_ids_out, float* topk_w_out,
                               float* logits_out, float* scores_out,
                               void* ws, size_t ws_bytes, void* stream);

/* ---- backward (page "M6.1 Routed Capacity", section 0x06F "Single-Device
 * Forward And Backward Integration Contract") ------------------------------
 * Gradients of a scalar loss L with upstream gradient dy = dL/dy, for the
 * forward relation the forward call froze: the chosen ids are metadata (no
 * gradient; the selection bias only chooses), the gates w = rsf s_k / sum_j s_j
 * (or rsf s_k) carry the router's gradient to the chosen experts' logits
 * (dL/dz_k = dL/ds_k s_k (1 - s_k), zero for every other expert), the
 * combine's backward is dU = w dy_r and dL/dw = <dy_r, U>, the gather's
 * adjoint a scatter-add in ascending expert order, and the router, expert,
 * shared and (block) residual paths add at the input.  BF16 layers only
 * (MOE_ERR_UNSUPPORTED otherwise); BF16 operands, FP32 accumulation; the
 * ReLU^2 derivative 2 relu(a) is taken as 2 sqrt(h) from the forward's stored
 * h.  Weight gradients are ADDED to the given FP32 buffers (zero them once
 * per step; a NULL buffer skips that gradient); experts without routes are
 * left untouched (their gradient is zero).                                  */
typedef struct moe_grads {
  float* d_router;    /* [E, d]      */
  float* d_lat_down;  /* [L, d]      latent shapes */
  float* d_lat_up;    /* [d, L]      latent shapes */
  float* d_up;        /* [E, I, de]  */
  float* d_down;      /* [E, de, I]  */
  float* d_sh_up;     /* [S, d]      shared expert */
  float* d_sh_down;   /* [d, S]      shared expert */
  float* d_norm_w;    /* [d]         moe_block_backward only */
} moe_grads_t;

/* Bytes of the backward scratch `bws` for T tokens (0 on an invalid config). */
size_t moe_backward_workspace_bytes(const moe_config_t* cfg, int32_t T);

/* Where the backward scratch keeps its BF16 operands and the gate gradient
 * after a backward call (host arithmetic only), so a caller can inspect them:
 *   MOE_BWS_DU         [T*K, de] bf16  dU = bf16(w dy_r), packed row order
 *   MOE_BWS_DA         [T*K, I]  bf16  da = bf16((dU W_down) * 2 sqrt(h))
 *   MOE_BWS_DZ         [T, K]    FP32  dL/dz of the chosen experts' logits
 *   MOE_BWS_DX_LATENT  [T, L]    bf16  the latent input gradient (latent shapes)
 *   MOE_BWS_DA_SHARED  [T, S]    bf16  the shared expert's da
 *   MOE_BWS_DY_LATENT  [T, L]    bf16  dy_r = bf16(dy W_lu) (latent shapes)  */
enum {
  MOE_BWS_DU = 0, MOE_BWS_DA = 1, MOE_BWS_DZ = 2, MOE_BWS_DX_LATENT = 3, MOE_BWS_DA_SHARED = 4,
  MOE_BWS_DY_LATENT = 5
};
moe_status_t moe_backward_workspace_region(const moe_config_t* cfg, int32_t T, int32_t region,
                                           size_t* offset, size_t* bytes);

/* Backward of moe_layer_forward.  `ws` must be the workspace of a
 * moe_layer_forward call on the same x, weights and T, with no other call on
 * it since (its route tables, h, u, latent rows and shared h are the saved
 * forward state).  topk_ids / topk_w / scores: the forward's router outputs
 * ([T, K] int32, [T, K] FP32, [T, E] FP32; its *_out buffers, or the
 * workspace regions MOE_WS_TOPK_IDS / _TOPK_W / _SCORES when they were NULL).
 *   x [T, d] the forward's input; dy [T, d] act_dtype upstream gradient;
 *   dx [T, d] FP32 out: dL/dx through the router, the experts (and latent
 *   pair) and the shared expert.                                           */
moe_status_t moe_layer_backward(const moe_config_t* cfg, int32_t T, const void* x,
                                const moe_weights_t* w, const void* dy,
                                const int32_t* topk_ids, const float* topk_w, const float* scores,
                                float* dx, const moe_grads_t* grads,
                                const void* ws, size_t ws_bytes, void* bws, size_t bws_bytes,
                                void* stream);

/* Backward of moe_block_forward (out = x + layer(RMSNorm(x))): dout [T, d]
 * act_dtype; dx [T, d] FP32 = dout (the residual) + the RMSNorm's backward of
 * the layer's input gradient; grads->d_norm_w gets dL/dgamma added.  x_norm:
 * the forward's x_norm_out buffer, or NULL when the forward kept the rows in
 * the workspace.  Same state rules as moe_layer_backward.                   */
moe_status_t moe_block_backward(const moe_config_t* cfg, int32_t T, const void* x,
                                const float* norm_w, float norm_eps, const void* x_norm,
                                const moe_weights_t* w, const void* dout,
                                const int32_t* topk_ids, const float* topk_w, const float* scores,
                                float* dx, const moe_grads_t* grads,
                                const void* ws, size_t ws_bytes, void* bws, size_t bws_bytes,
                                void* stream);

/* ---- paged attention for verify blocks ------------------------------------
 * The attention of a decoder layer over a paged KV cache, for single tokens,
 * chains and trees of drafted tokens (page "Nemotron Is Not One Circuit:
 * Mamba, Attention, and MoE Routing", section "The Four Layer Kinds CKE Must
 * Preserve": the attention layer beside the MoE layer; page "NemotronH
 * (Nemotron 3.5 Lightning, Bolt, Super VL)", section "Speculation": verify
 * blocks of several drafted rows).  Three operators: moe_paged_plan builds the
 * step's block tables and slot maps, moe_rope_append turns the rows by their
 * positions and writes K and V into the cache, moe_tree_attention reads it.
 *
 * A step has R requests.  Request r holds ctx_len[r] tokens in the cache and
 * brings n_r = new_len[r] >= 0 new ones, its nodes; the nodes of all requests
 * are packed, request after request, as T = sum n_r rows, those of request r at
 * q_start[r] .. q_start[r+1] - 1.  Node i of request r lies in the cache at
 * token ctx_len[r] + i, and token p of request r at offset p % page_size of
 * page block_table[r][p / page_size].  kv_len[r] = ctx_len[r] + n_r.
 *
 * Conventions beyond those above: integer arrays need their type's alignment
 * only; rows and caches 16 bytes.  Row strides (q_ld, ...) are in elements, a
 * multiple of 16 bytes, the heads of a row head_dim apart, so that q, k and v
 * may be parts of one projection's rows.  `ws` is a workspace of
 * moe_attn_workspace_bytes: zero its first MOE_ATTN_HEADER_BYTES once; calls
 * that may overlap on the GPU need a workspace each.  Its error word is sticky:
 * these entry points set bits and never clear it (moe_get_device_error,
 * moe_clear_device_error).                                                   */
#define MOE_ATTN_HEADER_BYTES 4096

typedef struct moe_attn_config {
  int32_t n_heads;           /* H: query heads, a multiple of n_kv_heads            */
  int32_t n_kv_heads;        /* Hkv; H / Hkv <= 128 query heads share a KV head      */
  int32_t head_dim;          /* D: 8..128, a multiple of 8                           */
  int32_t page_size;         /* tokens a page: a power of two, 8..1024               */
  int32_t n_pages;           /* pages of the cache                                   */
  int32_t max_pages;         /* entries of a block-table row                         */
  int32_t rot_dim;           /* leading dims of a head that rotate: even, 0..D       */
  int32_t rope_interleaved;  /* pairs (2i, 2i+1); 0: (i, i + rot_dim/2)              */
  float softmax_scale;       /* multiplies q.k; > 0                                  */
  moe_dtype_t dtype;         /* MOE_DT_BF16 or MOE_DT_F32: rows and caches           */
  /* where K and V of token offset o, head h of page p start in k_cache and in
   * v_cache, in elements: p * page_stride + o * token_stride + h * head_stride
   * (so both [page][token][head][D] and [page][head][token][D] caches fit)     */
  int64_t page_stride, token_stride, head_stride;
} moe_attn_config_t;

/* Validates a configuration without touching any pointer. */
moe_status_t moe_check_attn_config(const moe_attn_config_t* cfg);

/* Bytes of the workspace of the entry points below (0 on an invalid
 * configuration): one size, whatever the lengths and the batch.              */
size_t moe_attn_workspace_bytes(const moe_attn_config_t* cfg);

/* Block tables, slot maps, positions and tree masks of a step from its
 * lengths, on the device.  With held(c) = ceil(c / page_size), request r needs
 * held(ctx + n) - held(ctx) more pages.  Requests take them in ascending r from
 * free_pages[*free_head], free_pages[*free_head + 1], ...
 *   R          requests, 0..16384;  T: rows of the outputs, T >= sum n_r
 *   ctx_len, new_len [R] int32
 *   parents    [T] int32 or NULL: the node a node hangs from, an earlier one of
 *              its request, or -1 (a root).  NULL: chains
 *   block_table [R, max_pages] int32: entries held(ctx) .. held(ctx + n) - 1 are
 *              written, the others kept
 *   free_pages [n_free] int32 page ids;  free_head [1] int32: entries already used
 *   free_head_out [1] int32 out: *free_head + pages taken; may be free_head
 *   q_start    [R+1] int32 out: exclusive prefix sum of new_len
 *   kv_len     [R] int32 out: ctx_len + new_len
 *   positions  [T] int32 out: ctx_len + depth of the node (chain: + its index)
 *   slot_map   [T] int64 out: page * page_size + offset, or -1
 *   tree_mask  [T, mask_words] int32 out (with parents), bit j % 32 of word
 *              j / 32: node j is the row's node or one of its ancestors
 * Pages come back by writing them before free_pages[*free_head] and lowering
 * *free_head (a finished request's, or those of a draft's rejected end).
 * Rows past the last node get position 0, slot -1 and an empty mask, so that a
 * captured graph may run at a fixed T.  Out of free pages (or of the table's
 * row): MOE_DEVERR_PAGES, entries and slots -1.  Bad lengths, parents and page
 * ids: MOE_DEVERR_CACHE; a negative length counts as 0, a bad parent as -1,
 * nodes past T or past 32 * mask_words are dropped from the rows or the mask. */
moe_status_t moe_paged_plan(const moe_attn_config_t* cfg, int32_t R, int32_t T, const int32_t* ctx_len,
                            const int32_t* new_len, const int32_t* parents, int32_t* block_table,
                            const int32_t* free_pages, int32_t n_free, const int32_t* free_head,
                            int32_t* free_head_out, int32_t* q_start, int32_t* kv_len, int32_t* positions,
                            int64_t* slot_map, int32_t* tree_mask, int32_t mask_words, void* ws, size_t ws_bytes,
                            void* stream);

/* Rotary frequencies as turns: entry i < rot_dim / 2 of the HOST table is
 * f_i / (2 pi) * 2^64, made in FP64 (relative error 2^-51 at most), with
 * f_i = theta^(-2i / rot_dim) radians a position.  position * entry mod 2^64 is
 * the angle's fraction of a turn without further rounding, however far the
 * position: the angle is off by at most 2^-51 position f_i radians from the table
 * and, in the kernels, by 2^-33 turns and an FP32 rounding.  Host arithmetic only;
 * the caller copies the table to the device once.
 *   scaling  MOE_ROPE_PLAIN; MOE_ROPE_LINEAR: f_i / factor; MOE_ROPE_YARN: the
 *            method of "YaRN: Efficient Context Window Extension of Large
 *            Language Models" (Peng et al., 2023): f_i / factor where a pair
 *            turns fewer than 1 time over original_context tokens, f_i where it
 *            turns more than 32 times, a ramp between, and *rot_scale =
 *            0.1 ln(factor) + 1 (otherwise 1).  The ramp is linear in the pair's
 *            index i, from low = max(floor(i32), 0) to high = min(ceil(i1),
 *            rot_dim - 1) (at least 0.001 apart), where i32 and i1 are the indexes
 *            at which a pair turns 32 times and once, as models are trained with */
enum { MOE_ROPE_PLAIN = 0, MOE_ROPE_LINEAR = 1, MOE_ROPE_YARN = 2 };
moe_status_t moe_rope_table(int32_t rot_dim, double theta, int32_t scaling, double factor,
                            int64_t original_context, uint64_t* table_host, float* rot_scale);

/* Rotary positions of T rows of `heads` heads: each pair (a, b) of the first
 * rot_dim dims becomes rot_scale * (a cos - b sin, a sin + b cos), the other dims
 * are copied.  inverse: the transposed map, which is its backward (the gradient
 * of the input from the gradient of the output).  FP32, rounded once.
 *   x, out [T, heads, D] with row strides; out may be x (same
 *   stride), and overlap it in no other way;  positions [T] int32 >= 0
 *   table  [rot_dim / 2] of moe_rope_table, on the device (NULL if rot_dim is 0) */
moe_status_t moe_rope(const moe_attn_config_t* cfg, int32_t T, int32_t heads, const void* x, int64_t x_ld,
                      const int32_t* positions, const uint64_t* table, float rot_scale, int32_t inverse, void* out,
                      int64_t out_ld, void* stream);

/* The rows of a step on their way into the attention: q rotated to q_out, k
 * rotated into k_cache and v copied into v_cache at slot_map (one pass; rows
 * with slot -1 are not cached, a slot outside the cache is skipped with
 * MOE_DEVERR_CACHE).
 *   q [T, H, D], k and v [T, Hkv, D] with row strides;  q_out [T, H, D], may be q */
moe_status_t moe_rope_append(const moe_attn_config_t* cfg, int32_t T, const void* q, int64_t q_ld, const void* k,
                             int64_t k_ld, const void* v, int64_t v_ld, const int32_t* positions,
                             const uint64_t* table, float rot_scale, const int64_t* slot_map, void* q_out,
                             int64_t q_out_ld, void* k_cache, void* v_cache, void* ws, size_t ws_bytes, void* stream);

/* Attention of the step's rows over the cache.  Row i (node i - q_start[r] of
 * request r) sees the tokens before its request's nodes, kv_len[r] - n_r of
 * them, and the nodes that its mask row names; without a mask the nodes up to
 * itself (a chain).  Head h reads KV head h / (H / Hkv).
 *   out = sum_k softmax_k(softmax_scale q.k) v_k over the keys the row sees
 *   R          requests, 0..4096;  T rows of q, T >= q_start[R]
 *   q, out     [T, H, D] with row strides (out must not overlap q)
 *   q_start [R+1], kv_len [R], block_table [R, max_pages] int32: moe_paged_plan's
 *   tree_mask  [T, mask_words] int32 or NULL
 *   lse        [T, H] FP32 out or NULL: the natural log of the sum of exponentials
 * A row that sees no key, and a row that belongs to no request, gets zeros and
 * lse = -inf.  Keys that no row sees (stale or unwritten cache memory) do not
 * enter, whatever they hold, NaN and infinities included; nor do a node's K and
 * V enter the rows that do not see that node.  FP32 scores and softmax; BF16:
 * the probabilities enter the second product in BF16.  Where kv_len ends past the
 * block table's row, the tokens past it (nodes among them) are seen by no row and
 * the others stay where they are; a kv_len below the number of nodes counts as
 * that number; pages outside the cache read as zeros; all with
 * MOE_DEVERR_CACHE.  (T + R) * Hkv * (ceil(max_pages * page_size / 128) + 5) and
 * 32 * T * H must stay below 2^31 (MOE_ERR_UNSUPPORTED).  FP32 runs on the CUDA
 * cores and is made for the sizes of FP32 layers.                             */
moe_status_t moe_tree_attention(const moe_attn_config_t* cfg, int32_t R, int32_t T, const void* q, int64_t q_ld,
                                const int32_t* q_start, const int32_t* kv_len, const int32_t* block_table,
                                const void* k_cache, const void* v_cache, const int32_t* tree_mask,
                                int32_t mask_words, void* out, int64_t out_ld, float* lse, void* ws, size_t ws_bytes,
                                void* stream);

/* ---- requests that share pages ---------------------------------------------
 * Several requests may hold one page in their rows of the block table (samples
 * of one prompt, a system prompt, beams).  page_shares[p] counts the holders of
 * page p beyond its first: 0 for a page that one request holds and for a free one,
 * so that moe_paged_plan, whose pages have one holder, need not know of it.  Only
 * whole pages are shared; what a request writes next lies in a page of its own.
 * That is the caller's to keep: cut a request (release) inside a page that others
 * hold, and its next tokens would be theirs; fork it onto another row instead.   */

/* Continues requests by others: fork i makes row dst_rows[i] of dst_table hold the
 * first lengths[i] tokens of row src_rows[i] of src_table.  Its whole pages are
 * shared (page_shares + 1 each, any number of forks of one row); the tokens of a
 * partly filled last one are copied, K and V, into a page taken from the list of
 * free ones, the forks' pages in ascending i.
 *   n          forks, 0..4096;  src_rows, dst_rows, lengths [n] int32
 *   src_table, dst_table [R, max_pages] int32, R 0..16384: one table, or two that
 *              do not overlap (beams: the new step's rows from the old ones)
 *   page_shares [n_pages] int32, in and out
 *   free_pages [n_free], free_head, free_head_out: as in moe_paged_plan
 * Written: entries 0 .. ceil(lengths[i] / page_size) - 1 of row dst_rows[i] (pages that
 * it held before are not given back), the counts, the copied tokens.  A row is
 * the destination of one fork and, within one table, no source: of forks that meet
 * in a destination the first is done, one whose source is another's destination, or
 * whose row or length is out of range, is not, with MOE_DEVERR_CACHE.  Such a fork
 * still takes its page if its rows and length are in range.  Page ids outside the cache
 * become -1 entries (MOE_DEVERR_CACHE); out of free pages: entry -1, MOE_DEVERR_PAGES.
 * 2 * n_kv_heads * head_dim * page_size elements in pieces of 16 bytes must be below
 * 2^31 (MOE_ERR_UNSUPPORTED).
 * Layers that share a table, its counts and its list: one call as above, with another
 * free_head_out than free_head; then, for each other layer, the same call with its
 * caches, src_table the table, and a dst_table, page_shares and free_head_out that
 * nobody reads (memory of their own): it takes the same pages, and copies its tokens
 * there.  (A fork of a row onto itself would take a page in these calls.)            */
moe_status_t moe_paged_fork(const moe_attn_config_t* cfg, int32_t n, const int32_t* src_rows, const int32_t* dst_rows,
                            const int32_t* lengths, int32_t R, const int32_t* src_table, int32_t* dst_table,
                            int32_t* page_shares, const int32_t* free_pages, int32_t n_free, const int32_t* free_head,
                            int32_t* free_head_out, void* k_cache, void* v_cache, void* ws, size_t ws_bytes,
                            void* stream);

/* Moves the kept tokens of each request to the front, K and V, in place: of the
 * tokens from first[r] on (the nodes of a step, say), number keep[keep_start[r] + i]
 * goes to token first[r] + i.  The accepted path of a drafted tree (its nodes
 * ascend), or what an eviction leaves of a context (first 0).
 *   R          requests, 0..16384;  N: entries of keep
 *   first [R], keep_start [R+1], keep [N] int32: ascending numbers, from 0, a request
 *   page_shares [n_pages] int32 or NULL: where given, a shared page is not written to
 *   len_out    [R] int32 out or NULL: first + number of kept tokens; not the memory of
 *              first, keep_start or keep (MOE_ERR_INVALID_ARG)
 * Kept numbers that do not ascend, tokens past the table's row, pages outside the
 * cache and shared pages that would be written: the token is not moved, with
 * MOE_DEVERR_CACHE (so is a request whose keep_start or first is out of range left
 * as it is, with len_out = max(first, 0)).  The pages stay the request's; the ones behind the
 * kept tokens go back with moe_paged_release.  For long lists the blocks of a
 * cooperative launch wait for one another, 4 seconds at most: then MOE_DEVERR_TIMEOUT, and
 * some tokens are not moved.                                                      */
moe_status_t moe_paged_compact(const moe_attn_config_t* cfg, int32_t R, int32_t N, const int32_t* first,
                               const int32_t* keep_start, const int32_t* keep, const int32_t* block_table,
                               const int32_t* page_shares, int32_t* len_out, void* k_cache, void* v_cache, void* ws,
                               size_t ws_bytes, void* stream);

/* Gives pages back: those that request r holds for its first held_len[r] tokens but
 * not for its first keep_len[r] (a rejected part of a draft; 0: a finished request).
 * A page that others hold loses a holder; one that is left without any goes back to
 * the list, before free_pages[*free_head], in the table's order (where several
 * rows give one up in this call, at the last of them).
 *   R          requests, 0..16384, R * max_pages < 2^31
 *   held_len, keep_len [R] int32;  block_table [R, max_pages] int32: entries given
 *              back become -1
 *   page_shares [n_pages] int32, in and out, or NULL: no page is shared
 *   free_pages [n_free] int32, free_head [1] int32, in and out
 * Entries -1 are passed over.  Negative lengths (count as 0), page ids outside the
 * cache, a page given back more often than it is held, and more pages than the list
 * gave out (the first ones are dropped): MOE_DEVERR_CACHE.  Blocks wait for one
 * another as in moe_paged_compact where R * max_pages is above 4096; after
 * MOE_DEVERR_TIMEOUT the list and the table are as they were, the counts need not be.
 * It may overlap with moe_rope_append, moe_tree_attention and moe_prefix_attention of
 * the same workspace and configuration that do not look at what it gives back
 * (requests that ended before their step, on another stream).                        */
moe_status_t moe_paged_release(const moe_attn_config_t* cfg, int32_t R, const int32_t* held_len,
                               const int32_t* keep_len, int32_t* block_table, int32_t* page_shares,
                               int32_t* free_pages, int32_t n_free, int32_t* free_head, void* ws, size_t ws_bytes,
                               void* stream);

/* moe_tree_attention for requests in groups with a common prefix: its pages are
 * attended once for all rows of the group, the requests' other tokens by themselves,
 * and a row's two parts joined (FP32 partial sums, maxima and exponential sums).
 *   n_groups   groups, 0..R (R 0..2048);  group_start [n_groups+1] int32, ascending:
 *              group g is requests group_start[g] .. group_start[g+1] - 1; requests
 *              before the first and behind the last group share nothing
 *   prefix_row [n_groups] int32: the block-table row (any of the R) that the prefix
 *              is read through
 *   prefix_len [n_groups] int32: the common tokens.  Their whole pages are
 *              attended once; a partly filled last one through each request's own row
 *   ws         moe_prefix_workspace_bytes(cfg, T)
 * The others as in moe_tree_attention; a request's tokens are counted from its
 * context's start as there, prefix included.  A request whose context (kv_len
 * without its nodes) is shorter than the prefix's whole pages, and a group of fewer
 * than two requests, are attended through their own rows alone.  Bad groups (bounds
 * or rows out of range, a prefix past the table's row): MOE_DEVERR_CACHE, and they
 * share nothing; where group_start does not ascend, no group of the call does.  (2 T + R + n_groups) * Hkv *
 * (ceil(max_pages * page_size / 128) + 5) and 32 * T * H must stay below 2^31.
 * FP32 reads the prefix through prefix_row for each row by itself.                  */
size_t moe_prefix_workspace_bytes(const moe_attn_config_t* cfg, int32_t T);
moe_status_t moe_prefix_attention(const moe_attn_config_t* cfg, int32_t R, int32_t T, const void* q, int64_t q_ld,
                                  const int32_t* q_start, const int32_t* kv_len, const int32_t* block_table,
                                  int32_t n_groups, const int32_t* group_start, const int32_t* prefix_row,
                                  const int32_t* prefix_len, const void* k_cache, const void* v_cache,
                                  const int32_t* tree_mask, int32_t mask_words, void* out, int64_t out_ld, float* lse,
                                  void* ws, size_t ws_bytes, void* stream);

/* ---- rotary positions with several axes -------------------------------------
 * A token of an image or a video has a position on each of a few axes (time,
 * height, width); every rotating pair turns by the position of one of them, text
 * tokens having the same position on all.  moe_rope_axes_table makes the pairs' axes
 * and frequencies on the HOST: sections[a] pairs belong to axis a (their sum is
 * rot_dim / 2), in one piece after another, or (interleaved) dealt out one
 * at a time to the axes that have pairs left.  One ladder of frequencies,
 * theta^(-2i / rot_dim) for pair i, or (own_ladders) one for each axis,
 * theta^(-j / sections[a]) for its j-th pair; scaling as in moe_rope_table.
 *   table_host [rot_dim / 2] uint64, axis_host [rot_dim / 2] uint8 out
 * moe_rope_axes and moe_rope_append_axes are moe_rope and moe_rope_append with
 *   n_axes     1..4;  positions [n_axes, T] int32
 *   axis       [rot_dim / 2] uint8 on the device (NULL if rot_dim is 0); a number
 *              past the last axis counts as the last                                */
#define MOE_ROPE_MAX_AXES 4
moe_status_t moe_rope_axes_table(int32_t n_axes, const int32_t* sections, int32_t interleaved, int32_t own_ladders,
                                 double theta, int32_t scaling, double factor, int64_t original_context,
                                 uint64_t* table_host, uint8_t* axis_host, float* rot_scale);
moe_status_t moe_rope_axes(const moe_attn_config_t* cfg, int32_t T, int32_t heads, const void* x, int64_t x_ld,
                           int32_t n_axes, const int32_t* positions, const uint8_t* axis, const uint64_t* table,
                           float rot_scale, int32_t inverse, void* out, int64_t out_ld, void* stream);
moe_status_t moe_rope_append_axes(const moe_attn_config_t* cfg, int32_t T, const void* q, int64_t q_ld,
                                  const void* k, int64_t k_ld, const void* v, int64_t v_ld, int32_t n_axes,
                                  const int32_t* positions, const uint8_t* axis, const uint64_t* table,
                                  float rot_scale, const int64_t* slot_map, void* q_out, int64_t q_out_ld,
                                  void* k_cache, void* v_cache, void* ws, size_t ws_bytes, void* stream);

/* Synchronises `stream`, copies the device error word of `ws` to *code (host
 * pointer) and returns MOE_ERR_DEVICE if any bit is set, else MOE_OK.         */
moe_status_t moe_get_device_error(const void* ws, void* stream, int32_t* code);

/* Enqueues a clear of the device error word. */
moe_status_t moe_clear_device_error(void* ws, void* stream);

/* How the activations of NVFP4 experts enter their products (process-wide;
 * applies to the calls made after it):
 *   n = -1    the default: three terms on the FP4 tensor path for 8 to 64
 *             tokens, the FP16 path otherwise (the faster one at each size
 *             as measured on GB300)
 *   n = 1..4  the FP4 tensor path: every expert input row and every row of h
 *             is split into n NVFP4 terms, each encoding what the earlier ones
 *             left (E2M1 values, one E4M3 scale per 16 values, one FP32 scale
 *             per row), and the block-scaled FP4 MMA multiplies them with the
 *             NVFP4 weights; n = 1 is plain W4A4.  Each term leaves at most
 *             ~0.18 of the previous residual of a 16-value block, so the
 *             default's n = 3 represents every activation to within ~0.006 of
 *             its block's largest magnitude.  h is stored as BF16.
 *   n = 0     the FP16 path: the weights are decoded to FP16 inside the kernels
 *             and multiplied with FP16 copies of the BF16 activations (exact
 *             for magnitudes up to 65504; a larger activation overflows).
 * Returns the previous setting, or -2 (nothing changed) for n outside -1..4.
 * The block format is the one of page "Nemotron-3.5-Super 120B on an 8 GB
 * GPU", section "The engine, step by step", item 4.                        */
int32_t moe_set_nvfp4_act_terms(int32_t n);

/* The activation terms a call with T tokens uses under the current setting
 * (0: the FP16 path).  Never fails. */
int32_t moe_nvfp4_act_terms_for(int32_t T);

/* Where a workspace for T tokens keeps the layer's route tables, so a caller
 * can read what moe_layer_forward decided (host arithmetic only; no CUDA call).
 * After moe_layer_forward (same cfg, T and workspace) the regions hold:
 *   MOE_WS_COUNTS          [E]     int32  routes per expert
 *   MOE_WS_OFFSETS         [E+1]   int32  exclusive prefix sum of the counts
 *   MOE_WS_ROUTE_TOKEN     [T*K]   int32  token of each packed row
 *   MOE_WS_ROUTE_SLOT      [T*K]   int32  slot of each packed row
 *   MOE_WS_TOKEN_SLOT_ROW  [T, K]  int32  packed row of route (t, k)
 *   MOE_WS_TOPK_IDS        [T, K]  int32  chosen experts   } only when the
 *   MOE_WS_TOPK_W          [T, K]  FP32   routing weights  } matching optional
 *   MOE_WS_LOGITS          [T, E]  FP32   router logits    } output of
 *   MOE_WS_SCORES          [T, E]  FP32   sigmoid scores   } moe_layer_forward is NULL
 *   MOE_WS_X_LATENT        [T, L]  act    latent rows (latent shapes)
 *   MOE_WS_X_PACKED        [T*K, de]      rows packed for the tensor-core path
 *                                         (above 64 BF16 tokens: act_dtype, or
 *                                         FP16 copies of the BF16 values with
 *                                         NVFP4 experts on the FP16 path)
 *   MOE_WS_H               [T*K, I]  act  the experts' ReLU^2 rows h, packed order
 * NVFP4 experts on the FP4 tensor path (moe_set_nvfp4_act_terms n > 0), term
 * j of packed row r of the expert input rows (X) and of h (H):
 *   MOE_WS_X_TERMS / MOE_WS_H_TERMS        [4][T*K][de/2 | I/2] u8  E2M1 codes, even
 *                                           element in the low nibble (terms >= n unused)
 *   MOE_WS_X_TERM_SCALES / _H_TERM_SCALES  [4][T*K][ld] u8  E4M3 scale per 16 values,
 *                                           ld = (K/16 rounded up to 16) for K = de | I
 *   MOE_WS_X_ROW_SCALES / _H_ROW_SCALES    [T*K] FP32  the rows' scale g
 * After moe_block_forward without x_norm_out:
 *   MOE_WS_X_NORM          [T, d]  act    the RMSNorm rows xn
 * *offset receives the region's byte offset from the workspace start, *bytes
 * its size.  MOE_ERR_INVALID_ARG for an unknown region or T < 0.           */
enum {
  MOE_WS_COUNTS = 0, MOE_WS_OFFSETS = 1, MOE_WS_ROUTE_TOKEN = 2, MOE_WS_ROUTE_SLOT = 3,
  MOE_WS_TOKEN_SLOT_ROW = 4, MOE_WS_TOPK_IDS = 5, MOE_WS_TOPK_W = 6, MOE_WS_LOGITS = 7,
  MOE_WS_SCORES = 8, MOE_WS_X_LATENT = 9, MOE_WS_X_PACKED = 10, MOE_WS_H = 11, MOE_WS_X_TERMS = 12,
  MOE_WS_X_TERM_SCALES = 13, MOE_WS_X_ROW_SCALES = 14, MOE_WS_H_TERMS = 15, MOE_WS_H_TERM_SCALES = 16,
  MOE_WS_H_ROW_SCALES = 17, MOE_WS_X_NORM = 18
};
moe_status_t moe_workspace_region(const moe_config_t* cfg, int32_t T, int32_t region, size_t* offset,
                                  size_t* bytes);

/* Number of kernel launches this library has enqueued in this process (a host
 * counter, incremented once per kernel launch; memset and copy operations are
 * not counted).  Never fails. */
int64_t moe_launch_count(void);

/* Router step that allocates nothing and takes no workspace.  The pages have
 * no counterpart: this serves callers that cannot allocate device memory at
 * call time, such as code running after a host framework's memory pool has
 * claimed the device, serving loops that forbid allocation once started, or
 * work enqueued where cudaMalloc is not permitted.  Same arguments and
 * results as moe_router without logits/scores outputs (the same kernels,
 * bit-identical results); its scratch (logits, scores, the BF16 split of the
 * router matrix and the four K-split logit slabs used above 64 BF16 tokens,
 * and the error word) lives in a static device array of
 * MOE_NOALLOC_MAX_ROUTER_ELEMS * 24 + MOE_NOALLOC_MAX_SPLIT_ELEMS * 2 + 256
 * bytes (about 17 MiB) that every GPU loading this library keeps until exit.
 *   - Returns MOE_ERR_WORKSPACE, before enqueuing anything, when
 *     T * n_experts > MOE_NOALLOC_MAX_ROUTER_ELEMS, or when T > 64 BF16
 *     tokens need the split router matrix and 3 * n_experts * d_model >
 *     MOE_NOALLOC_MAX_SPLIT_ELEMS.
 *   - The first call on a device looks the array up (cudaGetSymbolAddress,
 *     once per device, with that device current) and keeps the address for
 *     the life of the process: it assumes the device's primary context is
 *     never reset (cudaDeviceReset) while the library is loaded.
 *   - All calls share the array: calls whose work overlaps on the GPU race.
 *     Each call clears the error word first; device error bits are not
 *     reported by this entry point.
 *   - Calls no allocation routine (no cudaMalloc/cudaFree).                  */
#define MOE_NOALLOC_MAX_ROUTER_ELEMS 131072
#define MOE_NOALLOC_MAX_SPLIT_ELEMS 7340032
moe_status_t moe_router_noalloc(const moe_config_t* cfg, int32_t T, const void* x,
                                const float* w_router, const float* router_bias,
                                int32_t* topk_ids, float* topk_w, void* stream);

/* End-to-end convenience call with HOST buffers: copies x_host [T, d] to
 * x_dev, runs moe_layer_forward, copies y to y_host and synchronises the
 * stream.  x_dev / y_dev / ws are caller-owned device buffers; the host
 * buffers should be pinned for asynchronous copies.                          */
moe_status_t moe_layer_forward_host(const moe_config_t* cfg, int32_t T, const void* x_host,
                                    void* x_dev, const moe_weights_t* w, void* y_dev,
                                    void* y_host, void* ws, size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* MOE_GB300_H */
