/*
 * weight_patches.h -- C ABI of the GB300 (sm_103a) dynamic-LoRA linear library.
 *
 * Computes the dynamic, unmerged LoRA linear
 *
 *     Y = X W^T + bias + sum_p s_p (X A_p^T) B_p^T,
 *     s_p = alpha_p / rank_p * strength_p * request_scale,
 *
 * and its siblings (stacked column groups, closed-form backward, dense patches) on
 * one GPU.  Sources of the operations, cited by page title and section:
 *   - sglang PR "[diffusion] Add the dynamic LoRA delta inside the second GEMM",
 *     Motivation and Modifications: the combined scale multiplies the rank-wide
 *     intermediate X A^T as a runtime value, the second low-rank GEMM accumulates
 *     straight onto the base output so the [tokens, out] delta is never stored, the
 *     bias lives in the base GEMM's epilogue, stacked q/k/v (gate/up) adapters take
 *     one update per column group, an FP32 adapter keeps FP32 GEMMs and adds once;
 *   - InvokeAI sidecar-patch article, sections 三-四: several patches on one layer are
 *     summed, each weighted by its own strength;
 *   - Unsloth fast_lora walkthrough, sections 2-4: 4-bit base weights dequantised
 *     into the matmul, and the closed-form backward dX, dA, dB;
 *   - FastVideo API docs, fastvideo.models.loader.lora_patch, DenseLoRAPatch:
 *     .diff / .diff_b additive deltas summed in float32 and .set_weight replacement.
 *
 * Conventions for every entry point:
 *   - All tensors are row-major.  X [T, in], W [out, in], A [r, in], B [out, r],
 *     bias [1, out], Y [T, out].  "ld" is the row pitch in elements.
 *   - Every data pointer is a DEVICE pointer on the current CUDA device; the caller
 *     owns all memory.  The library allocates no device memory, never synchronises
 *     and launches only on the caller's stream (`stream` is a cudaStream_t; NULL is
 *     the legacy default stream).  Inputs are never written.
 *   - Return value: WP_OK (0) or a negative WP_ERR_* code.  Argument checks run on
 *     the host before anything is launched; a rejected call launches nothing.
 *   - An empty batch (a matrix of zero rows: T = 0 tokens) is legal and its pointers may
 *     be null; such a call writes nothing, except lora_linear_bwd, whose dA and dB are
 *     then sums over no tokens and are set to zero.
 *   - A kernel whose bounded wait expires records WP_ERR_TIMEOUT in a device status
 *     word instead of hanging; read it with lora_device_status() after the stream has
 *     been synchronised.  The word is sticky until reset: while it reads WP_ERR_TIMEOUT,
 *     the outputs of every call made since the last reset are undefined (a kernel that
 *     gave up leaves its outputs partly written, and a later pass of the same call may
 *     have combined stale scratch), even though each of those calls returned WP_OK.
 */
#ifndef WEIGHT_PATCHES_H
#define WEIGHT_PATCHES_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* storage types */
enum {
  WP_BF16 = 0, /* bfloat16 */
  WP_FP32 = 1, /* IEEE binary32 */
  WP_NF4 = 2   /* 4-bit NormalFloat: packed codes + one fp32 absmax per 64 elements */
};

/* status codes */
enum {
  WP_OK = 0,
  WP_ERR_INVALID = -1,     /* null pointer, non-finite alpha/strength/scale, rank <= 0, bad kind */
  WP_ERR_SHAPE = -2,       /* dimensions disagree (e.g. payload numel != parameter numel) */
  WP_ERR_DTYPE = -3,       /* unsupported storage type or combination */
  WP_ERR_ALIGN = -4,       /* a pointer or row pitch breaks the 16-byte alignment rule */
  WP_ERR_WORKSPACE = -5,   /* workspace missing or smaller than lora_workspace_size() */
  WP_ERR_CUDA = -6,        /* a CUDA runtime/driver call or a launch failed */
  WP_ERR_TIMEOUT = -7,     /* a bounded device wait expired (device status word) */
  WP_ERR_UNSUPPORTED = -8  /* a size beyond the documented limits */
};

/* dense-patch kinds */
enum { WP_PATCH_ADD = 0, WP_PATCH_SET = 1 };

/* An input matrix.  For WP_NF4, `data` holds rows*cols/2 bytes (row-major; byte k of
 * the stream holds element 2k in its high nibble and element 2k+1 in its low
 * nibble), `absmax` holds rows*cols/64 fp32 scales (one per 64 consecutive
 * elements), cols % 64 == 0, and `ld` must equal `cols`. */
typedef struct wp_mat {
  const void* data;
  int32_t dtype;
  int64_t rows, cols, ld;
  const float* absmax;
} wp_mat;

/* An output matrix (WP_BF16 or WP_FP32). */
typedef struct wp_out {
  void* data;
  int32_t dtype;
  int64_t rows, cols, ld;
} wp_out;

/* One low-rank patch.  A [r, in], B [out, r] (for grouped calls, out = the group's
 * width); both WP_BF16, or both WP_FP32 for an FP32 adapter.  The combined scale
 * s = alpha / r * strength * request_scale is formed on the host in double and
 * rounded once to fp32; an adapter whose s is exactly +-0 contributes nothing.
 * bias_B: the optional vector older PEFT/Wan adapters carry beside A and B (their
 * lora_B.bias; piper-offload docs, "LoRA merge"), [out] contiguous on the device,
 * WP_BF16 or WP_FP32 (bias_B_dtype), or NULL.  The forwards add s * bias_B to the
 * adapter's output columns (also when the layer has no bias of its own); lora_merge adds
 * it to the module's bias; the backward's dX, dA and dB do not depend on it. */
typedef struct wp_adapter {
  wp_mat A;
  wp_mat B;
  double alpha;
  double strength;
  const void* bias_B;
  int32_t bias_B_dtype;
} wp_adapter;

/* Operation ids for lora_workspace_size(). */
enum { WP_OP_FWD = 0, WP_OP_FWD_GROUPED = 1, WP_OP_BWD = 2, WP_OP_FWD_HOST = 3, WP_OP_SWIGLU_FWD = 4, WP_OP_MERGE = 5,
       WP_OP_FWD_EXACT = 6, WP_OP_NORM_BWD = 7, WP_OP_RESIDUAL_NORM_BWD = 8 };

/* Norm kinds: layer norm (mean taken out) and the form without a mean (RMS norm). */
enum { WP_NORM_NONE = -1, WP_NORM_LAYER = 0, WP_NORM_RMS = 1 };

/*
 * lora_linear_fwd -- Y = X W^T + bias + sum_p s_p (X A_p^T) B_p^T.
 * (sglang PR "Add the dynamic LoRA delta inside the second GEMM", Modifications;
 *  InvokeAI sidecar-patch article, section 四, for the sum over patches.)
 *
 *   X        [T, in], WP_BF16 (tensor-core path) or WP_FP32 (exact FP32 path).
 *   W        [out, in], WP_BF16 or WP_NF4 with a bf16 X, WP_FP32 with an fp32 X;
 *            NULL computes the low-rank delta only.
 *   bias     [1, out] WP_BF16 or WP_FP32, or NULL; added in the epilogue.  With adapters
 *            that carry a legacy bias_B (and a non-zero s), bias + sum_p s_p bias_B_p is
 *            first formed in fp32 in the workspace (the first ceil256(4 out) bytes) and
 *            that vector is what the epilogue adds.
 *   adapters n_adapters patches (0..12); bf16 adapters on a bf16 X run on the tensor
 *            cores.  FP32 adapters on a bf16 X run there too, as three bf16 pieces per
 *            factor (every product above 2^-24 of the leading one is kept), when the
 *            call's rank columns allow; otherwise they run in FP32 on the CUDA cores.
 *            Either way their terms join the same FP32 accumulator before the single
 *            output rounding.
 *   Y        [T, out] WP_BF16 or WP_FP32, ld >= out; must not overlap the inputs.
 *   workspace device scratch of at least lora_workspace_size(WP_OP_FWD, ...) bytes
 *            (may be NULL when that size is 0).
 * Alignment (tensor-core path): every base pointer 16-byte aligned, every ld a
 * multiple of 8 elements (bf16) / 4 (fp32), in % 8 == 0, out % 8 == 0.
 * Limits (tensor-core path): at most 8 adapters on the tensor cores, each of rank <= 256.
 * A bf16 adapter counts ceil(r / 16) * 16 rank columns, an FP32 adapter as pieces
 * 3 * ceil(r / 16) * 16.  When the adapters' rank columns fit one 256-column accumulator,
 * s X A^T of all of them comes from one extra pass over X per 256 token rows; otherwise
 * the adapters (whole) are grouped into several such rank passes of at most 256 columns
 * each (e.g. three rank-128 q/k/v adapters: two passes), and FP32 adapters then take the
 * CUDA-core route (at most 4 of them), as they do whenever their pieces do not fit.
 * Few tokens (bf16 X and adapters): one to four tokens with in % 256 == 0 stream the
 * weight once on the CUDA cores; up to 64 tokens with a WP_NF4 weight (4 with bf16)
 * stream it through swapped tensor-core MMAs.  Both keep the same W_eff and the single
 * bf16 rounding of s X A^T, sum in fp32, and leave fp32 partial sums in the workspace
 * (lora_workspace_size counts them).
 */
int lora_linear_fwd(const wp_mat* X, const wp_mat* W, const wp_mat* bias,
                    const wp_adapter* adapters, int32_t n_adapters, double request_scale,
                    const wp_out* Y, void* workspace, size_t workspace_bytes, void* stream);

/*
 * lora_linear_fwd_grouped -- stacked column groups (q/k/v, gate/up):
 *   Y[:, g*out_g:(g+1)*out_g] = X W_g^T + bias_g + s_g (X A_g^T) B_g^T,
 * with W_stacked = [W_0; ...; W_{G-1}] of shape [G*out_g, in] and one adapter per
 * group (adapters[g], B_g of shape [out_g, r_g]).
 * (sglang PR, Modifications: one update per group on column views of the output;
 *  Unsloth walkthrough, section 4, LoRA_QKV.)
 * Same dtypes, alignment and ownership as lora_linear_fwd; 1 <= n_groups <= 8,
 * out_g % 8 == 0.
 */
int lora_linear_fwd_grouped(const wp_mat* X, const wp_mat* W_stacked, const wp_mat* bias,
                            int32_t n_groups, const wp_adapter* adapters, double request_scale,
                            const wp_out* Y, void* workspace, size_t workspace_bytes,
                            void* stream);

/*
 * lora_linear_fwd_host -- lora_linear_fwd (n_groups == 0) or lora_linear_fwd_grouped
 * (n_groups >= 1) with X and Y in host memory, for callers whose activations live on the
 * host.  A deployment variant with no counterpart in the pages.
 *
 * The rows are processed in chunks of 2048: the host-to-device copy of chunk i + 1, the
 * forward of chunk i and the device-to-host copy of chunk i - 1 run at the same time on
 * three streams owned by the library (created on the first call per device); the call
 * returns at once and `stream` waits for the whole operation.  X and Y should be pinned
 * (page-locked) for the copies to overlap; pageable memory works, serialised.
 *   X_host  [T, in] WP_BF16 (or WP_FP32 for the all-FP32 layer), host pointer.
 *   W, bias, adapters, request_scale: as lora_linear_fwd / lora_linear_fwd_grouped (device).
 *   Y_host  [T, out] WP_BF16 or WP_FP32, host pointer, ld >= out.
 *   workspace  device scratch of at least lora_workspace_size(WP_OP_FWD_HOST, X_host, W,
 *              adapters, n_adapters) bytes: two device chunks of X and of Y, and the
 *              forward's own scratch for one chunk.
 * Errors as lora_linear_fwd; a failure found after copies were queued still returns its
 * status, and `stream` then does not wait for the internal streams.
 */
int lora_linear_fwd_host(const wp_mat* X_host, const wp_mat* W, const wp_mat* bias,
                         int32_t n_groups, const wp_adapter* adapters, int32_t n_adapters,
                         double request_scale, const wp_out* Y_host, void* workspace,
                         size_t workspace_bytes, void* stream);

/*
 * lora_merge -- bake adapters into the base weight in place (piper-offload docs, "LoRA
 * merge" and "Quantized weight support"; the PEFT merge):
 *     W <- W + sum_p s_p B_p A_p,   s_p = alpha_p / r_p * strength_p * scale,
 *     bias <- bias + sum_p s_p bias_B_p   (adapters that carry the legacy vector),
 * every adapter of the call taken as one update, accumulated in fp32 and rounded once:
 *   W WP_BF16 [out, in] (device): bf16_rne(fl32(W) + ...);
 *   W WP_NF4 (codes [out, in/2] and absmax [out*in/64], device, both rewritten): dequantised
 *     to W_eff, the update added in fp32, re-encoded with deterministic round-to-nearest: per
 *     64-element block absmax' = max |u|, code = the nearest level of u / absmax' (a value on
 *     a midpoint between two levels takes the lower code), an all-zero block keeps scale 0.
 *   adapters: bf16 A [r, in], B [out, r]; strength 0 skips one; scale -1 undoes an earlier
 *   merge of the same adapters up to the roundings.
 *   workspace: lora_workspace_size(WP_OP_MERGE, NULL, W, adapters, n) bytes (A^T copies, and
 *   an fp32 [out, in] buffer for several adapters on a bf16 W, or for a 4-bit W with a rank
 *   above 256; a 4-bit W with ranks up to 256 is dequantised, updated and requantised block by
 *   block in one pass, with the same arithmetic).
 *   bias: the module's bias [out] (WP_BF16 or WP_FP32, device, rewritten in place) or NULL.
 *   The legacy vectors are added in fp32 in call order (each term fl32(s_p * v)) and the
 *   sum rounded once to the bias's dtype; for one adapter that is the dense patch's add.
 * Errors: WP_ERR_SHAPE, WP_ERR_DTYPE (fp32 adapters), WP_ERR_ALIGN (bf16 W rows must be
 * 16-byte aligned), WP_ERR_WORKSPACE; WP_ERR_INVALID, before anything is written, when an
 * adapter with a non-zero s carries a legacy vector and bias is NULL (the merge does not
 * create a bias the module does not have).  With no non-zero adapter nothing is launched.
 */
int lora_merge(const wp_mat* W, const wp_out* bias, const wp_adapter* adapters, int32_t n_adapters,
               double scale, void* workspace, size_t workspace_bytes, void* stream);

/*
 * lora_merge_seeded -- lora_merge with the stochastic re-encoding of a 4-bit weight
 * (piper-offload docs, "LoRA merge": the default for quantised merges, so that updates smaller
 * than one quantisation step are not rounded away systematically).  The block scales are the
 * deterministic ones (absmax' = max |u|); only each code is sampled, between the two levels
 * around x = fl32(u / absmax'): x on a level keeps that level's code, otherwise the upper
 * level lo < x < hi is taken when U * w < d * 2^23 (d = fl32(x - lo), w = fl32(hi - lo)), U
 * being the element's 23-bit draw: word e % 4 of Philox4x32-10 (Salmon et al., SC 2011) of
 * counter (e / 4 as two 32-bit words, 0, 0) under key (the seed's low and high 32 bits), shifted
 * right by 9, e = row * in + column the element's logical index -- so the codes depend on the
 * seed and the data only, not on the launch.  The same seed gives the same codes.  A bf16 W has
 * no code to sample: the call is lora_merge.  Arguments, workspace and errors as lora_merge.
 */
int lora_merge_seeded(const wp_mat* W, const wp_out* bias, const wp_adapter* adapters, int32_t n_adapters,
                      double scale, uint64_t rounding_seed, void* workspace, size_t workspace_bytes,
                      void* stream);

/*
 * lora_swiglu_fwd -- the front half of a SwiGLU LoRA MLP in one pass: the gate and up
 * LoRA linears and the activation,
 *     e = X W_gate^T + bias_gate + s_g (X A_g^T) B_g^T,
 *     g = X W_up^T   + bias_up   + s_u (X A_u^T) B_u^T,
 *     h = silu(e) g,   silu(e) = e / (1 + exp(-e)).
 * (Unsloth fast_lora walkthrough, section 4, LoRA_MLP forward: e and g by two LoRA
 *  matmuls, h by the SwiGLU kernel, e and g kept for the backward.)
 *   X [T, in] WP_BF16; W_gate_up [2F, in] WP_BF16 or WP_NF4, gate rows 0..F-1 then up
 *   rows F..2F-1; bias [2F] (gate then up) or NULL; adapters[0] the gate adapter
 *   (B [F, r]), adapters[1] the up adapter (strength 0 disables one); bf16 adapters, or
 *   FP32 ones small enough to ride as bf16 pieces.
 *   H [T, F] WP_BF16 output.  EG [T, 2F] WP_BF16 or NULL: receives e | g.
 * e and g are rounded to bf16 once (EG holds exactly those values, bit-equal to
 * lora_linear_fwd_grouped with n_groups = 2), h = bf16(silu(e) * g) from them, so the
 * h that lora_swiglu_bwd recomputes from EG is bit-equal to H.
 *   workspace: lora_workspace_size(WP_OP_SWIGLU_FWD, X, W_gate_up, adapters, 2) bytes.
 * Limits: as lora_linear_fwd_grouped; F % 8 == 0.  Errors as lora_linear_fwd.
 */
int lora_swiglu_fwd(const wp_mat* X, const wp_mat* W_gate_up, const wp_mat* bias,
                    const wp_adapter* adapters, double request_scale, const wp_out* H,
                    const wp_out* EG, void* workspace, size_t workspace_bytes, void* stream);

/*
 * lora_swiglu_bwd -- the SwiGLU step of the LoRA MLP backward, elementwise.  From the
 * gradient dH at h (the dX of the down projection) and the saved e | g:
 *     f = silu(e),  dg = dH f,  de = dH g sigmoid(e) (1 + e (1 - sigmoid(e))),
 * and, when H is given, h = f g again (for the down adapter's gradients).
 * (Unsloth fast_lora walkthrough, section 4, LoRA_MLP backward: one kernel gives h and
 *  the gradients at g and e.)
 *   dH [T, F], EG [T, 2F] WP_BF16 inputs; dEG [T, 2F] WP_BF16 output, de | dg (the
 *   stacked output gradient for the grouped gate/up backward); H [T, F] WP_BF16 or NULL.
 * Every product is one float32 rounding, each output one bf16 rounding.
 * Errors: WP_ERR_SHAPE, WP_ERR_DTYPE (not bf16), WP_ERR_ALIGN (16-byte bases, F and
 * row pitches multiples of 8 elements).  Outputs must not overlap the inputs.
 */
int lora_swiglu_bwd(const wp_mat* dH, const wp_mat* EG, const wp_out* dEG, const wp_out* H,
                    void* stream);

/*
 * lora_linear_bwd -- closed-form gradients of Y = X W_g^T + s_g (X A_g^T) B_g^T over
 * n_groups column groups (n_groups = 1 for a plain layer), with G_g = dY_g B_g:
 *     dX   = sum_g dY_g W_g + s_g G_g A_g          [T, in]
 *     dA_g = s_g G_g^T X                          [r_g, in]
 *     dB_g = s_g dY_g^T (X A_g^T)                 [out_g, r_g]
 * (Unsloth fast_lora walkthrough, sections 2 and 4: dX, dA, dB by hand, no
 *  autograd graph, only X kept from the forward.)
 *   X [T, in] WP_BF16; W [G*out_g, in] WP_BF16 or WP_NF4; dY [T, G*out_g] WP_BF16.
 *   dX: WP_BF16 or WP_FP32 output, or NULL to skip; dA[g], dB[g]: WP_FP32 outputs.
 *   dA/dB are overwritten (not accumulated).
 * Limits: bf16 adapters, r_g <= 128 each (any sum over the groups); in % 8 == 0 and
 * out_g % 8 == 0.
 */
int lora_linear_bwd(const wp_mat* X, const wp_mat* W, const wp_mat* dY, int32_t n_groups,
                    const wp_adapter* adapters, double request_scale, const wp_out* dX,
                    const wp_out* dA, const wp_out* dB, void* workspace,
                    size_t workspace_bytes, void* stream);

/*
 * lora_dense_patch -- the dense half of an adapter, applied in place to `param`.
 * (FastVideo API docs, fastvideo.models.loader.lora_patch, DenseLoRAPatch.apply_to
 *  and replacement_for.)
 *   kind WP_PATCH_ADD (.diff / .diff_b): param = cast(fp32(param) + fp32(payload) * k)
 *   kind WP_PATCH_SET (.set_weight):     param = cast(fp32(payload) * k)
 * where k = (float)strength, the product and the sum are separate float32 roundings
 * (no fused multiply-add) and cast is round-to-nearest-even into param_dtype.
 *   param: param_numel elements of param_dtype (WP_BF16 or WP_FP32), device.
 *   payload: payload_numel elements of payload_dtype (WP_BF16 or WP_FP32), device.
 * Errors: WP_ERR_SHAPE if payload_numel != param_numel; WP_ERR_INVALID for a
 * non-finite strength or unknown kind.  param and payload must not overlap.
 */
int lora_dense_patch(void* param, int32_t param_dtype, int64_t param_numel,
                     const void* payload, int32_t payload_dtype, int64_t payload_numel,
                     int32_t kind, double strength, void* stream);

/*
 * lora_linear_fwd_exact -- the unfused dynamic-LoRA chain, the "exact" tier.
 * (sglang PR "[diffusion] Add the dynamic LoRA delta inside the second GEMM", Motivation:
 *  the chain every dynamic layer ran before the fused design; Modifications: the exact
 *  tier keeps that chain and skips multiplications by a unit scale, which leaves every bit
 *  of the output as it was.)
 *     Y = bf16(X W^T + bias)
 *     for each adapter p, in order (its column group when n_groups > 0):
 *       t = bf16(X A_p^T);  d = bf16(t B_p^T [+ bias_B,p])
 *       d = bf16(d * c) for c = fl32(alpha_p / r_p), fl32(strength_p), fl32(request_scale)
 *       Y = bf16(Y + d)
 *   An FP32 adapter keeps its two GEMMs and its scaling in FP32 (s = alpha/r * strength *
 *   request_scale formed in double) and is added once: Y = bf16(Y + fl32 delta).
 *   skip_unit_scales != 0 skips each scale multiplication whose c is exactly 1.0 (the PR's
 *   exact tier); 0 runs every one (the chain before the PR).  The two give bit-identical Y.
 *   Every elementwise step is the correctly rounded bf16 of its exact result; the GEMMs sum
 *   in fp32 on the tensor cores.  This path materialises t and d (it is the reference the
 *   fused lora_linear_fwd improves on), so it is slower by design.
 *   X [T, in] WP_BF16; W [n_groups * out_g, in] (or [out, in]) WP_BF16 or WP_NF4; bias as
 *   lora_linear_fwd; adapters: n_adapters (== n_groups when n_groups > 0); Y [T, out] WP_BF16.
 *   workspace: lora_workspace_size(WP_OP_FWD_EXACT, X, W, adapters, n_adapters) bytes.
 * Limits: bf16 adapters of rank r % 8 == 0 (t is a GEMM output); out_g % 8 == 0; the
 * alignment rules of lora_linear_fwd.  Errors as lora_linear_fwd.
 */
int lora_linear_fwd_exact(const wp_mat* X, const wp_mat* W, const wp_mat* bias, int32_t n_groups,
                          const wp_adapter* adapters, int32_t n_adapters, double request_scale,
                          int32_t skip_unit_scales, const wp_out* Y, void* workspace, size_t workspace_bytes,
                          void* stream);

/*
 * lora_linear_fwd_noalloc -- lora_linear_fwd for callers that cannot provide or allocate
 * device scratch memory.  The pages have no counterpart: this is a deployment variant.
 *
 * Who needs it: code embedded in a host that owns all device memory through its own
 * allocator and gives plug-ins no allocation rights, fixed-budget inference servers, and
 * latency-critical paths where cudaMalloc/cudaFree (which may synchronise the device)
 * are not acceptable.  Such a caller still passes its inputs and output; the scratch that
 * lora_workspace_size(WP_OP_FWD, ...) reports (on the tensor-core path about T x sum of the
 * ranks rounded up to 16 x 2 bytes for the bf16 s * X A^T rows, plus the FP32 adapters'
 * share; on the all-FP32 path T x sum of the ranks floats) comes from a fixed 4 MiB array
 * inside the library, held on every device that uses it until the process exits.  The
 * call allocates nothing.
 *
 * Same arguments, dtypes, alignment rules and errors as lora_linear_fwd, minus the
 * workspace.  A call whose general path would need more than 4 MiB of scratch (the
 * minimum above, not counting the few-token routes' partial sums) is rejected with
 * WP_ERR_WORKSPACE before anything is launched (lora_last_cuda_error() says how much was
 * needed).  A call of 1 to 64 tokens takes a few-token route only when that route's fp32
 * partial sums (splits x T x (out + sum of the ranks rounded up to 16) x 4 bytes) fit the
 * array as well; otherwise it runs on the general path, with the same results within the
 * tolerances of lora_linear_fwd.  The first call on each device looks up the array's device address
 * (cudaGetSymbolAddress) with that device current; make that first call before any stream
 * capture.  Every call on a device shares the one array and leaves its contents behind
 * (the call clears the few flags it needs on its stream; every other scratch element is
 * written before it is read): calls whose kernels overlap on the GPU, e.g. on two streams
 * at once, race on it and must be serialised by the caller.
 */
int lora_linear_fwd_noalloc(const wp_mat* X, const wp_mat* W, const wp_mat* bias,
                            const wp_adapter* adapters, int32_t n_adapters, double request_scale,
                            const wp_out* Y, void* stream);

/* ------------------------------------------------------------ adapters of many requests
 * A bank holds the adapters of one layer, one per slot, each padded to the bank's rank with
 * zero rows of A (zero columns of B):
 *   A [n_slots, n_groups * rank, in]   group g's rows g * rank .. (g + 1) * rank - 1
 *   B [n_slots, out, rank]             out = n_groups * out_g stacked output rows
 * both WP_BF16, contiguous, 16-byte aligned; scale [n_slots] fp32 (alpha / r * strength of
 * each adapter), all on the device.  rank % 8 == 0, 8 <= rank <= 256. */
typedef struct wp_bank {
  const void* A;
  const void* B;
  const float* scale;
  int32_t dtype;
  int32_t n_slots, n_groups, rank;
  int64_t in, out;
} wp_bank;

/*
 * lora_linear_fwd_multi -- one shared projection for rows that belong to the requests of many
 * adapters (sglang PR, Motivation: the adapter and its scale belong to the request):
 *   Y[t, g] = X[t] W_g^T + bias_g + s_t (X[t] A_{a,g}^T) B_{a,g}^T,   a = slot[t],
 *   s_t = scale[a] * row_scale[t] * request_scale
 * (products of fp32, rounded one after another), per column group g of bank->n_groups.
 *   X        [T, in] WP_BF16.
 *   W        [out, in] WP_BF16 or WP_NF4, or NULL (the adapters' term alone).
 *   bias     [out] WP_BF16 or WP_FP32, or NULL.
 *   slot     [T] int32 on the device, in any order; a value outside 0 .. n_slots - 1 (-1 by
 *            convention) means that the row uses no adapter.  The values may change between
 *            replays of a captured graph.
 *   row_scale [T] fp32 on the device or NULL (1): the scale of each row's request.
 *   Y        [T, out] WP_BF16 or WP_FP32; must not overlap the inputs.
 * A row's result is that row's and its adapter's: values that are not finite in one slot or row
 * do not reach rows of other slots, and a row without an adapter, or whose s_t is exactly 0, is
 * bit for bit the row that this call gives when no row of the batch has one.  The order of an
 * adapted row's sums, and so its last bits, go by the batch as well (its rows, and how many of
 * them share a slot); the same call gives the same bits.  As in lora_linear_fwd, s X A^T is rounded
 * once to bf16 (one or two rows of few ranks keep it in fp32), sums are fp32 and the output is
 * rounded once.
 *   workspace: lora_multi_workspace_size(X, W, bank) bytes, 16-byte aligned; the size for more
 *   rows serves fewer, too, and a larger one changes nothing.
 * Alignment: as lora_linear_fwd's tensor-core path (16-byte bases and pitches, in % 8 == 0,
 * out_g % 8 == 0); n_groups <= 8.  Errors as lora_linear_fwd; WP_ERR_DTYPE for a bank that is
 * not bf16, WP_ERR_UNSUPPORTED for a rank above 256.
 */
int lora_linear_fwd_multi(const wp_mat* X, const wp_mat* W, const wp_mat* bias, const wp_bank* bank,
                          const int32_t* slot, const float* row_scale, double request_scale,
                          const wp_out* Y, void* workspace, size_t workspace_bytes, void* stream);

/* Bytes of device workspace that lora_linear_fwd_multi needs (0: a rejected shape). */
size_t lora_multi_workspace_size(const wp_mat* X, const wp_mat* W, const wp_bank* bank);

/* ------------------------------------------------------------------------- norms
 * lora_norm_fwd -- y = (x - mu) r w + b over the rows of X, r = 1 / sqrt(var + eps)
 *   WP_NORM_LAYER: mu the row's mean, var its mean squared distance from mu;
 *   WP_NORM_RMS:   mu = 0, var the mean square.
 * (FastVideo API docs, DenseLoRAPatch: .diff / .diff_b payloads on norm vectors; this is the
 *  layer those vectors belong to, and lora_norm_bwd gives the gradients that train them.)
 *   X [T, C] WP_BF16 or WP_FP32, any row pitch; weight, bias [C] WP_BF16 or WP_FP32 or NULL
 *   (1 and 0); Y [T, C] of X's dtype.
 *   stats [2, T] fp32 or NULL: the rows' mu and r, for the backward.
 * Sums are fp32, the mean taken out before squaring; one output rounding.  eps >= 0, finite.
 */
int lora_norm_fwd(const wp_mat* X, const wp_mat* weight, const wp_mat* bias, int32_t kind, double eps,
                  const wp_out* Y, float* stats, void* stream);

/*
 * lora_norm_bwd -- with xh = (x - mu) r and h = dy w:
 *   dx = r (h - mean(h) - xh mean(h xh))      (WP_NORM_RMS: without mean(h))
 *   dw = sum over rows of dy xh,   db = sum over rows of dy.
 *   dY, X [T, C] of one dtype (WP_BF16 or WP_FP32); stats [2, T] as lora_norm_fwd wrote them;
 *   dX [T, C] of X's dtype or NULL; dW, dB [1, C] WP_FP32 or NULL, overwritten (zero for no
 *   rows).  weight NULL: 1.
 *   workspace: lora_workspace_size(WP_OP_NORM_BWD, X, NULL, NULL, 0) bytes when dW or dB is
 *   asked for.  Row sums are added in a fixed order: the same call gives the same bits.
 */
int lora_norm_bwd(const wp_mat* dY, const wp_mat* X, const wp_mat* weight, const float* stats, int32_t kind,
                  const wp_out* dX, const wp_out* dW, const wp_out* dB, void* workspace,
                  size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------------- between two blocks
 * A block's output gated onto the residual stream, and the norm ahead of the next block with its factor
 * and shift:
 *   u  = norm1(y) post_weight (post_kind WP_NORM_NONE: u = y),   x1 = x + alpha gate u,
 *   h  = norm2(x1) (mul_offset + mul) + add
 * gate, mul, add: [n, C], row g for the g-th of n equal runs of consecutive rows (one vector for all rows:
 * n = 1; one per sample of a batch: n samples; T % n == 0; mul and add of the same n), or NULL (gate, and the
 * factor as a whole, 1; add 0).  A learned weight is mul with mul_offset 0, a modulation mul with
 * mul_offset 1.  post_weight [1, C] or NULL (1).  All WP_BF16 or WP_FP32, any address of their type. */
typedef struct wp_residual_norm {
  const wp_mat* gate;
  const wp_mat* mul;
  const wp_mat* add;
  const wp_mat* post_weight;
  double alpha, mul_offset, eps, post_eps;
  int32_t kind;        /* norm2: WP_NORM_LAYER or WP_NORM_RMS */
  int32_t post_kind;   /* norm1: these, or WP_NORM_NONE */
} wp_residual_norm;

/*
 * lora_residual_norm_fwd
 *   X [T, C] the stream, WP_FP32 or WP_BF16; Y [T, C] the block's output or NULL (h of X alone; then no
 *   gate, post norm or X_out); X_out [T, C] of X's type or NULL (not wanted), X itself included; H [T, C] of
 *   Y's type.  Y and H are WP_BF16, or WP_FP32 with a WP_FP32 stream.
 *   stats [4, T] fp32 or NULL: mean and factor of norm2, then (rows 2 and 3, with a post norm only) of norm1.
 *   Outputs overlap no input but for X_out in X's place.
 * C <= 16384, T < 2^30, any pitch; 16-byte aligned rows are fastest.  Sums are fp32, means taken out before squaring;
 * h is formed from x1 before its rounding to X_out's type; one rounding per output.  The order of a row's sums, and so
 * the last bits, go by the rows' length and types and by the addresses' and pitches' alignment, not by the rows' number; the
 * same call gives the same bits.
 */
int lora_residual_norm_fwd(const wp_mat* X, const wp_mat* Y, const wp_residual_norm* a, const wp_out* X_out,
                           const wp_out* H, float* stats, void* stream);

/*
 * lora_residual_norm_bwd -- from dH at h and dX1 (NULL: zero) at the new stream, X1 and Y as the forward wrote
 * and read them, and its stats:
 *   dX [T, C] of X1's type (the gradient at x), dY [T, C] of dH's type; either may be NULL.  dX may be dX1; outputs overlap no
 *   other input.
 *   dgate, dmul, dadd [n, C], dpost_weight [1, C]: WP_FP32, or NULL; overwritten (zero for no rows).  dgate, dmul
 *   and dpost_weight need their vector in `a`; of a->add only dadd's shape matters.
 *   workspace: lora_workspace_size(WP_OP_RESIDUAL_NORM_BWD, X1, NULL, NULL, 0) bytes, 16-byte aligned, when one of those
 *   four is asked for.  Sums are added in a fixed order: the same call gives the same bits.
 */
int lora_residual_norm_bwd(const wp_mat* dH, const wp_mat* dX1, const wp_mat* X1, const wp_mat* Y, const float* stats,
                           const wp_residual_norm* a, const wp_out* dX, const wp_out* dY, const wp_out* dgate,
                           const wp_out* dmul, const wp_out* dadd, const wp_out* dpost_weight, void* workspace,
                           size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------------- rotary positions
 * The heads of a query or key tensor: element (t, h, d) at data[t ld_token + h ld_head + d], so a view of
 * the stacked q/k/v output ([T, 3 C]: ld_token 3 C, ld_head dim) and a [heads, tokens, dim] tensor both are. */
typedef struct wp_heads {
  const void* data;   /* written where the struct is an output */
  int32_t dtype;      /* WP_BF16 or WP_FP32 */
  int64_t tokens, heads, dim;
  int64_t ld_token, ld_head;
} wp_heads;

/* Which elements turn together: neighbours (2i, 2i + 1), or halves (i, i + rot / 2). */
enum { WP_ROPE_PAIRS = 0, WP_ROPE_HALF = 1 };

/*
 * lora_rope -- rotary positions of q and, in the same launch, k (NULL: q alone):
 *   (a, b) <- factor (a cos th - b sin th, a sin th + b cos th),   th = positions[axis(i)][t] inv_freq[i]
 * for the pairs i = 0 .. rot / 2 - 1 of the first rot elements of every head; the rest of a head is copied
 * (in place: left alone).  inverse: th negated, which is the gradient's way back (the same factor).
 *   positions [n_axes, T] int32 on the device, ld_positions apart (any value; a video's frame, row and
 *   column are three axes); axis_pairs (host) [n_axes]: how many of the pairs, in order, go by each axis,
 *   adding up to rot / 2.  inv_freq [rot / 2] fp64 on the device (a context that was lengthened by other
 *   frequencies passes those, and its scale as factor).
 *   The angle is reduced exactly (in 64-bit fractions of a turn), so far positions lose nothing; products are
 *   fp32, the output is rounded once.
 *   Q_out, K_out of their input's type and sizes: the input itself (in place, with its strides), or memory
 *   that does not overlap the inputs; no two of its elements may share memory.
 * Limits: n_axes <= 4, dim <= 1024, rot even; a frequency of 2^52 or more (or not finite) gives NaN.  Any strides and
 * element-aligned addresses; 16-byte aligned ones are fastest.
 */
int lora_rope(const wp_heads* Q, const wp_heads* K, const int32_t* positions, int64_t ld_positions,
              const double* inv_freq, int32_t rot, int32_t n_axes, const int32_t* axis_pairs, int32_t layout,
              double factor, int32_t inverse, const wp_heads* Q_out, const wp_heads* K_out, void* stream);

/* ------------------------------------------------------------------------- loss
 * lora_ce_fwd -- softmax cross entropy of every row of X against a vocabulary's weight, without
 * keeping the logits (a training step's loss; the score of a token):
 *   z[t, v] = logit_scale sum_k X[t, k] W[v, k],   lse[t] = log sum_v exp z[t, v],
 *   loss[t] = lse[t] - z[t, target[t]]
 *   X [T, K], W [V, K] WP_BF16, K % 8 == 0, K <= 2^24, 16-byte aligned bases and pitches.
 *   target [T] int32 or int64 (target_bits 32 or 64) on the device.  A row whose target is outside
 *   0 .. V - 1 (-100 by convention) does not count: its loss and lse are 0, and nothing in it, not
 *   even NaN, is read into another row's result.  Of more than 256 rows it costs nothing either; up to
 *   256, W's one pass is the cost, whatever the rows.
 *   loss, lse [T] fp32; either may be NULL.
 *   workspace: lora_ce_workspace_size(X, W, 0) bytes, 16-byte aligned; the size for more rows serves
 *   fewer, too, and a larger one changes nothing.  (No two calls that may run at once may share one.)
 * Products are exact and summed in fp32: at most 1024 of them at a time on the tensor core, which cuts its sum every 16
 * products, and these sums with rounding to nearest: a logit is within about 2^-20 of its terms' magnitudes, and half a
 * step of fp32 for each further 1024 of K.  The same call gives the same bits; a row's last bits go by the number of rows,
 * too, whose forms change at 16, 32, 64, 128 and 256.
 */
int lora_ce_fwd(const wp_mat* X, const wp_mat* W, const void* target, int32_t target_bits, double logit_scale,
                float* loss, float* lse, void* workspace, size_t workspace_bytes, void* stream);

/*
 * lora_ce_bwd -- from the gradient dloss [T] fp32 at the rows' losses and the lse of lora_ce_fwd:
 *   G[t, v] = dloss[t] logit_scale (exp(z[t, v] - lse[t]) - [v = target[t]])   (0 in rows that do not count)
 *   dX = G W,   dW = G^T X
 *   dX [T, K], dW [V, K], WP_BF16 or WP_FP32, either NULL: not wanted; overwritten (dW of no rows: zeros).  They may not
 *   overlap an input.
 * The logits are formed again, a piece of the vocabulary at a time; a row of G over its own 1 - p[target] is rounded
 * once to bf16 (the target's entry is then exact), whatever the outputs' types; sums are fp32, outputs are rounded once.
 * dX takes the row's factor, dloss (1 - p[target]), in fp32.  dW takes it times X, in two bf16 parts (2^-16 of it is left)
 * while at most 512 rows count; beyond, in one, so that each term of dW is rounded to bf16 a second time.  Rows that do
 * not count change nothing in this.  Logits and both products are summed as the loss's logits, but 4096 products at a time:
 * each is within about 2^-17 of its terms' magnitudes, and half a step for each further 4096.  p is exp(z - lse) with the fp32 lse, so G's entries
 * are off by up to about p 2^-23 (|lse| + 1), and p times the logit's error, beyond their rounding: a row whose target has all
 * but some 1e-6 of the probability has a gradient of that size and no digits.  The same call gives the same bits.  dloss
 * and lse of rows that do not count are not read into anything.
 *   workspace: lora_ce_workspace_size(X, W, 1) bytes, 16-byte aligned, as above.
 */
int lora_ce_bwd(const wp_mat* X, const wp_mat* W, const void* target, int32_t target_bits, const float* lse,
                const float* dloss, double logit_scale, const wp_out* dX, const wp_out* dW, void* workspace,
                size_t workspace_bytes, void* stream);

/* Bytes of device workspace of lora_ce_fwd (backward 0) or lora_ce_bwd (1); 0: no rows, or a rejected shape. */
size_t lora_ce_workspace_size(const wp_mat* X, const wp_mat* W, int32_t backward);

/* ------------------------------------------------------------------------- AdamW
 * One tensor of an adapter set.  param [numel] WP_BF16 or WP_FP32; master [numel] fp32 or NULL:
 * when given (with a bf16 param) the step updates the master and param is its rounding.
 * state_bits 32: m, v [numel] fp32.  state_bits 8: m [numel] int8 codes, v [numel] uint8 codes
 * and one fp32 scale per 256 consecutive elements (m_absmax, v_absmax [ceil(numel / 256)]): a
 * code q of a block of scale a stands for
 *     m: a sign(q) (|q| / 127)^2,      v: a (q / 255)^4,
 * the nearest code in the root's domain, a v above zero never coded as zero.  Zeroed codes and
 * scales are the initial state. */
typedef struct wp_adamw_tensor {
  void* param;
  float* master;
  void* m;
  void* v;
  float* m_absmax;
  float* v_absmax;
  int64_t numel;
  int32_t param_dtype;
  int32_t state_bits;
} wp_adamw_tensor;

/* A prepared set: filled by lora_adamw_plan_init; `table` is the caller's device memory. */
enum { WP_ADAMW_MAX_LAUNCHES = 16, WP_ADAMW_TENSORS_PER_LAUNCH = 3900 };
typedef struct wp_adamw_plan {
  void* table;
  int32_t n_tensors;
  int32_t n_launches;
  int64_t unit_begin[WP_ADAMW_MAX_LAUNCHES + 1];
  uint32_t launches_8bit;  /* bit l: launch l has tensors with 8-bit moments */
} wp_adamw_plan;

/* The step's scalars.  g = grad * grad_scale (* grad_scale_dev[0] when not NULL: a clip or loss
 * scale formed on the device); step counts from 1. */
typedef struct wp_adamw_args {
  double lr, beta1, beta2, eps, weight_decay, grad_scale;
  int64_t step;
  const float* grad_scale_dev;
} wp_adamw_args;

/* Device bytes of a set's table (0 for a rejected list). */
size_t lora_adamw_plan_size(const wp_adamw_tensor* tensors, int32_t n);

/* Writes the set's table into `table` (16-byte aligned device memory of lora_adamw_plan_size
 * bytes, which has to live as long as the plan is used) with small kernels on `stream`, and
 * fills *plan; a step on another stream has to be ordered after them.  At most 62400 tensors; every
 * pointer aligned to its element type; no two arrays may overlap (a tensor listed twice would be
 * updated by two CTAs at once: WP_ERR_INVALID). */
int lora_adamw_plan_init(const wp_adamw_tensor* tensors, int32_t n, void* table, size_t table_bytes,
                         wp_adamw_plan* plan, void* stream);

/*
 * lora_adamw_step -- one AdamW step (decoupled weight decay) over the whole set, in place:
 *     m <- b1 m + (1 - b1) g,   v <- b2 v + (1 - b2) g^2
 *     p <- p (1 - lr wd) - lr / (1 - b1^step) * m / (sqrt(v) / sqrt(1 - b2^step) + eps)
 * (the dA, dB of lora_linear_bwd and dW, dB of lora_norm_bwd are its gradients).  The scalars are
 * formed in double and rounded once to fp32; moments and parameters are fp32 while they are
 * updated (8-bit moments are coded again after p has used them), each product and sum of m and v
 * a separate rounding.  A gradient that is not finite reaches its element's p, m and v, and every
 * value of its 8-bit block.
 * The scalars travel with the launch: a captured graph replays the step number, rate and scale that it
 * was captured with (only *grad_scale_dev is read anew), so a graph serves one step number.
 *   grads: host array of n_tensors device pointers, all of grad_dtype (WP_FP32 or WP_BF16); NULL
 *   leaves that tensor and its state untouched.  Read before the call returns.
 * Errors: WP_ERR_INVALID for a scalar that is not finite, betas outside [0, 1), eps < 0, step < 1.
 */
int lora_adamw_step(const wp_adamw_plan* plan, const void* const* grads, int32_t grad_dtype,
                    const wp_adamw_args* args, void* stream);

/* The fp32 values of 8-bit moments: codes [numel] (int8 when is_signed, else uint8), absmax
 * [ceil(numel / 256)], out [numel]. */
int lora_block8_decode(const void* codes, int32_t is_signed, const float* absmax, int64_t numel, float* out,
                       void* stream);

/* Bytes of device workspace the given call needs (0 if none).  `op` is WP_OP_*;
 * the other arguments are those of the call (adapters: n_adapters, or n_groups). */
size_t lora_workspace_size(int32_t op, const wp_mat* X, const wp_mat* W,
                           const wp_adapter* adapters, int32_t n_adapters);

/* Human-readable text for a status code (static storage). */
const char* lora_status_string(int status);

/* Reads (and, if `reset` != 0, clears) the device status word of the current device:
 * WP_OK or WP_ERR_TIMEOUT.  Synchronous: call after the stream has finished. */
int lora_device_status(int32_t reset);

/* How long every bounded device wait of the library's kernels spins (mbarriers, the fused
 * forward's row-block flags) before the kernel records WP_ERR_TIMEOUT in the device status
 * word, drains its own copies in flight, frees its tensor memory and returns.  Applies to
 * calls made after it, process-wide.  Default 2 s; accepted range 1 ms .. 60 s, otherwise
 * WP_ERR_INVALID and the setting is unchanged.  Not in the pages: a safety bound of this
 * library's persistent kernels. */
int lora_set_wait_limit(uint64_t timeout_ns);

/* Test hook for the timeout path (not in the pages): while `on` is non-zero, the tiles of
 * every fused forward launched afterwards wait for one more release of their row-block flag
 * than any rank item gives, every one-pass 4-bit merge (ranks up to 256) leaves the MMAs
 * of its CTAs' last jobs unissued, and the residual norm's kernels for rows beyond 256 columns
 * send for none of them, so those bounded waits run out (after
 * lora_set_wait_limit's limit) and the call's outputs are left undefined;
 * lora_device_status() then reads WP_ERR_TIMEOUT.  Process-wide; 0 restores normal
 * operation.  Always returns WP_OK. */
int lora_debug_hold_flags(int32_t on);

/* The library's 16 NormalFloat levels in ascending order (host memory, fp32). */
void lora_nf4_codebook(float out[16]);

/* The last CUDA error text the library saw on this host thread ("" if none). */
const char* lora_last_cuda_error(void);

#ifdef __cplusplus
}
#endif

#endif /* WEIGHT_PATCHES_H */
