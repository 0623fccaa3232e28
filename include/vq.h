/*
 * vq.h -- C ABI of libvqmi.so: fused vector-quantized (VQ) weight matmul on
 * AMD MI355X (gfx950).
 *
 * The operation.  A weight matrix W [rows = out][cols = in] is stored as
 *   - codes: each run of d consecutive weights of a row (along cols) is one
 *     B-bit index (B = log2 K) into a K-entry codebook.  Paper "Data-Free
 *     Vector Quantization Beats Affine Quantization at Matched Bytes Below 5
 *     Bits", Abstract and §1 Notation (geometry dN/KM, log2(K)/d bits/weight).
 *   - codebook: K entries of d fp16 values, one codebook per tensor.  Model
 *     card "Qwen3.5-397B-A17B-VQ-2.4bpw", Methodology (per-tensor fp16
 *     codebook); paper §2.2 (codebook fit on max-abs-scaled subvectors).
 *   - scales: one fp16 scale per (row, group of g weights), g = 64 or 128.
 *     Same card, Methodology (an fp16 scale for each row and 64-weight group); model card
 *     "aquaman164/Qwen3.6-35B-A3B-MLX-VQ-2.4bpw", Recipe (+0.125 bpw: g = 128).
 * and dequantized on the fly:
 *   W[r][c] = fp16( codebook[code(r, c/d)][c % d] * scale[r][c/g] )  (one RNE
 * rounding; the product of two fp16 values is exact in fp32), then
 *   y[t][r] = sum_c W[r][c] * x[t][c]   (fp32 accumulation, fp32 output).
 * The GEMV kernels fold the scale out of each group's inner sum (the sum is
 * formed from exact fp16 x fp16 products in fp32 and multiplied by the scale
 * once per group), which differs from rounding W to fp16 first only by that
 * rounding; vq_dequant and the MFMA GEMM use the rounded W exactly.
 *
 * Code layout (codes packed to their true bit width into uint32 words, each
 * row on its own in blocks of 32 codes: 397B card, Methodology; paper §2.3
 * Packing).  Row r of expert
 * e starts at word (e*rows + r) * Wr, Wr = ceil(cols/d/32) * B.  Code j of a
 * row occupies bits [j*B, (j+1)*B) of the row's little-endian bit stream
 * (least significant bit first); 12-bit codes straddle words.  For B = 8 an
 * array of uint8 codes [rows][cols/d] already is this layout and can be
 * passed as is (397B card, Runtime update: zero-copy packed-8 view).
 *
 * Conventions for every entry point:
 *   - Pointers named as device data point to device memory the caller owns.
 *     The library never allocates device memory; scratch (vq_moe_gemm,
 *     vq_encode, vq_fp8_gemm, vq_mx4_gemm, vq_mx4_moe) comes from the caller's
 *     workspace.
 *   - fp16 values travel as uint16_t bit patterns.
 *   - `stream` is a hipStream_t (NULL = the default stream).  Work is enqueued
 *     on it without host synchronisation.
 *   - All arguments are validated on the host before anything is enqueued.
 *     On error nothing is enqueued, outputs are untouched, a status is
 *     returned and vq_last_error() describes it.  No C++ exception crosses
 *     the ABI.  Launch failures return VQ_ERR_HIP with HIP's error text.
 *   - Values inside device buffers (codes, expert ids) cannot be checked on
 *     the host.  Every code is in range by construction (B bits).  An expert
 *     id outside [0, num_experts) means "skip": that slot's output row is
 *     written as zeros.
 *   - Calls on one stream are ordered; the library keeps no state between
 *     calls apart from the thread-local error text and the thread's last plans
 *     of vq_fp8_gemm and vq_mx4_gemm, which depend on a call's sizes alone.
 */
#ifndef VQMI_VQ_H
#define VQMI_VQ_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  VQ_OK = 0,
  VQ_ERR_NULL = 1,      /* a required pointer is NULL                          */
  VQ_ERR_GEOMETRY = 2,  /* (d, log2_k, group) not supported                    */
  VQ_ERR_SHAPE = 3,     /* sizes inconsistent (see each check below)           */
  VQ_ERR_ALIGN = 4,     /* a buffer is not aligned as required                 */
  VQ_ERR_WORKSPACE = 5, /* a call's workspace is missing or too small           */
  VQ_ERR_HIP = 6        /* a HIP runtime call or kernel launch failed          */
} vq_status;

/*
 * One VQ tensor (dense: num_experts = 1; stacked MoE experts: num_experts = E,
 * one tensor per (layer, projection) holding all experts -- paper, Appendix A,
 * on expert modules).
 *
 * Supported geometry: d in {2, 4, 8}, log2_k in 4 .. 14 (K = 16 ... 16384;
 * the paper's builds run from d2/K16 to d4/K16384, section 1 Notation; the
 * published ones use 8 and 12 bits), group in {64, 128}.  Codebooks of up to
 * 64 KiB (K * d * 2 bytes) are read from LDS, larger ones (d4/K16384,
 * d8/K8192, d8/K16384) from device memory, which is slower (paper section
 * 3.1 on codebooks past threadgroup memory).
 * Shape rules (else VQ_ERR_SHAPE): rows >= 1; cols >= 1; cols % group == 0;
 * group % d == 0; (cols / d) % 32 == 0 (rows hold whole 32-code blocks, so
 * no row needs padding); num_experts >= 1; codebook_per_expert in {0, 1};
 * codebook_elems == E_cb * K * d with E_cb = num_experts if
 * codebook_per_expert else 1.  A codebook sliced across devices or views has
 * the wrong length and is refused rather than read out of bounds (model card
 * "Qwen3.8-27B-VQ-4.5bpw", Multi-machine note: codebooks must be replicated,
 * never sliced, and a sliced one must fail loudly).
 * Buffer lengths (else VQ_ERR_SHAPE): code_words == E * rows * Wr and
 * scale_elems == E * rows * (cols / group), so codes packed for another
 * geometry or a short buffer are refused instead of read past their end.
 * Alignment (else VQ_ERR_ALIGN): codes 16 bytes; codebook 16 bytes; scales 4
 * bytes.  Size limit (else VQ_ERR_SHAPE): one expert's codes and its scales
 * each fit in 2 GiB - 1 bytes (the kernels address them with 32-bit offsets).
 */
typedef struct vq_tensor {
  const uint32_t *codes;    /* device [E][rows][Wr] packed codes                 */
  const uint16_t *codebook; /* device [E_cb][K][d] fp16 bits, entry-major        */
  const uint16_t *scales;   /* device [E][rows][cols/group] fp16 bits            */
  int32_t rows;             /* output features per expert                        */
  int32_t cols;             /* input features                                    */
  int32_t d;                /* subvector length: 2, 4 or 8                       */
  int32_t log2_k;           /* bits per code B: 4 .. 14 (K = 2^B)                */
  int32_t group;            /* weights per scale along a row: 64 or 128          */
  int32_t num_experts;      /* E; 1 for a dense tensor                           */
  int32_t codebook_per_expert; /* 0: one codebook for the tensor; 1: one per expert */
  int64_t codebook_elems;   /* number of fp16 values behind `codebook`           */
  int64_t code_words;       /* number of uint32 words behind `codes`             */
  int64_t scale_elems;      /* number of fp16 values behind `scales`             */
} vq_tensor;

/*
 * Input/output types and fused output steps of one call (the *_ex entry
 * points; the plain entry points are x fp16, y fp32, no epilogue).
 *
 *   x_dtype: VQ_DTYPE_F16 or VQ_DTYPE_BF16 (bit patterns).  The runtime the
 *     paper scores takes and returns bf16 (paper, §7 Reproducibility: the v2
 *     profile).  bf16 x is converted to fp16 as it is staged (round to nearest
 *     even): exact for 2^-17 <= |x| <= 65504 and for 0; smaller magnitudes
 *     lose low bits (at most 2^-25 absolutely), larger ones become +-inf.
 *   y_dtype: VQ_DTYPE_F32, VQ_DTYPE_F16 or VQ_DTYPE_BF16: the fp32 results
 *     (or the SwiGLU value below) rounded to nearest even on the final store.
 *   epilogue:
 *     VQ_EPILOGUE_NONE    y = x W^T as for the plain calls.
 *     VQ_EPILOGUE_SWIGLU  the gate and up projections of an MLP stored as one
 *       tensor of 2I interleaved rows (row 2i = gate row i, row 2i + 1 = up
 *       row i; rows must be even): y[..][i] = silu(g_i) * u_i with g, u the
 *       fp32 results and silu(g) = g / (1 + exp(-g)); y has rows / 2 values
 *       per token (dense) or per (token, slot) (routed).  The paper (§2.1)
 *       quantizes the MLP trio, the gate, up and down projections; the
 *       activation between them is not stated, and SiLU gating (SwiGLU), that
 *       of the model family the pages quantize, is the reading taken.  Gate
 *       and up share x, so both are read in one pass and the activation
 *       never leaves the kernel.
 *     VQ_EPILOGUE_COMBINE routed calls only: y[t][r] = sum over the slots s
 *       of token t with 0 <= ids[t][s] < E of route_weights[t][s] *
 *       (W_e x_row)[r], the router-weighted top-k combine; y is [T][rows],
 *       y_dtype must be VQ_DTYPE_F32.  The library zeroes y on the stream
 *       first and the slots add into it atomically, so the fp32 addition
 *       order over slots, and with it the last bits, may vary between runs.
 *   route_weights: device [T][top_k] fp32, 4-byte aligned (COMBINE only;
 *     otherwise ignored).
 * Errors (VQ_ERR_SHAPE): an unknown dtype or epilogue; SWIGLU on odd rows;
 * COMBINE on a dense call or with y_dtype != F32; VQ_ERR_NULL / VQ_ERR_ALIGN
 * for route_weights.  The streaming GEMV holds at most 20480 input features
 * per pass over x and adds further slices into an fp32 y, so vq_gemv_ex /
 * vq_moe_gemv_ex with cols > 20480 accept only y_dtype F32 and no SWIGLU.
 * A NULL io means the defaults.
 */
/* E4M3 and E2M1: 8- and 4-bit values with block scales, for the calls that name them. */
typedef enum {
  VQ_DTYPE_F32 = 0,
  VQ_DTYPE_F16 = 1,
  VQ_DTYPE_BF16 = 2,
  VQ_DTYPE_E4M3 = 3,
  VQ_DTYPE_E2M1 = 4
} vq_dtype;
typedef enum { VQ_EPILOGUE_NONE = 0, VQ_EPILOGUE_SWIGLU = 1, VQ_EPILOGUE_COMBINE = 2 } vq_epilogue;

typedef struct vq_io {
  int32_t x_dtype;             /* vq_dtype: F16 (default) or BF16                  */
  int32_t y_dtype;             /* vq_dtype: F32 (default), F16 or BF16             */
  int32_t epilogue;            /* vq_epilogue                                     */
  int32_t reserved;            /* must be 0                                       */
  const float *route_weights;  /* COMBINE: device [T][top_k] fp32 router weights  */
} vq_io;

/* uint32 words per row of packed codes: ceil(cols/d/32) * log2_k -- each row
 * holds its codes in row-local blocks of 32 codes packed LSB-first into
 * log2_k words (model card "Qwen3.5-397B-A17B-VQ-2.4bpw", Methodology, on the
 * packed index format; paper §2.3 Packing: codes stored at their true bit
 * width).  Returns -1 for a non-positive cols or an unsupported d / log2_k. */
int32_t vq_words_per_row(int32_t cols, int32_t d, int32_t log2_k);

/*
 * Dequantize expert `expert` of `w` to fp16: w_out[r][c] = W[r][c], exactly as
 * defined above (bit-exact).  Used to check the unpack/gather/scale step on
 * its own (397B card and paper §3.4: kernels are accepted on bit-identity
 * with a reference path).  w_out: device [rows][cols] uint16, 16-byte aligned.
 * expert outside [0, num_experts) -> VQ_ERR_SHAPE.
 */
vq_status vq_dequant(const vq_tensor *w, int32_t expert, uint16_t *w_out, void *stream);

/*
 * Decode-shaped product y = x W^T for a dense tensor (num_experts == 1):
 *   x: device [T][cols] fp16 bits, 16-byte aligned;
 *   y: device [T][rows] fp32, 16-byte aligned.
 * A stack of E experts (num_experts = E > 1) multiplies every expert by the
 * same x in one launch, y [T][E][rows] (y[t][e] = W_e x[t]), as vq_gemm
 * describes: an MLP's gate and up for a few decode tokens.
 * T >= 0 (T == 0 enqueues nothing).  Any T is accepted.  The streaming
 * kernel reads every code once per token slice: the fast path for small T
 * (the fused decode-and-matmul of paper §3.4; two tokens: a two-token
 * speculative verify step, 35B card, Experimental MTP).  On matrices of at
 * least 16 rows per compute unit, 2 to 4 tokens (up to 16 when y is plain
 * fp32: 160 / its one-pass column slices, d = 2: 640 columns, d = 4: 768,
 * d = 8: 512) run on its matrix-core variant, whose partial sums of long
 * rows' column slices (and, above four tokens, of every item) are added
 * atomically into y, zeroed first: those outputs may differ in the last
 * bits from run to run.  Above a token count measured per shape (that cap
 * there; otherwise 2 for d = 2/4 matrices, 4 for d = 8, 6 for matrices of
 * at most 16M weights) vq_gemv runs the MFMA kernel of vq_gemm instead,
 * with the same result contract.
 */
vq_status vq_gemv(const vq_tensor *w, const uint16_t *x, int32_t T, float *y, void *stream);

/*
 * Prefill-shaped product, same arguments and result as vq_gemv: dequantized
 * weight tiles feed fp16 MFMA instructions with fp32 accumulation.  Any T is
 * accepted; it is the fast path for large T (paper §2.5: scoring runs a
 * prefill-shaped path; §3.4 prefill).  Tiles of 32 or 128 tokens, whichever
 * a time model of the call rates faster.  When the output tiles do not fill
 * whole rounds of the GPU's compute units, the tiles of the last, partial
 * round may be split along the columns and their partial sums added
 * atomically into y (zeroed first on the same stream): those outputs may
 * differ in the last bits from run to run (fp32 addition order), within the
 * stated tolerance; all others are deterministic.  The environment variable
 * VQMI_GEMM_TILE = 32 or 128 forces the tile shape (for tests).
 * A stack of E experts (num_experts = E > 1; codebook_per_expert = 1 keeps
 * each tensor's own codebook) multiplies every expert by the same x: y is
 * [T][E][rows] (rows / 2 under SWIGLU), y[t][e] = W_e x[t], each expert's
 * rows computed exactly as a call on that expert alone with the same tile
 * shape and split.  This runs an MLP's gate and up projections, which share
 * their input (paper §2.1: the MLP trio), as one launch whose tiles fill the
 * GPU's rounds together instead of leaving two partial last rounds.  The
 * tile shape and split are chosen for the whole stack, so they (and, for
 * split tiles, the last bits) can differ from separate calls.  T * E at most
 * 2^24.
 */
vq_status vq_gemm(const vq_tensor *w, const uint16_t *x, int32_t T, float *y, void *stream);

/*
 * Routed-expert (top-k MoE) product, decode-shaped: for every token t and
 * slot s, with e = expert_ids[t][s],
 *   y[t][s][:] = W_e x_row  if 0 <= e < num_experts, else zeros,
 * where x_row = x[t] (x_per_slot == 0: gate/up projections, x is [T][cols])
 * or x[t][s] (x_per_slot == 1: down projection, x is [T][top_k][cols]).
 * No router-weight multiply and no combine over slots.  Duplicate ids in a
 * token are computed independently.  (aquaman164 card, Run: fused decode
 * kernels for all expert tiers; Experimental MTP note: decode cost is the
 * routed experts' bytes.)
 *   expert_ids: device [T][top_k] int32, 4-byte aligned;
 *   y: device [T][top_k][rows] fp32, 16-byte aligned;  T >= 0, top_k >= 1,
 *   T * top_k <= 65535 (larger batches belong to vq_moe_gemm), x at most
 *   2 GiB - 1 bytes.
 * Dense projections that share their input (an MLP's gate and up) can be
 * stored as an expert stack (codebook_per_expert = 1 keeps each tensor's own
 * codebook) and run by this call in one launch, with expert_ids {0, 1, ...}
 * in every token: the same results as one vq_gemv per tensor, bit for bit,
 * at one launch's fixed cost.  Routed gate and up projections likewise: with
 * gate_e and up_e stored as experts 2e and 2e + 1 of one stack, expert_ids
 * (2e, 2e + 1) per routed slot and top_k doubled give both outputs of every
 * slot in one launch, bit for bit those of the two separate calls.
 */
vq_status vq_moe_gemv(const vq_tensor *w, const uint16_t *x, int32_t x_per_slot,
                      const int32_t *expert_ids, int32_t T, int32_t top_k, float *y,
                      void *stream);

/*
 * The calls above with the input/output types and epilogue of `io` (see
 * vq_io).  x and y are typeless device pointers whose element types `io`
 * names; shapes and alignment as for the plain calls, y's row length
 * rows / 2 under SWIGLU and y [T][rows] under COMBINE.
 */
vq_status vq_gemv_ex(const vq_tensor *w, const vq_io *io, const void *x, int32_t T, void *y,
                     void *stream);
vq_status vq_gemm_ex(const vq_tensor *w, const vq_io *io, const void *x, int32_t T, void *y,
                     void *stream);
vq_status vq_moe_gemv_ex(const vq_tensor *w, const vq_io *io, const void *x, int32_t x_per_slot,
                         const int32_t *expert_ids, int32_t T, int32_t top_k, void *y, void *stream);

/* Bytes of workspace vq_moe_gemm needs for these sizes (0 if T*top_k == 0);
 * returns 0 and sets the error text for negative or overflowing sizes. */
size_t vq_moe_workspace_bytes(int32_t T, int32_t top_k, int32_t num_experts);

/*
 * Routed-expert product, prefill-shaped: same arguments and result as
 * vq_moe_gemv (paper, Appendix A, on expert modules, and §3.4 on the prefill
 * path; model card "aquaman164/Qwen3.6-35B-A3B-MLX-VQ-2.4bpw", Experimental
 * MTP section, on its top-8 MoE).  On the device, the (token, slot) pairs are
 * counted, scanned and scattered by expert, a grouped MFMA GEMM runs over the
 * flat list of (expert, token tile) work items with gathered x rows, and
 * results are written straight to y[t][s].  No host synchronisation.  Token
 * tiles hold 32 pairs, or 128 for an expert's whole 128s (and a remainder
 * above 64) when the call is large enough to fill the GPU twice over; the two
 * kinds group the columns of the k-steps differently, so a row's fp32 value
 * can differ in the last bits between calls that tile its expert differently
 * (within the stated tolerance; each call is deterministic).
 *   workspace: device, >= vq_moe_workspace_bytes(T, top_k, num_experts)
 *   bytes, 16-byte aligned, owned by the caller; contents on entry are
 *   ignored and on return are undefined.  Concurrent calls need separate
 *   workspaces.
 * The stacked gate/up layouts described for vq_moe_gemv apply here too
 * (workspace sized for the doubled top_k and expert count): each output row
 * depends only on its expert, its x row and its tile kind, so the results are
 * bit for bit those of separate calls, unless only the stacked call (twice
 * the pairs) is large enough for 128-pair tiles.
 */
vq_status vq_moe_gemm(const vq_tensor *w, const uint16_t *x, int32_t x_per_slot,
                      const int32_t *expert_ids, int32_t T, int32_t top_k, float *y,
                      void *workspace, size_t workspace_bytes, void *stream);

/* vq_moe_gemm with the input/output types and epilogue of `io`. */
vq_status vq_moe_gemm_ex(const vq_tensor *w, const vq_io *io, const void *x, int32_t x_per_slot,
                         const int32_t *expert_ids, int32_t T, int32_t top_k, void *y,
                         void *workspace, size_t workspace_bytes, void *stream);

/*
 * vq_moe_gemm for callers that cannot allocate device memory (code under HIP
 * graph capture, tight serving loops, harnesses that forbid hipMalloc): the
 * same arguments and results as vq_moe_gemm, bit for bit, without the
 * workspace.  Its routing scratch is a static device array of 4 MiB inside the
 * library, one per GPU, held until the process ends; calls whose
 * vq_moe_workspace_bytes(T, top_k, num_experts) exceeds 4 MiB return
 * VQ_ERR_WORKSPACE (about 950 thousand (token, slot) pairs for 256 experts).  The
 * scratch of the current device is used: `stream` must belong to it.  Nothing
 * is allocated and the scratch needs no clearing (every call writes what it
 * reads).  All calls on one GPU share that array: calls that overlap in time
 * on one GPU (other streams, other threads) race and give wrong results;
 * calls ordered on one stream are safe.
 */
vq_status vq_moe_gemm_no_alloc(const vq_tensor *w, const uint16_t *x, int32_t x_per_slot,
                               const int32_t *expert_ids, int32_t T, int32_t top_k, float *y,
                               void *stream);

/*
 * The fit that produces a VQ tensor from fp32 weights (paper, §2.2 The fit:
 * d-dimensional subvectors, each group of `group` weights of a row scaled by
 * its maximum absolute value, a K-entry codebook fit by k-means with k-means++
 * initialization on a random subsample and plain Lloyd iterations; §2.3:
 * codes packed to their true bit width; §2.6: relative reconstruction error
 * ||W - W_hat|| / ||W||).  Outputs are the layout of vq_tensor (dense, one
 * codebook), so the result feeds vq_gemv / vq_gemm directly.
 *   w: device [rows][cols] fp32, 16-byte aligned; geometry and shape rules as
 *     for vq_tensor (d, log2_k, group supported; cols % group == 0;
 *     (cols / d) % 32 == 0); rows * cols / d <= 2^30 subvectors;
 *   sample_idx: device [n_sample] int32, the subvectors (row-major order)
 *     k-means++ draws from, 1 <= n_sample <= 2^24 (an index outside the
 *     subvector range is reduced modulo their count);
 *   uniforms: device [K] fp64 in [0, 1): the draws of k-means++ (the first
 *     centre is sample point floor(u_0 * n_sample));
 *   iters >= 0 Lloyd iterations (a converged iteration changes nothing);
 *   codes: device [rows][Wr] uint32, 16-byte aligned; codebook: device [K][d]
 *   fp16, 16-byte aligned; scales: device [rows][cols/group] fp16, 4-byte
 *   aligned; relerr: device, one fp64;
 *   workspace: device, >= vq_encode_workspace_bytes(...) bytes, 256-byte
 *   aligned, owned by the caller (about rows * cols * 8 bytes).
 * The random numbers are inputs, so a fit is reproducible: its arithmetic is
 * fixed (fp32 squared distances summed in coordinate order without fused
 * multiply-add, ties to the lowest centroid; k-means++ draws and Lloyd means
 * from exact integer sums of values in units of 2^-32), and codes, codebook
 * and scales are the same bits on every run.
 */
size_t vq_encode_workspace_bytes(int32_t rows, int32_t cols, int32_t d, int32_t log2_k, int32_t n_sample);
vq_status vq_encode(const float *w, int32_t rows, int32_t cols, int32_t d, int32_t log2_k, int32_t group,
                    const int32_t *sample_idx, int32_t n_sample, const double *uniforms, int32_t iters,
                    uint32_t *codes, uint16_t *codebook, uint16_t *scales, double *relerr, void *workspace,
                    size_t workspace_bytes, void *stream);

/*
 * Routing to experts: the expert ids and route weights that vq_moe_gemv and
 * vq_moe_gemm (VQ_EPILOGUE_COMBINE) take, from a router's logits.  Per token,
 * with logits l_e:
 *   score   VQ_SCORE_SOFTMAX p_e = exp(l_e) / sum over the experts in play, or
 *           VQ_SCORE_SIGMOID p_e = 1 / (1 + exp(-l_e)).
 *   in play an expert whose logit (and bias, if given) is neither NaN nor
 *           -inf; an infinite logit counts as the largest finite fp32 value.
 *           Logits of a type's lowest finite value are ordinary values.
 *   key     l_e without a bias (the order of the scores), p_e + bias[e] with
 *           one (a balance bias moves the choice, never the weights).
 *   groups  of num_experts / groups consecutive experts; a group's score is
 *           its largest key (VQ_GROUP_MAX) or the sum of its two largest
 *           (VQ_GROUP_TOP2; of p_e without a bias; of one where only one is in
 *           play).  The best top_groups groups stay, ties to the lowest
 *           group; groups without an expert in play never stay.  groups = 1:
 *           no group step (top_groups must be 1).
 *   choice  the top_k largest keys left, in descending order, ties to the
 *           lowest expert; slots nothing is left for get id -1 (skipped by
 *           the routed products) and weight 0.  Scores are compared in 64
 *           bits where they decide the choice.
 *   weight  scale * p_e, with renormalize scale * p_e / (sum of the chosen
 *           p_e; 0 where that sum is 0), in fp32.  A p_e that is 0 in 64 bits
 *           (a sigmoid of l_e < -709.78, a softmax 745 below its largest
 *           logit) counts as 0.
 * logits: device [T][num_experts] of logits_dtype (vq_dtype), aligned to
 * their element; expert_ids: device [T][top_k] int32 and route_weights:
 * device [T][top_k] fp32, 4-byte aligned; bias: device [num_experts] fp32,
 * 4-byte aligned, or NULL.  T >= 0 (0 enqueues nothing).  One launch, no
 * workspace; the same inputs give the same bits.
 * Errors (VQ_ERR_SHAPE): num_experts outside [1, 1024]; top_k outside [1, 64]
 * or above top_groups * num_experts / groups; groups outside [1, 64] or not a
 * divisor of num_experts; top_groups outside [1, groups]; an unknown score,
 * group_score or logits_dtype; renormalize not 0 or 1; a scale that is not
 * finite; reserved not 0; T above 2^25.
 */
typedef enum { VQ_SCORE_SOFTMAX = 0, VQ_SCORE_SIGMOID = 1 } vq_score;
typedef enum { VQ_GROUP_MAX = 0, VQ_GROUP_TOP2 = 1 } vq_group_score;

typedef struct vq_router {
  int32_t num_experts;  /* E                                                      */
  int32_t top_k;        /* slots per token                                        */
  int32_t score;        /* vq_score                                               */
  int32_t logits_dtype; /* vq_dtype                                               */
  int32_t groups;       /* 1: none                                                */
  int32_t top_groups;   /* groups that stay                                       */
  int32_t group_score;  /* vq_group_score                                         */
  int32_t renormalize;  /* 0 or 1                                                 */
  float scale;          /* factor of every weight                                 */
  int32_t reserved;     /* must be 0                                              */
  const float *bias;    /* device [E] fp32, or NULL                               */
} vq_router;

vq_status vq_moe_route(const vq_router *r, const void *logits, int32_t T, int32_t *expert_ids,
                       float *route_weights, void *stream);

/*
 * Tensors in 8-bit floating point with a scale for each block of 128, for the
 * parts of a model that are not vector-quantized (shared experts, projections
 * kept in 8 bits): values are OCP e4m3 (largest 448, no infinities, codes
 * 0x7f and 0xff NaN), a value stands for code * scale.
 *
 * A weight: values [rows][cols], one fp32 scale for each 128 x 128 block (the
 * last block of rows or columns may be partial).  rows >= 1; cols a positive
 * multiple of 16, at most 2^20 (else VQ_ERR_SHAPE).  value_bytes == rows *
 * cols and scale_elems == ceil(rows/128) * ceil(cols/128), so a short or
 * sliced buffer is refused.  values 16-byte, scales 4-byte aligned.
 * Activations: x [T][cols] with x_scales [T][ceil(cols/128)], one scale for a
 * token's 128 columns, as vq_fp8_quant and vq_norm leave them.
 */
typedef struct vq_fp8_tensor {
  const uint8_t *values; /* device [rows][cols] e4m3                             */
  const float *scales;   /* device [ceil(rows/128)][ceil(cols/128)] fp32         */
  int32_t rows;          /* output features                                     */
  int32_t cols;          /* input features                                      */
  int64_t value_bytes;   /* number of bytes behind `values`                      */
  int64_t scale_elems;   /* number of fp32 values behind `scales`                */
} vq_fp8_tensor;

/*
 * Quantize activations: for each token and 128 columns,
 *   scale = max |x| / 448 rounded to fp32 (1 where that is 0),
 *   q = the e4m3 value nearest to x / scale (ties to even; exact, no double
 *       rounding), at most 448 in magnitude.
 * NaN and infinite x become NaN codes and do not count for the scale, so they
 * spoil only their own token's results.
 *   x: device [T][cols] of x_dtype (F16 or BF16), 16-byte aligned;
 *   q: device [T][cols] e4m3, 16-byte aligned; scales: device
 *   [T][ceil(cols/128)] fp32, 4-byte aligned.  cols as for vq_fp8_tensor;
 *   T >= 0 (0 enqueues nothing), T * ceil(cols/128) <= 2^28 - 16.
 */
vq_status vq_fp8_quant(const void *x, int32_t x_dtype, int32_t T, int32_t cols, uint8_t *q, float *scales,
                       void *stream);

/*
 * Product of e4m3 activations with an e4m3 weight:
 *   y[t][r] = sum_b x_scales[t][b] * scales[r / 128][b] *
 *             sum over the 128 columns of block b of x[t][c] * w[r][c],
 * exact products (the fp16 matrix instructions hold them), all sums in fp32,
 * rounded to y's type once.  Any T: decode and prefill shapes run different
 * kernels, and few output tiles are split along the columns into planes of
 * the workspace and joined in order, as a time model of the call rates best.
 * The same call gives the same bits every time; the order of the fp32 sums,
 * and with it a row's last bits, depends on T.  The environment variable
 * VQMI_FP8_PLAN = "kernel,splits" forces the choice (for tests).
 *   io: y_dtype and epilogue (NONE or SWIGLU on interleaved gate/up rows: y
 *     has rows / 2 values per token) as for vq_gemm_ex; x_dtype must be
 *     VQ_DTYPE_E4M3.  NULL: fp32 y, no epilogue.
 *   x: device [T][cols] e4m3, 16-byte aligned; x_scales: device
 *     [T][ceil(cols/128)] fp32, 4-byte aligned; y: device, 16-byte aligned.
 *   workspace: device, >= vq_fp8_workspace_bytes(rows, cols, T) bytes (enough
 *     for both calls, any y type and epilogue), 16-byte aligned, owned by the caller (may be NULL where that is 0); contents on
 *     entry are ignored and on return are undefined.  Calls that overlap in
 *     time need separate workspaces.
 * T >= 0 (0 enqueues nothing), T <= 2^24, rows <= 2^24, and a launch holds
 * ceil(rows/256) * ceil(T/128) < 2^22 tiles (more: VQ_ERR_SHAPE).
 *
 * vq_fp8_gemm_fast: the same call for a 16-bit y (io with y_dtype F16 or BF16;
 * VQ_ERR_SHAPE otherwise) that may use the e4m3 matrix instructions, which do
 * twice the operations a second.  They cut every product of eight consecutive
 * columns (8j to 8j + 7) 13 bits below the leading bit of the eight's largest
 * product, so that y[t][r] is off by up to
 *   sum_b x_scales[t][b] * scales[r / 128][b] *
 *   sum over the eights of block b of 7 * 2^-13 * max |x[t][c] * w[r][c]|
 * more than vq_fp8_gemm's: 1.6e-5 of y's norm on normal inputs, but without a
 * limit relative to an output whose large products cancel.  Whether a call
 * uses them depends on T, rows and cols (a few tokens or rows are summed
 * exactly), so a token's accuracy depends on the batch it is in.
 */
size_t vq_fp8_workspace_bytes(int32_t rows, int32_t cols, int32_t T);
vq_status vq_fp8_gemm(const vq_fp8_tensor *w, const vq_io *io, const uint8_t *x, const float *x_scales, int32_t T,
                      void *y, void *workspace, size_t workspace_bytes, void *stream);
vq_status vq_fp8_gemm_fast(const vq_fp8_tensor *w, const vq_io *io, const uint8_t *x, const float *x_scales,
                           int32_t T, void *y, void *workspace, size_t workspace_bytes, void *stream);

/*
 * Tensors in microscaled 4-bit floating point: OCP e2m1 values (0, 0.5, 1, 1.5,
 * 2, 3, 4, 6 and their negatives: codes 0 to 7, plus 8 for the sign; no
 * infinities, no NaN) with an e8m0 scale for each 32 columns (byte b stands for
 * 2^(b - 127), 255 for NaN).  A value stands for code * scale, a block whose
 * scale is 255 for NaN throughout.  Values of 2^128 and above, which fp32 does
 * not hold (4 and 6 under byte 253, 2 and above under 254; vq_mx4_quant leaves
 * at most 252), are infinite to vq_mx4_dequant, and in a weight make products
 * with 16-bit activations, vq_mx4_moe's included, infinite or NaN; products
 * with 4-bit activations take them as they are.
 *
 * One tensor or a stack of experts: values [E][rows][cols/2], two codes a byte,
 * the even column in the low half; scales [E][rows][cols/32].  rows >= 1; cols
 * a positive multiple of 32, at most 2^20; num_experts >= 1 (else
 * VQ_ERR_SHAPE).  value_bytes == E * rows * cols / 2 and scale_bytes == E *
 * rows * cols / 32, so a short or sliced buffer is refused.  values 16-byte
 * aligned; scales anywhere.
 * Activations: x [T][cols/2] with x_scales [T][cols/32], as vq_mx4_quant leaves
 * them.
 */
typedef struct vq_mx4_tensor {
  const uint8_t *values; /* device [E][rows][cols/2]                             */
  const uint8_t *scales; /* device [E][rows][cols/32]                            */
  int32_t rows;          /* output features per expert                           */
  int32_t cols;          /* input features                                       */
  int32_t num_experts;   /* E; 1 for a single tensor                             */
  int32_t reserved;      /* must be 0                                            */
  int64_t value_bytes;   /* number of bytes behind `values`                      */
  int64_t scale_bytes;   /* number of bytes behind `scales`                      */
} vq_mx4_tensor;

/*
 * Quantize x [T][cols] (activations, or the rows of a weight): for each row and
 * 32 columns, with m = max |x|,
 *   scale = 2^k, k = floor(log2(m)) - 2, at least -127; 1 where m is 0;
 *   q = the e2m1 value nearest to x / scale (ties to the even code; exact), at
 *       most 6 in magnitude (values above 6 * scale, where m is above it, stop
 *       there); the sign of zeros is kept.
 * A block that holds a NaN or an infinity gets the scale 255 and codes 0.
 *   x: device [T][cols] of x_dtype (F32, F16 or BF16), 16-byte aligned;
 *   q: device [T][cols/2], 16-byte aligned; scales: device [T][cols/32] bytes.
 *   cols as for vq_mx4_tensor; T >= 0 (0 enqueues nothing), T * cols <= 2^34.
 *
 * vq_mx4_dequant: y[t][c] = code * scale, rounded to y_dtype (F32, F16 or BF16)
 * once: exact in fp32 and bf16 below 2^128, and in fp16 where that can hold it
 * (larger ones become infinite, smaller ones round).  y: device [T][cols], 16-byte aligned.
 */
vq_status vq_mx4_quant(const void *x, int32_t x_dtype, int32_t T, int32_t cols, uint8_t *q, uint8_t *scales,
                       void *stream);
vq_status vq_mx4_dequant(const uint8_t *q, const uint8_t *scales, int32_t T, int32_t cols, int32_t y_dtype, void *y,
                         void *stream);

/*
 * Product with a 4-bit weight (num_experts == 1), y = x W^T:
 *   io->x_dtype VQ_DTYPE_E2M1: x [T][cols/2] with x_scales [T][cols/32];
 *   io->x_dtype F16 or BF16: x [T][cols], x_scales NULL.
 * Products are exact, sums are in fp32 (4-bit x: the 32 products of a block sum
 * exactly; sums below 2^-126 lose bits), y is rounded to its type once.  Any T:
 * decode and prefill shapes run different kernels, and few output tiles may be
 * split along the columns into planes of the workspace and joined in order, as
 * a time model of the call rates best.  The same call gives the same bits every
 * time; the order of the sums, and with it a row's last bits, depends on T.
 * The environment variable VQMI_MX4_PLAN = "kernel,splits" forces the choice
 * (for tests).
 *   io: y_dtype F32, F16 or BF16, epilogue NONE or SWIGLU (interleaved gate/up
 *     rows: y has rows / 2 values per token) as for vq_gemm_ex.  NULL: 4-bit x,
 *     fp32 y, no epilogue.
 *   x, y: device, 16-byte aligned; x_scales: device, any alignment.
 *   workspace: device, >= vq_mx4_workspace_bytes(rows, cols, T) bytes (enough
 *     for every x and y type and epilogue), 16-byte aligned, owned by the
 *     caller (may be NULL where that is 0); contents on entry are ignored and
 *     on return are undefined.  Calls that overlap in time need separate
 *     workspaces.
 * T >= 0 (0 enqueues nothing), T <= 2^24, rows <= 2^24, ceil(rows/16) *
 * ceil(T/16) <= 2^30, and the call has to fit a launch (else VQ_ERR_SHAPE).
 */
size_t vq_mx4_workspace_bytes(int32_t rows, int32_t cols, int32_t T);
vq_status vq_mx4_gemm(const vq_mx4_tensor *w, const vq_io *io, const void *x, const uint8_t *x_scales, int32_t T,
                      void *y, void *workspace, size_t workspace_bytes, void *stream);

/*
 * A whole mixture-of-experts layer for a few tokens over stacks of 4-bit
 * experts, from the router's logits to the weighted sum:
 *   ids, weights = vq_moe_route(r, logits)
 *   g, u = rows 2i and 2i + 1 of W_gate_up[e] x[t],  e = ids[t][s]
 *   h[t][s][i] = silu(g) * u, kept in fp32
 *   y[t] = sum over the slots s with ids[t][s] >= 0 of weights[t][s] *
 *          W_down[e] h[t][s]
 * Products are exact, sums are in fp32, y is rounded to its type once.  A token
 * without an expert gets zeros.  The call is for decode batches: gate and up
 * rows of an expert are read once for 2 to 8 of its tokens, down rows for 4, or
 * (a token or a few that share little) once for every token and slot.  A
 * token's slots are added in their order, on the latter path those 8 apart
 * first, then these sums in order.  The same call gives the same bits every
 * time; a token's last bits depend on the batch.
 *   r: as for vq_moe_route, with num_experts those of both stacks;
 *   gate_up: [E][2 * inter][hidden], interleaved gate and up rows; down:
 *   [E][hidden][inter];
 *   io: x_dtype F16 (default) or BF16, y_dtype F32 (default), F16 or BF16;
 *   epilogue NONE;
 *   logits: device [T][E] of r->logits_dtype, aligned to their element;
 *   x: device [T][hidden], y: device [T][hidden], 16-byte aligned;
 *   expert_ids: device [T][top_k] int32, route_weights: device [T][top_k]
 *   fp32, 4-byte aligned: outputs, as vq_moe_route leaves them;
 *   workspace: device, >= vq_mx4_moe_workspace_bytes(T, top_k, hidden, inter)
 *   bytes, 16-byte aligned, as for vq_mx4_gemm.
 * 0 <= T <= 64 (0 enqueues nothing), T * top_k <= 1024, and T * top_k * hidden
 * and T * top_k * inter <= 2^26 (else VQ_ERR_SHAPE; larger batches belong to
 * vq_moe_route and products of their own).
 */
size_t vq_mx4_moe_workspace_bytes(int32_t T, int32_t top_k, int32_t hidden, int32_t inter);
vq_status vq_mx4_moe(const vq_router *r, const vq_mx4_tensor *gate_up, const vq_mx4_tensor *down, const vq_io *io,
                     const void *logits, const void *x, int32_t T, void *y, int32_t *expert_ids, float *route_weights,
                     void *workspace, size_t workspace_bytes, void *stream);

/*
 * The norms before and after a block, fused with its gate and the scaled
 * residual sum: what stands between one block's products and the next one's.
 *   u = block * rsqrt(mean(block^2) + eps) * (post_weight + weight_offset),
 *       or block itself where post_weight is NULL;
 *   v = beta * residual + alpha * act(gate) * u;
 *   h = v * rsqrt(mean(v^2) + eps) * (pre_weight + weight_offset), or with a
 *       factor of 1 where pre_weight is NULL.
 * Means over a token's cols values.  All arithmetic in fp32; v and h are
 * rounded once, on their stores (h comes from the unrounded v).
 *   block:    device [T][cols] of block_dtype (the products' y: F32, F16 or
 *             BF16), or NULL: v = beta * residual (a plain norm).  Post norm
 *             and gate need a block.
 *   residual: device [T][cols] of residual_dtype (F32, F16 or BF16), or NULL:
 *             no residual term.  Not both NULL.
 *   gate:     VQ_GATE_NONE (1), VQ_GATE_CHANNEL gate_values [cols],
 *             VQ_GATE_TOKEN [T], VQ_GATE_FULL [T][cols]; gate_act
 *             VQ_ACT_NONE, VQ_ACT_SIGMOID or VQ_ACT_TANH is applied to them.
 *   post_weight, pre_weight: device [cols]; like gate_values of weight_dtype.
 *   residual_out: device [T][cols] of residual_dtype, v; may be `residual`
 *             itself; NULL: not stored.
 *   h:        device [T][cols] of h_dtype (F32, F16, BF16: the VQ products' x;
 *             E4M3: vq_fp8_gemm's, quantized as vq_fp8_quant does, with
 *             h_scales [T][ceil(cols/128)] fp32); NULL: not computed.  Not
 *             both outputs NULL.  No other buffers may overlap.
 * Pointers of [T][cols] and [cols] data 16-byte aligned, the others to their
 * element.  T >= 0 (0 enqueues nothing), T * ceil(cols/512) <= 2^26 - 4.
 * One launch, no workspace; the same inputs give the same bits.
 * Errors (VQ_ERR_SHAPE): cols outside [1, 32768], or not a multiple of 16 for
 * an E4M3 h; an unknown dtype, gate or gate_act; a gate_act without a gate; a
 * post norm or gate without a block; eps negative or not finite; alpha, beta
 * or weight_offset not finite; reserved not 0.
 */
typedef enum { VQ_GATE_NONE = 0, VQ_GATE_CHANNEL = 1, VQ_GATE_TOKEN = 2, VQ_GATE_FULL = 3 } vq_gate;
typedef enum { VQ_ACT_NONE = 0, VQ_ACT_SIGMOID = 1, VQ_ACT_TANH = 2 } vq_act;

typedef struct vq_norm_spec {
  int32_t cols;
  int32_t block_dtype;     /* vq_dtype                                           */
  int32_t residual_dtype;  /* vq_dtype                                           */
  int32_t weight_dtype;    /* vq_dtype of the weights and the gate               */
  int32_t h_dtype;         /* vq_dtype                                           */
  int32_t gate;            /* vq_gate                                            */
  int32_t gate_act;        /* vq_act                                             */
  int32_t reserved;        /* must be 0                                          */
  float alpha, beta, eps, weight_offset;
  const void *post_weight; /* device [cols], or NULL                             */
  const void *pre_weight;  /* device [cols], or NULL                             */
  const void *gate_values; /* device, see gate                                   */
} vq_norm_spec;

vq_status vq_norm(const vq_norm_spec *n, const void *block, const void *residual, int32_t T, void *residual_out,
                  void *h, float *h_scales, void *stream);

/* Text for the last non-OK status returned on this thread ("" if none). */
const char *vq_last_error(void);

/* Name of a status code ("VQ_OK", "VQ_ERR_SHAPE", ...). */
const char *vq_status_name(vq_status s);

#ifdef __cplusplus
}
#endif

#endif /* VQMI_VQ_H */
