/*
 * mole.h -- C ABI of libmole, the B200 (sm_100a) implementation of the
 * Mixture-of-Lookup-Experts (MoLE) inference lookup path.
 *
 * Source page ("MoLE page"): "ICML 2025 Spotlight | 华为诺亚提出端侧大模型新架构MoLE，
 * 内存搬运代价降低1000倍" (zejuncao.github.io, 2025-05-07).  The page states the
 * method in prose only (its formulas and figures were lost); the readings this
 * library takes are stated at each entry point.
 *
 * Conventions for every entry point:
 *   - Tensor pointers are DEVICE pointers owned by the caller, row-major and
 *     contiguous.  The library never frees or retains them.
 *   - Work is enqueued asynchronously on `stream` (0 = legacy default stream).
 *     Argument errors are detected on the host and returned synchronously;
 *     nothing is launched then.
 *   - Errors detected on the device (a token id outside [0, V), a wait that ran
 *     out of time) set a per-device error word; `mole_check` reads and clears
 *     it.  A token with a bad id gets a NaN output row.
 *   - The library allocates no device memory of its own apart from static
 *     per-device variables (the error word, and the fixed scratch array of
 *     mole_build_lut_noalloc).  Scratch memory, where the other entry points
 *     need it, is passed in by the caller.
 *   - bf16 tensors are IEEE bfloat16 bit patterns; fp16 scales are IEEE binary16.
 */
#ifndef MOLE_H_
#define MOLE_H_

#include <stddef.h>
#include <stdint.h>
#include <cuda_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  MOLE_OK = 0,
  MOLE_ERR_ARG = 1,          /* bad pointer, size or enum value */
  MOLE_ERR_ALIGN = 2,        /* a pointer is not 16-byte aligned where required */
  MOLE_ERR_UNSUPPORTED = 3,  /* valid but unsupported shape (see each call) */
  MOLE_ERR_WORKSPACE = 4,    /* scratch buffer missing or too small */
  MOLE_ERR_INDEX = 5,        /* (mole_check) a token id was outside [0, V) */
  MOLE_ERR_CUDA = 6,         /* a CUDA runtime/driver call failed */
  MOLE_ERR_TIMEOUT = 7,      /* (mole_check) host wait or device wait ran out */
  MOLE_ERR_NO_DEVICE = 8     /* no sm_100 device current */
} mole_status;

typedef enum { MOLE_F32 = 0, MOLE_BF16 = 1 } mole_dtype;

typedef enum {
  MOLE_ACT_GELU_ERF = 0,   /* x * Phi(x) (default reading of "GELU FFN") */
  MOLE_ACT_GELU_TANH = 1,  /* tanh approximation of GELU */
  MOLE_ACT_RELU = 2,
  MOLE_ACT_SILU = 3,
  MOLE_ACT_IDENTITY = 4
} mole_act;

/* Human-readable name of a status code (static storage). */
const char* mole_status_str(mole_status s);

/* Library version, major * 10000 + minor * 100 + patch. */
int mole_version(void);

/*
 * ---- Reparameterisation: build the lookup table (MoLE page, 推理阶段) ----
 *
 * Feeds the embedding matrix to every routed expert:
 *     LUT[v, j, :] = f_j(E[v, :]),   f_j(x) = act(x . W1[j]) . W2[j]
 * (expert form and activation are this library's reading; the page prints no
 * formula).  All routed experts are evaluated; the experts can be dropped
 * afterwards.
 *
 *   embed : [V, D]       dt
 *   W1    : [N, D, Dr]   dt
 *   W2    : [N, Dr, D]   dt
 *   lut   : [V, N, D]    dt  (output; token v's N rows are contiguous)
 *   workspace: scratch for the expert hidden activations H = act(E . W1[j]);
 *     at least mole_build_lut_workspace(...) bytes for one expert at a time,
 *     more lets several experts run per launch (up to all N).  Contents on
 *     return are unspecified.
 * dt == MOLE_BF16: bf16 in, fp32 accumulate on the tcgen05 tensor cores, H
 *   rounded to bf16, bf16 out.  Tensor-core path needs D % 64 == 0 and
 *   Dr % 64 == 0 and 16-byte aligned pointers; other shapes use a CUDA-core path.
 * dt == MOLE_F32: fp32 throughout on CUDA cores.
 * Returns MOLE_ERR_WORKSPACE if ws_bytes is below the one-expert minimum.
 */
size_t mole_build_lut_workspace(int64_t V, int64_t D, int32_t N, int64_t Dr, mole_dtype dt,
                                int32_t experts_per_launch);
mole_status mole_build_lut(const void* embed, const void* W1, const void* W2, int64_t V,
                           int64_t D, int32_t N, int64_t Dr, mole_act act, mole_dtype dt,
                           void* lut, void* workspace, size_t ws_bytes, cudaStream_t stream);

/*
 * mole_build_lut without caller-provided scratch, for callers that cannot
 * allocate device memory when they build a table: serving loops that allow no
 * device allocation after start-up (their memory footprint is fixed up
 * front), and plugin hosts that own all device memory and give plugins no
 * allocator.  The MoLE page has no counterpart; it is an interface
 * convenience.
 *
 * Same arguments, layouts and results as mole_build_lut, minus the workspace:
 * the hidden activations of each group of experts live in a fixed 16 MiB array
 * in this library's device memory (held by every GPU that loads the library
 * until the process exits).  One expert's activations, V * Dr * (2 bytes for
 * bf16, 4 for fp32), must fit in it, else MOLE_ERR_WORKSPACE and nothing is
 * launched; experts are built in groups of as many as fit.  The first call on
 * each device looks the array's device address up (cudaGetSymbolAddress, with
 * that device current), and looks it up again after the device's context has
 * changed (a device reset); make that first call before any stream capture.
 * Every call uses the same array, which keeps the last call's contents: calls
 * that overlap on the GPU (other streams, other threads) race on it.  The
 * array needs no clearing between calls (each expert's activations are
 * written before they are read).  No device memory is allocated or freed.
 */
mole_status mole_build_lut_noalloc(const void* embed, const void* W1, const void* W2, int64_t V,
                                   int64_t D, int32_t N, int64_t Dr, mole_act act, mole_dtype dt,
                                   void* lut, cudaStream_t stream);

/*
 * ---- Lookup-combine (MoLE page, 训练阶段 + 推理阶段) ----
 *
 * For each token t (router on the hidden state, all N routed experts active,
 * rows fetched by direct addressing on the token id):
 *     z_j = sum_d h[t, d] Wr[d, j]          (fp32 accumulate)
 *     g   = softmax(z)                        (max-subtracted, fp32)
 *     out[t, :] = sum_j g_j LUT[ids[t], j, :]  (fp32 accumulate)
 * Only the routed-expert mixture is produced; shared experts and the residual
 * are the caller's.
 *
 *   ids : [T] int32 in [0, V)    h : [T, D] dt    Wr : [D, N] dt
 *   lut : [V, N, D] dt           out : [T, D] fp32 (overwritten)
 * dt == MOLE_BF16 needs D % 16 == 0, N <= 32 and 16-byte aligned h, lut, out.
 * dt == MOLE_F32 needs D % 4 == 0, N <= 32 and 16-byte aligned h, lut, out.
 * T == 0 is a no-op.  A token with ids[t] outside [0, V) gets a NaN row and
 * sets the device error word (MOLE_ERR_INDEX from mole_check).
 */
mole_status mole_lookup_combine(const int32_t* ids, int64_t T, const void* h, const void* Wr,
                                const void* lut, int64_t V, int32_t N, int64_t D,
                                mole_dtype dt, float* out, cudaStream_t stream);

/*
 * ---- Token groups: the combine with each distinct row block read once ----
 * (MoLE page, 复杂度分析: a token's traffic is its N expert-output rows; a batch
 * that repeats an id needs that id's rows only once.  推理阶段: every MoLE
 * layer indexes its table with the same input token ids, so one grouping of
 * the batch serves all layers.)
 *
 * mole_token_groups_build groups the batch's tokens by id into `groups`, a
 * caller-owned device buffer of at least mole_token_groups_workspace(T, N)
 * bytes, 16-byte aligned (N = the experts of the layers it will serve).  Its
 * contents are opaque; the grouping stays valid until the buffer is rebuilt.
 * Ids outside [0, V) are left out of every group and set the device error
 * word (MOLE_ERR_INDEX).  One cooperative kernel launch (all of its CTAs
 * resident at once), then one plain launch that lists each SM's share of the
 * work for the per-layer kernels; the grouping therefore belongs to the
 * device it was built on (a layer call on a device with another SM count
 * writes no output and mole_check reports MOLE_ERR_ARG).
 *
 * mole_lookup_combine_groups is mole_lookup_combine (same arguments, layouts,
 * results bit for bit, and error behaviour) for a batch whose grouping was
 * built from the same ids, T and N: each distinct id's row block is read once
 * and applied to all of that id's tokens.  The call may also write one
 * layer's gates into `groups`, so calls that share a groups buffer must not
 * overlap on the GPU.  The grouped kernels serve bf16 inputs with T >= 1024;
 * other calls run the mole_lookup_combine kernels (the grouping is then
 * unused).
 *
 * mole_lookup_combine_grouped builds the grouping in `workspace` and runs
 * mole_lookup_combine_groups, for a single layer;
 * mole_lookup_combine_grouped_workspace equals mole_token_groups_workspace.
 * All three return MOLE_ERR_WORKSPACE if the buffer is NULL or too small
 * (T > 0) and MOLE_ERR_ALIGN if it is not 16-byte aligned.
 */
size_t mole_token_groups_workspace(int64_t T, int32_t N);
mole_status mole_token_groups_build(const int32_t* ids, int64_t T, int64_t V, int32_t N, void* groups,
                                    size_t bytes, cudaStream_t stream);
mole_status mole_lookup_combine_groups(const int32_t* ids, int64_t T, const void* groups, size_t bytes,
                                       const void* h, const void* Wr, const void* lut, int64_t V, int32_t N,
                                       int64_t D, mole_dtype dt, float* out, cudaStream_t stream);
size_t mole_lookup_combine_grouped_workspace(int64_t T, int32_t N);
mole_status mole_lookup_combine_grouped(const int32_t* ids, int64_t T, const void* h, const void* Wr,
                                        const void* lut, int64_t V, int32_t N, int64_t D, mole_dtype dt,
                                        float* out, void* workspace, size_t ws_bytes, cudaStream_t stream);

/*
 * ---- NF3 table compression (MoLE page, 实验结果: 3-bit table, e.g. NF3) ----
 *
 * Quantises a bf16 table [V, N, D] (D % 64 == 0) in blocks of 64 consecutive
 * elements of one (v, j) row, in IEEE fp32:
 *     s = fp16(min(max_e |x_e|, 65504))                 (ties to even)
 *     c_e = #{k : x_e / s > mid_k}   (s > 0; correctly rounded division)
 *     c_e = 3 (the level 0.0)        (s == 0)
 * with the NormalFloat k=3 levels (QLoRA construction, rounded to fp16; see
 * mole_nf3_levels) and mid_k the fp32 midpoints of adjacent levels.  Code e
 * occupies bits [3e, 3e+3) of the block's 24-byte little-endian bit string.
 *   codes  : [V, N, D/64, 24] uint8    scales : [V, N, D/64] fp16 bits
 * lut_bf16 must be 16-byte aligned; codes 8-byte aligned.
 */
mole_status mole_quantize_lut_nf3(const void* lut_bf16, int64_t V, int32_t N, int64_t D,
                                  uint8_t* codes, uint16_t* scales, cudaStream_t stream);

/*
 * mole_build_lut and mole_quantize_lut_nf3 in one pass: the bf16 table is
 * never written.  The second tensor-core GEMM's epilogue rounds each output
 * to bf16 (the value mole_build_lut would store), quantises every 64-element
 * block of a (v, j) row in registers and writes the codes and the fp16 scale;
 * the results equal mole_build_lut followed by mole_quantize_lut_nf3, bit for
 * bit.  bf16 only, on the tensor-core path (D % 64 == 0, Dr % 64 == 0,
 * 16-byte aligned embed, W1, W2 and workspace; else MOLE_ERR_UNSUPPORTED);
 * codes 8-byte aligned.  Workspace as for mole_build_lut (dt = MOLE_BF16).
 */
mole_status mole_build_lut_nf3(const void* embed, const void* W1, const void* W2, int64_t V, int64_t D,
                               int32_t N, int64_t Dr, mole_act act, uint8_t* codes, uint16_t* scales,
                               void* workspace, size_t ws_bytes, cudaStream_t stream);

/*
 * mole_lookup_combine over an NF3 table: the row element for (id, j, d) is
 * level[c] * s of its block (exact in fp32), dequantised in registers inside
 * the gather.  Same arguments and error behaviour as mole_lookup_combine,
 * with D % 64 == 0.
 */
mole_status mole_lookup_combine_nf3(const int32_t* ids, int64_t T, const void* h,
                                    const void* Wr, const uint8_t* codes,
                                    const uint16_t* scales, int64_t V, int32_t N, int64_t D,
                                    mole_dtype dt, float* out, cudaStream_t stream);

/*
 * mole_lookup_combine_nf3 for a batch whose token grouping was built from the
 * same ids, T and N (see mole_token_groups_build): each distinct id's code and
 * scale blocks are read and decoded once and applied to all of that id's
 * tokens.  Same arguments, results (bit for bit) and error behaviour as
 * mole_lookup_combine_nf3, plus the groups buffer (as for
 * mole_lookup_combine_groups).  The grouped kernels serve bf16 inputs,
 * T >= 1024, N <= 16 with N * D/64 a multiple of 8, and 16-byte aligned codes
 * and scales; other calls run the mole_lookup_combine_nf3 kernels.
 */
mole_status mole_lookup_combine_nf3_groups(const int32_t* ids, int64_t T, const void* groups, size_t bytes,
                                           const void* h, const void* Wr, const uint8_t* codes,
                                           const uint16_t* scales, int64_t V, int32_t N, int64_t D, mole_dtype dt,
                                           float* out, cudaStream_t stream);

/*
 * ---- Offloaded table (MoLE page, 推理阶段 and 复杂度分析) ----
 *
 * The page's deployment: the table lives in slower, larger memory (CPU memory
 * or storage) and per token only its N expert-output rows move to the
 * accelerator.  Here the table (or its NF3 codes and scales) stays in host
 * memory that is pinned and mapped into the device's address space
 * (cudaHostAlloc, or cudaHostRegister with cudaHostRegisterMapped; memory of
 * the current device is accepted too).  Per batch each distinct id's row
 * block crosses the link once, into a device staging buffer, and the combine
 * reads the staging buffer.  Both calls take a grouping of the batch built by
 * mole_token_groups_build (same T, V and N): it numbers the batch's distinct
 * ids 0..U-1, and the staging buffer holds the row block of distinct id u at
 * index u.
 *
 * mole_offload_staging_bytes: size of the staging buffer for a batch of T
 *   tokens over a table of V ids (room for min(T, V) row blocks).  nf3 = 0:
 *   the table has dtype dt, [V, N, D]; nf3 = 1: NF3 codes [V, N, D/64, 24]
 *   and fp16 scales [V, N, D/64] (D % 64 == 0).  0 for invalid arguments.
 *
 * mole_offload_stage copies the batch's distinct row blocks from `table`
 *   (and, NF3, `scales`) into `staging` (device, 16-byte aligned, at least
 *   mole_offload_staging_bytes bytes).  table must be 16-byte aligned (NF3
 *   codes 8-byte, scales 2-byte).  If n_rows is not NULL it receives U (one
 *   device int32).  Pageable (unregistered) host memory gives MOLE_ERR_ARG.
 *   One kernel launch; the host table must stay unchanged until it has run.
 *
 * mole_lookup_combine_offload is mole_lookup_combine (or, nf3 = 1,
 *   mole_lookup_combine_nf3) over the staged rows: the same results, bit for
 *   bit, as those calls on the table itself, and the same error behaviour
 *   (a token whose id is outside [0, V) gets a NaN row).  No ids argument:
 *   the grouping holds each token's dense index.  Calls that share a groups
 *   buffer must not overlap on the GPU (the call writes the layer's gates
 *   into it); a staging buffer may be refilled for the next layer once the
 *   combine that reads it has run, so two staging buffers let the next
 *   layer's copy overlap this layer's combine.
 *
 * Both return MOLE_ERR_WORKSPACE for a missing or too small groups or staging
 * buffer; T == 0 is a no-op.
 */
size_t mole_offload_staging_bytes(int64_t T, int64_t V, int32_t N, int64_t D, mole_dtype dt, int32_t nf3);
mole_status mole_offload_stage(int64_t T, const void* groups, size_t bytes, const void* table,
                               const uint16_t* scales, int64_t V, int32_t N, int64_t D, mole_dtype dt,
                               int32_t nf3, void* staging, size_t staging_bytes, int32_t* n_rows,
                               cudaStream_t stream);
mole_status mole_lookup_combine_offload(int64_t T, const void* groups, size_t bytes, const void* h,
                                        const void* Wr, const void* staging, size_t staging_bytes, int64_t V,
                                        int32_t N, int64_t D, mole_dtype dt, int32_t nf3, float* out,
                                        cudaStream_t stream);

/*
 * ---- FFN block: shared expert + routed-expert mixture + residual ----
 * (MoLE page, 训练阶段 and 推理阶段: the shared experts stay dense FFNs on the
 * previous layer's output at inference; only the routed experts become the
 * table.  The page gives no formula; this library's reading: one shared
 * expert of the routed experts' form, act(h . W1s) . W2s, and the block's
 * output is residual + shared expert + routed mixture.)
 *
 * mole_shared_ffn: out = act(h . W1s) . W2s + add + residual  (fp32)
 *   h : [T, D] bf16   W1s : [D, Ds] bf16   W2s : [Ds, D] bf16
 *   add, residual : [T, D] fp32 or NULL   out : [T, D] fp32 (may be add or
 *   residual: each element is read before it is written)
 *   Two tcgen05 GEMMs (fp32 accumulate); the hidden activation is rounded to
 *   bf16 in `workspace` (at least mole_shared_ffn_workspace(T, Ds) bytes);
 *   the additions happen in the second GEMM's epilogue.  Needs D % 64 == 0,
 *   Ds % 64 == 0 and 16-byte aligned pointers (else MOLE_ERR_UNSUPPORTED /
 *   MOLE_ERR_ALIGN).
 *
 * mole_ffn_block: out = residual + act(h . W1s) . W2s + sum_j g_j LUT[ids[t], j]
 *   The routed mixture is mole_lookup_combine_groups over `groups` (built from
 *   the same ids, T and N), written into the workspace and added in the
 *   shared expert's second GEMM epilogue.  bf16 inputs, D % 64 == 0,
 *   Ds % 64 == 0; workspace of mole_ffn_block_workspace(T, D, Ds) bytes; out
 *   may be residual.  Bad ids: NaN rows and MOLE_ERR_INDEX from mole_check,
 *   as for the combine.
 */
size_t mole_shared_ffn_workspace(int64_t T, int64_t Ds);
mole_status mole_shared_ffn(const void* h, const void* W1s, const void* W2s, int64_t T, int64_t D, int64_t Ds,
                            mole_act act, const float* add, const float* residual, float* out, void* workspace,
                            size_t ws_bytes, cudaStream_t stream);
size_t mole_ffn_block_workspace(int64_t T, int64_t D, int64_t Ds);
mole_status mole_ffn_block(const int32_t* ids, int64_t T, const void* groups, size_t groups_bytes, const void* h,
                           const void* Wr, const void* lut, int64_t V, int32_t N, const void* W1s, const void* W2s,
                           int64_t D, int64_t Ds, mole_act act, const float* residual, float* out,
                           void* workspace, size_t ws_bytes, cudaStream_t stream);

/*
 * ---- Training: one MoLE layer forward and backward (MoLE page, 训练阶段) ----
 *
 * In training the routed experts take the token's embedding row as input and
 * all N are active, mixed by the router on the previous layer's output h:
 *     out[t] = sum_j softmax(h[t] . Wr)_j f_j(E[ids[t]]),
 *     f_j(x) = act(x . W1[j]) . W2[j]   (hidden activation rounded to bf16)
 * A routed expert's output depends only on the token id, so the forward
 * evaluates the experts on the batch's distinct ids only (the table build on
 * those embedding rows, tcgen05 GEMMs) and mixes them with the combine
 * kernels: `out` equals mole_lookup_combine over a table built by
 * mole_build_lut, bit for bit.  The grouping (`groups`, from
 * mole_token_groups_build with the same ids, T, V and N) supplies the distinct
 * ids.  The forward reads their count back to the host (one stream
 * synchronisation) and returns it in *n_distinct; the backward takes it back.
 *
 * mole_train_backward adds (+=, fp32) the gradients of L = sum(out * dout)
 * (dout [T, D] fp32) to dh [T, D], dWr [D, N], dE [V, D] (the batch's rows
 * only), dW1 [N, D, Dr] and dW2 [N, Dr, D]; any of them may be NULL.  The
 * backward GEMMs (bf16 operands, fp32 accumulation) run in cuBLAS, whose
 * handle (created on a device's first backward call) holds cuBLAS's own device
 * memory; its operands dL/dY and dL/dpre are rounded to bf16 from fp32.  The
 * bf16 rounding of the hidden activation counts as identity in the backward.
 * Tokens with an id outside [0, V) get NaN outputs (MOLE_ERR_INDEX from
 * mole_check) and contribute no gradient.
 *
 *   h [T, D] bf16, Wr [D, N] bf16, E [V, D] bf16, W1 [N, D, Dr] bf16,
 *   W2 [N, Dr, D] bf16; out [T, D] fp32.  D % 64 == 0, Dr % 64 == 0, N <= 32,
 *   16-byte aligned pointers.  `cache` (device, 16-byte aligned) carries the
 *   forward's intermediates to the backward: at least
 *   mole_train_cache_bytes(T, V, N, D, Dr) bytes (room for min(T, V) distinct
 *   ids), not to be reused between a step's forward and backward.
 */
size_t mole_train_cache_bytes(int64_t T, int64_t V, int32_t N, int64_t D, int64_t Dr);
mole_status mole_train_forward(const int32_t* ids, int64_t T, const void* groups, size_t groups_bytes,
                               const void* h, const void* Wr, const void* E, const void* W1, const void* W2,
                               int64_t V, int32_t N, int64_t D, int64_t Dr, mole_act act, float* out, void* cache,
                               size_t cache_bytes, int32_t* n_distinct, cudaStream_t stream);
mole_status mole_train_backward(const int32_t* ids, int64_t T, const void* groups, size_t groups_bytes,
                                const void* h, const void* Wr, const void* E, const void* W1, const void* W2,
                                int64_t V, int32_t N, int64_t D, int64_t Dr, mole_act act, const float* dout,
                                void* cache, size_t cache_bytes, int32_t n_distinct, float* dh, float* dWr,
                                float* dE, float* dW1, float* dW2, cudaStream_t stream);

/*
 * ---- Around the layer in a training step: embedding, block norms, optimizer ----
 * (MoLE page, 训练阶段: the model trains end to end on the language-model loss;
 * the embedding matrix is the model's input table and the routed experts'
 * input.  The page gives no formulas for the parts around a layer; the forms
 * below are this library's reading.)  All of them run on the device that is
 * current, enqueue kernels only (no synchronisation, no allocation: a call can
 * be captured in a CUDA graph), and give the same bits on every run.
 *
 * mole_embed_forward: out[t, :] = scale * E[ids[t], :], the product in fp32,
 *   rounded once to dt_out.
 *     ids : [T] int32 in [0, V)   E : [V, D] dt_E   out : [T, D] dt_out
 *   A token with an id outside [0, V) gets a NaN row and sets the device error
 *   word (MOLE_ERR_INDEX from mole_check).
 *
 * mole_embed_backward: dE[v, :] += scale * sum over the tokens t with
 *   ids[t] == v of dout[t, :].  Sums in fp32 over the tokens in ascending
 *   order (in partial sums over fixed runs of the sorted tokens), one addition
 *   to dE per row; rows of ids that the batch does not hold are not touched.
 *   Ids outside [0, V) contribute nothing and set the device error word.
 *     dout : [T, D] dt   dE : [V, D] fp32 (added to)
 *     workspace : device, 16-byte aligned, at least
 *       mole_embed_backward_workspace(T, D) bytes; contents unspecified on
 *       return; calls that share one must not overlap on the GPU.
 *   More than 2048 tokens need a GPU that runs a cluster of 16 CTAs (a whole
 *   B200 does; a partition of one may not: MOLE_ERR_CUDA, and dE as it was).
 *
 * Both take any D up to 2^20 and T up to 2^31 - 1 (T == 0 is a no-op), and
 * pointers aligned to their element.  Rows that start on 4 elements (D a
 * multiple of 4, pointers aligned to 16 bytes, bf16 ones to 8) take the vector
 * kernels, and so does the lookup in a bf16 table of any D with such pointers.
 */
mole_status mole_embed_forward(const int32_t* ids, int64_t T, const void* E, int64_t V, int64_t D, float scale,
                               mole_dtype dt_E, void* out, mole_dtype dt_out, cudaStream_t stream);
size_t mole_embed_backward_workspace(int64_t T, int64_t D);
mole_status mole_embed_backward(const int32_t* ids, int64_t T, const void* dout, mole_dtype dt, int64_t V, int64_t D,
                                float scale, float* dE, void* workspace, size_t ws_bytes, cudaStream_t stream);

/*
 * The norms around a block, with its gate and the residual scale.  With
 * rms(u) = sqrt(mean_d u_d^2 + eps) per token:
 *     y  = w_post * f / rms(f)              (post-norm; y = f where w_post is NULL)
 *     x' = res_scale * x + gate[t] * y      (gate = 1 where gate is NULL; y = 0 where f is NULL)
 *     h  = w_pre * x' / rms(x')             (the next block's input)
 * so one call takes a block's output f (mole_ffn_block without its residual,
 * mole_lookup_combine, ...) to the next stream x' and the next block's input;
 * with f NULL it is the norm before the first block, with h NULL the end of
 * the last one.  All arithmetic in fp32 (the sum of a row's squares too: rows
 * whose sum passes 2^128, of values around 10^18, are not served); h is computed
 * from x' before x' is rounded to dt_x.
 *   x : [T, D] dt_x   f : [T, D] dt_f or NULL   w_post, w_pre : [D] fp32 or NULL
 *   gate : [T] fp32 or NULL   x_out : [T, D] dt_x or NULL (may be x)
 *   h : [T, D] dt_h or NULL (needs w_pre; not overlapping any other tensor)
 * At least one of x_out and h; w_post and gate need f; eps > 0.
 *
 * mole_block_norm_backward: from the gradients of x' and h (dx_out, dh; either
 * may be NULL = zero, not both),
 *     G  = dx_out + d(h)/d(x')^T dh         at x' as stored (x_out, dt_x)
 *     dx = res_scale * G,  dgate[t] = <G, y>,  df = gate[t] * d(y)/d(f)^T G
 *     dw_pre[d] += sum_t dh x'/rms(x'),  dw_post[d] += sum_t gate[t] G f/rms(f)
 * dx [T, D], df [T, D] and dgate [T] (fp32) are overwritten; dw_pre and dw_post
 * ([D] fp32) are added to.  Any output may be NULL, not all.  dh needs w_pre;
 * x_out may be NULL where dh is; dgate, w_post and dw_post need f (dw_post
 * needs w_post too).  dx may be dx_out, df may be dh, and dw_pre may be dw_post
 * (both norms' weights one vector: it gets both sums); other overlaps are not
 * allowed.  workspace (device, 16-byte aligned):
 * mole_block_norm_backward_workspace(T, D) bytes, needed for dw_pre and
 * dw_post only; calls that share one must not overlap on the GPU.
 *
 * Both take any D up to 8192 and T up to 2^31 - 1 (T == 0 is a no-op), and
 * pointers aligned to their element; where all pointers to rows and weights are
 * aligned to 16 bytes (bf16 ones to 8) the rows take vector accesses.  Where D
 * is not a multiple of 4 that goes up to D = 8189 in the forward pass, and in the
 * backward up to 5629 (x_out and f fp32), 6141 (one of them) or 6653 (bf16).
 */
mole_status mole_block_norm_forward(const void* x, mole_dtype dt_x, const void* f, mole_dtype dt_f,
                                    const float* w_post, const float* gate, float res_scale, const float* w_pre,
                                    float eps, int64_t T, int64_t D, void* x_out, void* h, mole_dtype dt_h,
                                    cudaStream_t stream);
size_t mole_block_norm_backward_workspace(int64_t T, int64_t D);
mole_status mole_block_norm_backward(const void* x_out, mole_dtype dt_x, const void* f, mole_dtype dt_f,
                                     const float* w_post, const float* gate, float res_scale, const float* w_pre,
                                     float eps, int64_t T, int64_t D, const float* dx_out, const float* dh, float* dx,
                                     float* df, float* dgate, float* dw_post, float* dw_pre, void* workspace,
                                     size_t ws_bytes, cudaStream_t stream);

/*
 * One AdamW step over a list of tensors (decoupled weight decay).  Per
 * element, in fp32, with g = grad_scale * grad, the weight p (master where
 * there is one, else param), and t the step number, counted from 1:
 *     m = beta1 m + (1 - beta1) g        v = beta2 v + (1 - beta2) g^2
 *     p = p - lr weight_decay p - lr m / (1 - beta1^t) / (sqrt(v / (1 - beta2^t)) + eps)
 * eps is 0 to 2^125, and one below 2^-126 counts as 2^-126: an element whose m
 * is zero takes a step of zero, also where v and eps are zero.
 * param = p rounded to its type (and master = p).  A bf16 param without a
 * master rounds to nearest every step, so updates below half a bf16 step of
 * the weight are lost; with a master they add up.
 *
 * state8 = 0: m and v are [n] fp32.
 * state8 = 1: m and v are [n] e4m3 codes in blocks of 128 consecutive
 *   elements with one fp32 scale each ([ceil(n / 128)]): m = code * m_scale,
 *   sqrt(v) = code * v_scale.  The update uses the new m and v in fp32; then
 *   scale = max(max |.| / 448, 2^-120) and codes round to nearest even, except
 *   that a v > 0 never gets the code 0 (its element would take a step of
 *   lr m / eps).  All-zero codes and scales are the initial state.  A
 *   gradient that is not finite spoils the states of its whole block.
 *
 * The step number and the rate come from the host struct, or, where step_dev
 * or lr_dev is not NULL, from device memory when the kernel runs (a captured
 * step then follows them on every replay; a device step below 1 is not noticed
 * and makes the weights NaN); grad_scale_dev (NULL = 1) is a factor on every
 * gradient, such as a clipping factor computed on the device.
 *
 * tensors and config are HOST structs, read before the call returns.  No
 * memory that a call writes may overlap anything else in its list
 * (MOLE_ERR_ARG).  Any n >= 0 and pointers aligned to their element; a
 * tensor whose pointers are all aligned to 4 elements takes vector accesses.
 * One launch per 128 tensors.
 */
typedef struct {
  void* param;         /* [n] dt_param, overwritten */
  const void* grad;    /* [n] dt_grad */
  float* master;       /* [n] fp32 or NULL (dt_param MOLE_F32: must be NULL) */
  void* m;             /* [n] fp32, or e4m3 codes */
  void* v;
  float* m_scale;      /* [ceil(n / 128)] (state8), else NULL */
  float* v_scale;
  int64_t n;
  float weight_decay;
  int32_t dt_param, dt_grad; /* mole_dtype */
} mole_adamw_tensor;

typedef struct {
  double lr, beta1, beta2, eps;
  int64_t step;                 /* >= 1 (ignored where step_dev is given) */
  const int64_t* step_dev;      /* device, or NULL */
  const float* lr_dev;          /* device, or NULL */
  const float* grad_scale_dev;  /* device, or NULL */
  int32_t state8;
} mole_adamw_config;

mole_status mole_adamw_step(const mole_adamw_tensor* tensors, int32_t n_tensors, const mole_adamw_config* config,
                            cudaStream_t stream);

/* The 8 NF3 levels as fp16 bit patterns (ascending; index 3 is 0.0) and the 7
 * fp32 decision midpoints.  Host-only; no device work. */
void mole_nf3_levels(uint16_t levels_f16[8]);
void mole_nf3_midpoints(float mid[7]);

/*
 * ---- Gather plan (the set of table rows a batch fetches; MoLE page, 复杂度分析) ----
 *
 * uniq[0..n_uniq) receives the distinct ids of the batch in ascending order,
 * slot[t] the index of ids[t] in uniq.  uniq has capacity T; n_uniq is one
 * device int32.  Needs V <= 524288 (the id set is kept on chip).  Ids outside
 * [0, V) are skipped (slot = -1) and set the device error word.
 */
mole_status mole_gather_plan(const int32_t* ids, int64_t T, int64_t V, int32_t* uniq,
                             int32_t* n_uniq, int32_t* slot, cudaStream_t stream);

/*
 * ---- Cross-layer row prefetch (MoLE page, 推理阶段 + 复杂度分析) ----
 *
 * Every MoLE layer indexes its own table with the step's input token ids, so
 * all layers' rows are known before the first layer runs.  For each of the
 * n_tables tables and each token t with 0 <= ids[t] < V, asks the GPU's L2
 * cache to fetch row ids[t] of that table (row_bytes bytes at
 * tables[l] + ids[t] * row_bytes): bulk L2 prefetches, issued from many SMs,
 * that move no data into the SMs and that nothing waits for.  Later calls
 * that read those rows (the layers' combines, in this stream or another)
 * then hit L2 while the rows stay resident (126 MB of L2: prefetch no more
 * than fits).  Results of every call are unchanged; this is a hint.
 *
 *   ids    : [T] int32 device; ids outside [0, V) are skipped (the combine
 *            that reads them reports them)
 *   tables : HOST array of n_tables (<= 64) device pointers, 16-byte aligned;
 *            an NF3 table is two tables (codes, row_bytes = N * D / 64 * 24;
 *            scales, row_bytes = N * D / 64 * 2)
 *   row_bytes : bytes of one row, a multiple of 16 (bf16 table: N * D * 2)
 * MOLE_ERR_ALIGN for unaligned tables or row_bytes, MOLE_ERR_UNSUPPORTED for
 * more than 64 tables.  T == 0 or n_tables == 0 is a no-op.
 */
mole_status mole_prefetch_rows(const int32_t* ids, int64_t T, const void* const* tables, int32_t n_tables,
                               int64_t V, int64_t row_bytes, cudaStream_t stream);

/*
 * Waits (polling, at most timeout_ms >= 0 milliseconds) for `stream` to drain,
 * then reads and clears this device's error word.  A negative timeout_ms is
 * rejected with MOLE_ERR_ARG (no host wait is unbounded).  Returns MOLE_OK,
 * MOLE_ERR_INDEX (bad token id), MOLE_ERR_TIMEOUT (stream still busy, or a
 * device-side wait gave up), MOLE_ERR_ARG (a grouping was used on a device
 * with another SM count than the one it was built on; the layer's output was
 * not written), or MOLE_ERR_CUDA (an asynchronous CUDA error).
 */
mole_status mole_check(cudaStream_t stream, int timeout_ms);

#ifdef __cplusplus
}
#endif

#endif /* MOLE_H_ */
