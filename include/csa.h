/*
 * csa.h -- C ABI of the GB300 (sm_103a) causal-attention-score library,
 * libcsa_gb300.so.
 *
 * Two products, each a persistent tcgen05/TMA kernel (plus, for dense rows no
 * tensor map can describe, one realigning copy into caller workspace launched
 * before it), and the calls built on them: the batched NT product
 * (batch_matmul_nt), the fused
 * causal softmax of the scores (causal_softmax_forward), the score product
 * over fp32 inputs (trimul_forward_f32), many dense layers sharing W in one
 * launch (dense_xwt_grouped), and an allocation-free score entry point
 * (trimul_forward_noalloc). For training on and answering with such layers: rotary
 * positions and their gradient (rotary_forward, rotary_backward), a paged 8-bit cache of
 * keys and values (kv_cache_write, kv_cache_read), and attention over that cache for single
 * tokens and whole prompts (cache_attention_forward). For several answers to one prompt: the
 * books of such a cache (kv_pages_extend, kv_cache_fork, kv_pages_free, kv_cache_copy,
 * kv_cache_compact), attention that reads what sequences share once
 * (cache_attention_shared_forward), and log probabilities of tokens with their gradient
 * (token_logprobs_forward, token_logprobs_backward). Each is documented at its declaration
 * below.
 *
 *  trimul_forward  the causal triangular score product of
 *                  "llm.c dev/cuda/trimat_forward.cu" (the CPU referee
 *                  trimul_cpu, Chapter I; the lower-tile skip of trimul_global,
 *                  Chapter II):
 *                    out[b][h][t][t2] = (Q[b][h][t][:] . K[b][h][t2][:]) / sqrt(HS)
 *                                       for t2 <= t, the mask value for t2 > t,
 *                  with Q[b][h][t][d] = qkv[b][t][0][h][d] and
 *                       K[b][h][t2][d] = qkv[b][t2][1][h][d].
 *
 *  dense_xwt       the dense layer of "DietCode tests/codegen/
 *                  test_1_local_padding.py" (test_local_padding docstring):
 *                    Y[i][j] = sum_k X[i][k] * W[j][k]   (Y = X W^T)
 *                  for any M, I, H >= 1; tails are handled only where data is
 *                  fetched (zero fill) and written back (clipped), never in the
 *                  compute stage ("local padding").
 *
 * Conventions shared by every entry point:
 *  - Pointers named as device pointers must point to memory of the current CUDA
 *    device (cudaMalloc'd or torch-allocated). The caller owns every buffer,
 *    scratch space included (dense_xwt_ws); no call allocates device memory.
 *    The library keeps, per device, only fixed arrays in its own image: the
 *    status word, the kernels' work-list counters and the scratch of
 *    trimul_forward_noalloc (plus the page-locked completion words below).
 *  - bf16 inputs are passed as `const void*` to raw 16-bit bfloat16 values.
 *  - Outputs are fp32 and fully overwritten (no read-modify-write), but for the rotary,
 *    cache, cache-attention, pages and logits calls, which name their types and what they leave.
 *  - `stream` is a cudaStream_t passed as void*; NULL is the legacy default
 *    stream. Calls are asynchronous on that stream; argument errors are
 *    returned synchronously before anything is launched.
 *  - Return value: CSA_OK (0) or a negative csa_status. A failed call launches
 *    nothing and leaves the output untouched; csa_last_error() then describes it.
 *  - Work-list counters (trimul_forward, trimul_forward_ex, trimul_forward_f32,
 *    causal_softmax_forward): these kernels take work from a set of counters
 *    that their last CTA resets. A launch outside stream capture uses its
 *    stream's set (launches on one stream run in order); a stream gets a set
 *    that was never used or whose last launch has reported completion (through
 *    a 2 KB page-locked host array per kernel and device, made at the first such
 *    launch on that device -- make it outside any stream capture). With launches
 *    still in flight on 256 other streams, the call returns CSA_ERR_BUSY. A
 *    launch captured into a CUDA graph gets a set of its own for good, at most
 *    1024 per kernel and process (then CSA_ERR_BUSY); a graph instantiated more
 *    than once must not have two instances running at once. Launches whose work
 *    is dealt statically (lower-only scores, batch_matmul_nt) use no set.
 *  - The library keeps one device status word per device. A kernel whose
 *    bounded wait ran out records CSA_ERR_TIMEOUT there and returns early
 *    (its output is then incomplete); csa_get_status() reports and clears it.
 *  - Thread safety: entry points may be called from several host threads; the
 *    error string is per thread. Each call works on the calling thread's current
 *    device (cudaGetDevice); the first call on a thread makes that device's
 *    primary context current there (cudaSetDevice).
 */
#ifndef CSA_GB300_H
#define CSA_GB300_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef int csa_status;

#define CSA_OK                 0
#define CSA_ERR_NULL          -1  /* a required pointer is NULL */
#define CSA_ERR_SHAPE         -2  /* a size is <= 0, C % NH != 0, or an index overflows */
#define CSA_ERR_ALIGN         -3  /* a pointer or stride breaks the 16-byte rule below */
#define CSA_ERR_UNSUPPORTED   -4  /* a size beyond what the kernel implements (HS > 256) */
#define CSA_ERR_ARCH          -5  /* the current device is not sm_103 (GB300) */
#define CSA_ERR_LAUNCH        -6  /* the kernel launch failed (see csa_last_error) */
#define CSA_ERR_TIMEOUT       -7  /* a device-side bounded wait ran out (csa_get_status) */
#define CSA_ERR_CUDA          -8  /* a CUDA runtime/driver call failed (no device, ...) */
#define CSA_ERR_CHECK         -9  /* a device-side index check of a debug build (built with
                                     -DCSA_DEBUG) failed (reported by csa_get_status) */
#define CSA_ERR_WORKSPACE    -10  /* dense_xwt_ws: workspace missing or smaller than
                                     dense_xwt_workspace_size reports */
#define CSA_ERR_BUSY         -11  /* no work-list counter set free: score or softmax
                                     launches in flight on 256 other streams, or more
                                     than 1024 of them captured into CUDA graphs */
#define CSA_ERR_INDEX        -12  /* a page number, row range or length in device memory was
                                     out of range; what it named was skipped (reported by
                                     csa_get_status) */

#define CSA_ERR_PAGES        -13  /* kv_pages_extend or kv_cache_fork found too few free pages;
                                     entries they were not enough for were left as they were
                                     (reported by csa_get_status) */

/* Causal mask bit patterns for the upper triangle (t2 > t). The page writes
 * NAN (the float quiet NaN, 0x7FC00000) and notes -inf would also do. */
#define CSA_MASK_NAN          0x7FC00000u
#define CSA_MASK_NEG_INF      0xFF800000u

/* trimul_forward_ex flags. */
#define CSA_TRIMUL_FULL        0u  /* write every element: scores below, mask above */
#define CSA_TRIMUL_LOWER_ONLY  1u  /* write only t2 <= t; leave t2 > t untouched
                                      (what the page's GPU kernels do, tri4's
                                      "don't write above the diagonal") */

/*
 * trimul_forward -- causal score product, NaN mask, default stream.
 *
 *   out  device, fp32, (B, NH, T, T) contiguous, fully overwritten.
 *   qkv  device, bf16, (B, T, 3, NH, HS) contiguous, HS = C / NH; read only.
 *   B, T, C, NH >= 1, C % NH == 0.
 *
 * Requirements (else CSA_ERR_ALIGN / CSA_ERR_UNSUPPORTED): qkv and out 16-byte
 * aligned; HS % 8 == 0 (the TMA row pitch of a head is HS*2 bytes and must be
 * a multiple of 16); HS <= 256. Any T >= 1 is accepted: rows and columns past
 * T are zero-filled on fetch and clipped on store. Scores are computed as
 * fp32 accumulations of exact bf16 products, then multiplied by the fp32
 * value of 1/sqrt(HS).
 */
csa_status trimul_forward(float* out, const void* qkv, int B, int T, int C, int NH);

/*
 * trimul_forward_ex -- as trimul_forward, with
 *   mask_bits  the 32-bit pattern written above the diagonal (CSA_MASK_NAN,
 *              CSA_MASK_NEG_INF or any other pattern);
 *   flags      CSA_TRIMUL_FULL or CSA_TRIMUL_LOWER_ONLY;
 *   stream     cudaStream_t (void*), NULL = default stream.
 */
csa_status trimul_forward_ex(float* out, const void* qkv, int B, int T, int C, int NH,
                             uint32_t mask_bits, uint32_t flags, void* stream);

/*
 * trimul_forward_f32 -- the causal score product over fp32 inputs, the
 * referee's own input type ("llm.c dev/cuda/trimat_forward.cu": trimul_cpu
 * takes const float* inp, and main fills it with fp32 random numbers), with no
 * rounding of the inputs to bf16.
 *
 *   out        device, fp32, (B, NH, T, T) contiguous; every element written
 *              (or only t2 <= t with CSA_TRIMUL_LOWER_ONLY).
 *   qkv        device, fp32, (B, T, 3, NH, HS) contiguous, HS = C / NH; read only.
 *   mask_bits, flags, stream   as trimul_forward_ex.
 *
 * Arithmetic: tcgen05 kind::tf32 with three products per input pair. Each
 * input x is split exactly into hi (x with its 13 lowest mantissa bits
 * cleared, a tf32 value: what the tensor core reads of x) and lo = x - hi;
 * each score accumulates
 * hi_q.hi_k + hi_q.lo_k + lo_q.hi_k in fp32, leaving out lo_q.lo_k, so each
 * product carries a relative error of a few units of 2^-20 on top of the fp32
 * accumulation, and the result is multiplied by the fp32 value of 1/sqrt(HS).
 *
 * Requirements (else CSA_ERR_ALIGN / CSA_ERR_UNSUPPORTED): qkv 16-byte and out
 * 4-byte aligned; HS % 4 == 0 (the TMA row pitch of a head is HS*4 bytes);
 * HS <= 256. Any T >= 1. Errors as trimul_forward_ex; nothing is written on
 * an argument error. The caller owns every buffer; nothing is allocated.
 */
csa_status trimul_forward_f32(float* out, const float* qkv, int B, int T, int C, int NH,
                              uint32_t mask_bits, uint32_t flags, void* stream);

/*
 * trimul_forward_noalloc -- trimul_forward_ex for callers that must not
 * allocate device memory. No passage of the pages has a counterpart: this
 * entry point exists for deployment, not for the method.
 *
 * Who needs it: code that runs where a new device allocation is not allowed or
 * not affordable -- under a memory manager that forbids allocations after
 * start-up, inside a region that must not trigger the device-wide
 * synchronisation cudaFree brings, or in plug-in hosts that only hand out
 * buffers. trimul_forward_ex itself never calls cudaMalloc either, but keeps
 * per-launch scheduling counters in a ring of slots; this variant instead
 * keeps its scratch -- the kernel's work-list counters (next position,
 * finished CTAs, next fill tile) -- in one fixed
 * 256-byte device array that every GPU loading the library holds until exit,
 * and calls no cudaMalloc, cudaFree or allocating library routine.
 *
 * Arguments, layouts, results and errors are those of trimul_forward_ex, plus:
 *  - The first call on each device looks up the array's device address
 *    (cudaGetSymbolAddress); make that first call before any stream capture.
 *  - Every call clears the counters (cudaMemsetAsync on `stream`) before its
 *    kernel starts. All calls on a device share the array, so two calls whose
 *    kernels overlap on the GPU (different streams, no ordering) race and may
 *    leave output tiles unwritten; serialise them.
 *  - A problem whose tile list exceeds what the 32-bit counters can index
 *    (2^31 - 2^20 output tiles of 128 x 128) is rejected with CSA_ERR_SHAPE.
 */
csa_status trimul_forward_noalloc(float* out, const void* qkv, int B, int T, int C, int NH,
                                  uint32_t mask_bits, uint32_t flags, void* stream);

/*
 * dense_xwt -- Y = X W^T, default stream.
 *
 *   Y  device, fp32, [M, H] row-major, fully overwritten.
 *   X  device, bf16, [M, I] row-major; W device, bf16, [H, I] row-major.
 *   M, I, H >= 1, any values (no tile-multiple requirement).
 *
 * X and W need only 2-byte alignment. When I*2 is a multiple of 16 and both are
 * 16-byte aligned, tiles are fetched by TMA straight from X and W. Otherwise
 * (rows no tensor map can describe, e.g. I = 770) this call, which has no
 * workspace, fetches them with loader warps; dense_xwt_ws computes the same
 * layer faster with caller workspace. Y is written by TMA when H*4 is a
 * multiple of 16 and Y is 16-byte aligned (4-byte alignment required
 * otherwise). Tiles are 128 x BN (BN 64..256) per CTA, or, for problems large
 * enough (csa_dense_tiling), 256 x BN per cluster of two CTAs (tcgen05
 * cta_group::2) when the rows are fetched by TMA. Sums are fp32 accumulations of
 * exact bf16 products, in the same order on every fetch path and tiling (results
 * are bit-identical). Nothing is allocated.
 */
csa_status dense_xwt(float* Y, const void* X, const void* W, int M, int I, int H);

/* dense_xwt_ex -- as dense_xwt on `stream` (cudaStream_t as void*). */
csa_status dense_xwt_ex(float* Y, const void* X, const void* W, int M, int I, int H,
                        void* stream);

/*
 * dense_xwt_workspace_size -- bytes of device workspace dense_xwt_ws needs for
 * these operands, written to *bytes: 0 when tensor maps describe the rows of X
 * and W as they are (I*2 % 16 == 0, both 16-byte aligned), else
 * 256 + ceil256(M*P*2) + H*P*2 with P = I rounded up to a multiple of 64 (a
 * copy of X and W whose rows start on 128-byte boundaries, and alignment
 * slack). Depends on the pointers' alignment and the sizes only.
 * CSA_ERR_NULL / CSA_ERR_SHAPE as dense_xwt (then *bytes = 0).
 */
csa_status dense_xwt_workspace_size(const void* X, const void* W, int M, int I, int H,
                                    size_t* bytes);

/*
 * dense_xwt_ws -- dense_xwt with caller-owned scratch, on `stream`. Where no
 * tensor map can describe the rows of X and W, a first kernel copies them into
 * `workspace` as rows of pitch P (128-byte multiples) and the product kernel
 * fetches every tile from that copy by TMA, with zero fill past M, H and I --
 * the local padding of "DietCode tests/codegen/test_1_local_padding.py"
 * (bounds handled only where data is fetched and written back).
 *   workspace        device, 16-byte aligned, at least dense_xwt_workspace_size
 *                    bytes (else CSA_ERR_WORKSPACE / CSA_ERR_ALIGN, nothing
 *                    launched); may be NULL when that size is 0.
 *   workspace_bytes  its size.
 * The workspace needs no clearing, and its content after a call is unspecified.
 * It is in use until the call's kernels complete on `stream`: calls that may
 * overlap on the GPU need separate workspaces. Results are bit-identical to
 * dense_xwt on the same operands. Nothing is allocated.
 */
csa_status dense_xwt_ws(float* Y, const void* X, const void* W, int M, int I, int H,
                        void* workspace, size_t workspace_bytes, void* stream);

/*
 * dense_xwt_grouped -- Y[g] = X[g] W^T for g = 0 .. n-1, asynchronous on `stream`:
 * n dense layers that share W (device, bf16, [H, I]), I and H, computed by one
 * persistent launch over all their tiles (one launch per 48 problems), so that
 * a batch of dynamic-shape calls costs one launch instead of n.
 *   Y  host array of n device pointers: Y[g] fp32 [M[g], H] row-major, fully
 *      overwritten.
 *   X  host array of n device pointers: X[g] bf16 [M[g], I] row-major.
 *   M  host array of n row counts, each >= 1.
 * The host arrays are read during the call only. Results are bit-identical to n
 * dense_xwt calls. When I * 2 is not a multiple of 16, or W or some X[g] is not
 * 16-byte aligned, this call (no workspace) makes n dense_xwt launches instead;
 * dense_xwt_grouped_ws keeps such a batch in one grouped launch. Alignment: X[g]
 * and W 2-byte, Y[g] 4-byte (Y written by TMA when H * 4 % 16 == 0 and every Y[g]
 * is 16-byte aligned). CSA_ERR_NULL / CSA_ERR_SHAPE / CSA_ERR_ALIGN name the first
 * offending problem; nothing is launched then.
 */
csa_status dense_xwt_grouped(float* const* Y, const void* const* X, const void* W, const int* M,
                             int n, int I, int H, void* stream);

/*
 * dense_xwt_grouped_workspace_size -- bytes of device workspace
 * dense_xwt_grouped_ws needs for these operands, written to *bytes: 0 when
 * tensor maps describe the rows of W and of every X[g] as they are, else
 * 256 + ceil256(H*P*2) + sum_g ceil256(M[g]*P*2), P = I rounded up to 64.
 * CSA_ERR_NULL / CSA_ERR_SHAPE (then *bytes = 0).
 *
 * dense_xwt_grouped_ws -- dense_xwt_grouped with caller-owned scratch. Where no
 * tensor map can describe the rows (e.g. I = 770), one copy launch per 48
 * problems writes W's and the X[g]'s rows into `workspace` as 128-byte-aligned
 * rows (W once, then the problems in order), and the grouped launch reads them
 * from there, instead of one loader-warp dense_xwt per problem. Same bits as n
 * dense_xwt calls. workspace NULL is dense_xwt_grouped itself; otherwise it
 * must be 16-byte aligned and at least the size above (else CSA_ERR_ALIGN /
 * CSA_ERR_WORKSPACE, nothing launched). It is in use until the call's kernels
 * complete on `stream`. Nothing is allocated.
 */
csa_status dense_xwt_grouped_workspace_size(const void* const* X, const void* W, const int* M,
                                            int n, int I, int H, size_t* bytes);
csa_status dense_xwt_grouped_ws(float* const* Y, const void* const* X, const void* W,
                                const int* M, int n, int I, int H, void* workspace,
                                size_t workspace_bytes, void* stream);

/*
 * csa_set_dense_fetch -- process-wide fetch mode of dense_xwt_ws for rows that
 * no tensor map can describe (I*2 not a multiple of 16, or X / W not 16-byte
 * aligned):
 *   CSA_DENSE_FETCH_AUTO     copy the rows into the caller's workspace, then TMA;
 *   CSA_DENSE_FETCH_LOADERS  loader warps, as dense_xwt (the workspace unused).
 * Both modes give the same bits. Returns CSA_OK, or CSA_ERR_SHAPE for an
 * unknown mode (the mode is unchanged).
 */
#define CSA_DENSE_FETCH_AUTO    0
#define CSA_DENSE_FETCH_LOADERS 1
csa_status csa_set_dense_fetch(int mode);

/*
 * csa_dense_tiling -- the tiling dense_xwt / dense_xwt_ws choose for one problem of M
 * rows and H output columns whose rows are fetched by TMA (I * 2 % 16 == 0 and
 * 16-byte aligned operands, or rows realigned into a workspace), on a device or
 * stream with `sms` SMs: *bn = the tile width along H (64, 128, 192 or 256) and
 * *pairs = 1 when clusters of two CTAs compute 256-row tiles together (tcgen05
 * cta_group::2), else 0. Informational: a call falls back to single CTAs when no
 * cluster of two fits, and rows fetched by loader warps always use single CTAs.
 * Host only; returns CSA_OK, CSA_ERR_NULL or CSA_ERR_SHAPE.
 */
csa_status csa_dense_tiling(int M, int H, int sms, int* bn, int* pairs);

/*
 * csa_set_stream_sm_limit -- later calls of this library on `stream` (a
 * cudaStream_t; NULL is the legacy default stream) size their grids and tilings for
 * at most `max_sms` SMs: persistent kernels launch at most that many CTAs (CTA
 * pairs: max_sms / 2 clusters). Each of these kernels holds a whole SM per
 * CTA (its shared memory), so a call limited to S SMs on one stream and a call
 * limited to the device's SM count minus S on another can run side by side on
 * disjoint SMs, as long as the first is launched first (clusters need whole pairs
 * of SMs). max_sms = 0 removes the limit; a limit above the device's SM count has
 * no effect. Results are the same bits under any limit, but for cache_attention_forward,
 * cache_attention_shared_forward and token_logprobs_forward, whose sums are split by it. The
 * rotary, cache, pages and logits calls and the last, short kernels of the attention calls have
 * small CTAs, of which a limit allows in proportion (2 to 48 for each of max_sms;
 * kv_pages_extend, kv_cache_fork and kv_pages_free take some for each entry): it bounds their
 * share of the memory system, not the SMs they are on. The two parts of
 * cache_attention_shared_forward run side by side on max_sms SMs between them; each begins as
 * max_sms CTAs, of which those that the division leaves without work end as soon as they have read
 * it. Limits are keyed by the stream's handle value, process-wide, for at most 64 streams at once (then
 * CSA_ERR_BUSY); a stream destroyed with a limit set should have it removed
 * first, since a new stream may reuse the handle. Returns CSA_OK, CSA_ERR_SHAPE
 * for max_sms < 0, or CSA_ERR_BUSY.
 */
csa_status csa_set_stream_sm_limit(void* stream, int max_sms);

/* csa_get_stream_sm_limit -- the limit set on `stream` (0: none) into *max_sms. */
csa_status csa_get_stream_sm_limit(void* stream, int* max_sms);

/*
 * causal_softmax_forward -- the causal score rows of trimul_forward followed by
 * a softmax over t2 <= t, in one kernel (the scores never reach memory):
 *   att[b][h][t][t2] = exp(s[t2] - m) / sum_{u <= t} exp(s[u] - m)  for t2 <= t,
 *   att[b][h][t][t2] = 0                                               for t2 > t,
 * s = Q[b][h][t] . K[b][h][t2] / sqrt(HS), m = max_{u <= t} s[u]. The score is
 * the referee of "llm.c dev/cuda/trimat_forward.cu" (taken, as its comment
 * says, from the attention forward pass, where this softmax follows); the
 * softmax is the two-pass form of the "Smallem" article 5 (row maximum and sum
 * of exponentials, then normalisation).
 *   att  device, fp32, (B, NH, T, T) contiguous, fully overwritten.
 *   qkv  device, bf16, (B, T, 3, NH, HS), HS = C / NH, HS % 8 == 0, HS <= 128.
 * qkv 16-byte aligned, att 4-byte aligned. Asynchronous on `stream`.
 */
csa_status causal_softmax_forward(float* att, const void* qkv, int B, int T, int C, int NH,
                                  void* stream);

/*
 * batch_matmul_nt -- the unmasked, unscaled batched NT product of
 * "DietCode tests/codegen/test_1_local_padding.py" (test_local_padding_ii
 * docstring, BatchMatmulNT):
 *   Y[i][j][k] = sum_l X[i][j][l] * W[i][k][l]
 *   Y  device, fp32, [batch, T1, T2] row-major, fully overwritten.
 *   X  device, bf16, [batch, T1, D]; W device, bf16, [batch, T2, D].
 *   batch, T1, T2 >= 1 (any values: rows and columns past T1 / T2 are
 *   zero-filled on fetch and clipped on store), D % 8 == 0, D <= 256.
 * X and W 16-byte aligned, Y 4-byte aligned (TMA stores when T2 % 4 == 0 and Y
 * is 16-byte aligned). Same kernel as trimul_forward with every tile computed
 * and no mask or scale. Asynchronous on `stream` (cudaStream_t as void*).
 */
csa_status batch_matmul_nt(float* Y, const void* X, const void* W, int batch, int T1, int T2,
                           int D, void* stream);

/* Element types of the calls below (rows of 16- or 32-bit values). */
#define CSA_BF16 0
#define CSA_F16  1
#define CSA_F32  2

/*
 * rotary_forward -- rotary positions: every head's first rot_dim elements are turned,
 * pair by pair, by the angle p * f[i] of their token's position p:
 *   y0 = a (x0 cos - x1 sin),   y1 = a (x1 cos + x0 sin),
 * pairs (i, i + rot_dim/2), or (2i, 2i + 1) when `interleaved`; elements from rot_dim on
 * are copied. Computed in fp32 and rounded once.
 *   out, x       device, [tokens][heads][head_size] of `dtype`, head elements contiguous,
 *                tokens and heads *_token_stride and *_head_stride elements apart (so the
 *                Q and K parts of a packed (B,T,3,NH,HS) tensor are rotated in one call
 *                with heads = 2 NH and token stride 3C). out == x with equal strides
 *                rotates in place (elements from rot_dim on are then not touched). Memory
 *                ranges that overlap otherwise are refused (CSA_ERR_UNSUPPORTED), but for
 *                slices side by side in one tensor (with one stride between tokens, or
 *                between heads), and so are strides with which rows of `out` would overlap
 *                (CSA_ERR_SHAPE).
 *   turns        device, rot_dim/2 values of csa_rotary_turns.
 *   amplitude    a, finite.
 *   positions    device, int32 [tokens]; a negative one marks padding, whose rows of out
 *                are left as they were. Or NULL: token t has position
 *                start + (period > 0 ? t % period : t), start >= 0.
 * Any head_size >= 2, rot_dim even, 2 <= rot_dim <= head_size. Pointers and strides need
 * only the type's alignment; rows of 16-byte multiples take 16-byte loads. Angles come
 * from 64-bit fixed-point turns, whose product with the position is exact: what they are off
 * by is the frequency's rounding in double precision, p f 2^-51 radians at position p (below
 * the rounding to fp32 up to p f = 2^27, 2^-20 near 2^31).
 * Asynchronous on `stream`.
 *
 * rotary_backward -- the gradient: dx = a R(-p f) dy, same arguments (dx for out, dy for x).
 */
csa_status rotary_forward(void* out, const void* x, int dtype, int64_t tokens, int heads,
                          int head_size, int rot_dim, int64_t out_token_stride,
                          int64_t out_head_stride, int64_t x_token_stride, int64_t x_head_stride,
                          const uint64_t* turns, float amplitude, const int32_t* positions,
                          int start, int period, int interleaved, void* stream);
csa_status rotary_backward(void* dx, const void* dy, int dtype, int64_t tokens, int heads,
                           int head_size, int rot_dim, int64_t dx_token_stride,
                           int64_t dx_head_stride, int64_t dy_token_stride,
                           int64_t dy_head_stride, const uint64_t* turns, float amplitude,
                           const int32_t* positions, int start, int period, int interleaved,
                           void* stream);

/*
 * csa_rotary_turns -- fills turns[0 .. rot_dim/2 - 1] (host memory) with
 * round(f[i] / 2pi * 2^64), the frequencies f[i] = base^(-2i/rot_dim) scaled for contexts
 * longer than a model was trained on:
 *   CSA_ROTARY_NONE      as they are;
 *   CSA_ROTARY_LINEAR    f / factor (positions interpolated);
 *   CSA_ROTARY_NTK       base * factor^(rot_dim / (rot_dim - 2)) in place of base;
 *   CSA_ROTARY_BY_PARTS  f (g + (1 - g) / factor) with g = clip((r - slow) / (fast - slow), 0, 1)
 *                        and r = original_length f / 2pi, the turns a frequency makes over the
 *                        trained length (Peng et al., 2023): fast pairs kept, slow ones
 *                        interpolated.
 * Host only. CSA_ERR_NULL; CSA_ERR_SHAPE for rot_dim odd or < 2, base <= 1, factor < 1, or
 * (BY_PARTS) original_length <= 0 or fast <= slow; CSA_ERR_UNSUPPORTED for another scaling.
 */
#define CSA_ROTARY_NONE     0
#define CSA_ROTARY_LINEAR   1
#define CSA_ROTARY_NTK      2
#define CSA_ROTARY_BY_PARTS 3
csa_status csa_rotary_turns(uint64_t* turns, int rot_dim, double base, int scaling, double factor,
                            double original_length, double slow, double fast);

/*
 * csa_kv_cache -- a paged cache of keys and values in 8 bits. A page holds page_tokens
 * tokens of one sequence; each (page, head) is a block with one fp32 scale for K and one
 * for V, and its values are code * scale.
 *   k, v              device, 8-bit codes [pages][heads][page_tokens][head_size], 16-byte aligned;
 *   k_scale, v_scale  device, fp32 [pages][heads]: 0 (a block of zeros), or from 2^-100 up,
 *                     finite;
 *   page_tokens       16, 32, 64 or 128;
 *   head_size         a multiple of 16, at most 128;
 *   format            CSA_KV_INT8 (codes -127 .. 127) or CSA_KV_E4M3 (the 8-bit float of 4
 *                     exponent and 3 fraction bits, no infinities).
 * Nothing needs clearing: pages and slots no token was written to are never interpreted.
 */
#define CSA_KV_INT8 0
#define CSA_KV_E4M3 1
typedef struct csa_kv_cache {
  void* k;
  void* v;
  float* k_scale;
  float* v_scale;
  int pages, heads, page_tokens, head_size, format;
} csa_kv_cache;

/*
 * csa_kv_batch -- which rows of a call are which tokens of which sequence. Sequence s has
 * rows [offsets[s], offsets[s + 1]) of the call's `rows` rows; they are its last tokens, the
 * final one at position lengths[s] - 1. Block b of the sequence (tokens b * page_tokens on)
 * is page table[s][b].
 *   offsets      device, int32 [sequences + 1], not decreasing, within [0, rows];
 *   lengths      device, int32 [sequences], tokens INCLUDING the rows of this call, within
 *                [0, table_width * page_tokens];
 *   table        device, int32 [sequences][table_width]; entries past a length are not read;
 *   max_new      at least every offsets[s + 1] - offsets[s] (it sizes the launch).
 * Rows past offsets[sequences] are left as they were. Rows before a sequence's beginning
 * (more rows than its length) are neither written nor read; attention gives zeros there.
 * sequences, table_width, rows and max_new are at least 1 (an empty batch is no call).
 * These arrays are read on the device: a sequence whose entries break the rules is skipped,
 * as is a block whose page number is outside [0, pages), and csa_get_status reports
 * CSA_ERR_INDEX. Pages that a call writes belong to one sequence each and are in its
 * table once (prefix pages that several sequences share are full, and only read). The
 * arrays must not change while a call is under way: what it computes is then undefined,
 * though it stays within the rows, the pages and the workspace.
 */
typedef struct csa_kv_batch {
  const int32_t* offsets;
  const int32_t* lengths;
  const int32_t* table;
  int sequences, table_width, rows, max_new;
} csa_kv_batch;

/*
 * kv_cache_write -- quantises the rows of K and V into the cache.
 *   k, v   device, CSA_BF16 or CSA_F16 rows [rows][heads][head_size], head elements contiguous,
 *          strides in elements; pointers 16-byte aligned, strides multiples of 8 elements.
 * A block's scale is s = max(scale of what it held, s(m)), m its new rows' largest finite
 * magnitude: for int8 s(m) is the smallest value of 8 significant bits with 127 s >= m, for
 * e4m3 the smallest power of two with 448 s >= m, and at least 2^-100. Codes are x / s
 * rounded to nearest even (NaN: 0; infinities: the largest code); when a block's scale
 * grows, its older codes become code * s_old / s, rounded again. The codes are those of
 * this definition in real numbers (no fp32 rounding shows). A call whose rows begin inside a
 * block takes the slots before them as written, with the scale that is there. Asynchronous on
 * `stream`.
 *
 * kv_cache_read -- the values code * scale of the batch's rows, rounded once to `dtype`
 * (CSA_BF16, CSA_F16 or CSA_F32), into k and v. The batch may name other rows than those of
 * a write: any sequence's last offsets[s + 1] - offsets[s] tokens. k and v must not share
 * elements.
 */
csa_status kv_cache_write(const csa_kv_cache* cache, const csa_kv_batch* batch, const void* k,
                          const void* v, int dtype, int64_t k_token_stride, int64_t k_head_stride,
                          int64_t v_token_stride, int64_t v_head_stride, void* stream);
csa_status kv_cache_read(void* k, void* v, int dtype, int64_t k_token_stride,
                         int64_t k_head_stride, int64_t v_token_stride, int64_t v_head_stride,
                         const csa_kv_cache* cache, const csa_kv_batch* batch, void* stream);

/*
 * cache_attention_forward -- attention of the batch's rows over the cache (their own K and V
 * written before): row j of sequence s at position p = lengths[s] - n + j, query head h
 *   out = sum_t w_t v_t / sum_t w_t,   w_t = exp(scale * q . k_t)
 * over the visible t: t <= p, and with window > 0 also p - t < window or t < sinks. Query
 * heads h share kv head h / (q_heads / heads). A row that sees nothing gives zeros.
 *   out, q     device, [rows][q_heads][head_size] of CSA_BF16 or CSA_F16, strides as above;
 *              out == q with equal strides is fine, and so are slices side by side in one
 *              tensor; ranges that overlap otherwise are refused (CSA_ERR_UNSUPPORTED);
 *   q_heads    a multiple of cache->heads;
 *   scale      finite (the framework's score uses 1/sqrt(head_size));
 *   window     0: none; sinks >= 0 (used with a window);
 *   workspace  device, 16-byte aligned, cache_attention_workspace_size bytes; needs no
 *              clearing, in use until the call's kernels complete: calls that may overlap on
 *              the GPU, replays of captured ones too, need separate workspaces.
 * Codes enter the tensor cores as exact 16-bit values; scores, the running maximum, sums and
 * the output accumulate in fp32; weights, with V's scale, are rounded to fp16 for the product
 * with V (to 11 bits, and to 2^-32 of a row's largest); the result is rounded once. Every
 * visible key counts in the denominator, however far apart V's scales are (for V of up to
 * 2^100). Visible codes must not be NaN (kv_cache_write stores none). What no row of a
 * sequence sees (behind every window, past the sinks) does not matter: codes, and for pages of
 * nothing else their scales and table entries, which are not read. A query with an infinity or
 * a NaN spoils its own rows only. The order of every sum is fixed: same inputs and SM limit,
 * same bits. Asynchronous on `stream`; nothing is allocated.
 */
csa_status cache_attention_forward(void* out, const void* q, int dtype, int q_heads,
                                   int64_t out_token_stride, int64_t out_head_stride,
                                   int64_t q_token_stride, int64_t q_head_stride,
                                   const csa_kv_cache* cache, const csa_kv_batch* batch,
                                   float scale, int window, int sinks, void* workspace,
                                   size_t workspace_bytes, void* stream);

/* cache_attention_workspace_size -- bytes of workspace cache_attention_forward needs, into
 * *bytes. Depends on cache and q_heads only (checked as there). Host only. */
csa_status cache_attention_workspace_size(const csa_kv_cache* cache, int q_heads, size_t* bytes);

/*
 * cache_attention_shared_forward -- cache_attention_forward (without a window) for a batch whose
 * sequences share long beginnings, such as answers sampled from one prompt or requests behind one
 * set of instructions: the keys of what a group of sequences shares are read, and multiplied with
 * the rows of all of them, once.
 *   groups     device, int32 [group_count + 1], not decreasing, within [0, sequences]: group g is
 *              sequences groups[g] .. groups[g + 1] - 1 of the batch, next to each other;
 *              sequences of no group share nothing;
 *   shared     device, int32 [group_count]: the tokens that the group's sequences share, whole
 *              pages (a multiple of page_tokens, at most table_width * page_tokens). They are
 *              looked up in the table's row of the group's FIRST sequence (which need not have
 *              rows); the others' entries for them are not read. 0: nothing is shared.
 *   workspace  cache_attention_shared_workspace_size bytes, otherwise as there.
 * Row j of sequence s, at position p = lengths[s] - n + j, sees the shared[g] tokens and its
 * sequence's own from there to p: with table rows that begin alike the result is
 * cache_attention_forward's, up to the order of sums. Rows lie behind what their sequence shares
 * (lengths[s] - n >= shared[g]); a sequence with rows that do not is left out and
 * csa_get_status reports CSA_ERR_INDEX, as is a group whose shared[g] breaks the rules; where the
 * bounds in `groups` do, nothing is computed. Numerics, outputs, in-place use, rows past the last
 * sequence's and the fixed order of sums as cache_attention_forward: in both parts weights are
 * rounded to fp16 for the product with V, relative to the largest that the part has seen so far;
 * maxima, sums and outputs of the parts, and their joining, are fp32. rows * q_heads up to 2^30.
 * For batches that share little cache_attention_forward is faster: one group of single tokens gains
 * from about 100 MB of codes that are not read again, groups of a few sequences each from more.
 *
 * cache_attention_shared_workspace_size -- bytes of workspace it needs for batches of up to this
 * many rows, sequences and groups, into *bytes: 556 bytes (heads of up to 64) or 1068 for each
 * row and query head, beside 26 or 51 MB whatever the batch. Host only.
 *
 * csa_set_shared_part -- process-wide, for later calls: whether what sequences share is worked out
 * apart where it keeps enough from being read again (CSA_SHARED_AUTO: from about 32 MB of codes,
 * decided on the device, from the lengths; elsewhere each sequence reads it for itself) or always (CSA_SHARED_ALWAYS). The function is the same, sums
 * are taken in another order. CSA_ERR_SHAPE for an unknown mode (the mode is unchanged).
 */
#define CSA_SHARED_AUTO   0
#define CSA_SHARED_ALWAYS 1
csa_status csa_set_shared_part(int mode);
csa_status cache_attention_shared_workspace_size(const csa_kv_cache* cache, int q_heads, int rows,
                                                 int sequences, int group_count, size_t* bytes);
csa_status cache_attention_shared_forward(void* out, const void* q, int dtype, int q_heads,
                                          int64_t out_token_stride, int64_t out_head_stride,
                                          int64_t q_token_stride, int64_t q_head_stride,
                                          const csa_kv_cache* cache, const csa_kv_batch* batch,
                                          const int32_t* groups, const int32_t* shared,
                                          int group_count, float scale, void* workspace,
                                          size_t workspace_bytes, void* stream);

/*
 * csa_kv_pages -- the books of a cache: which pages each of `sequences` places has.
 *   refs         device, int32 [pages]: how many table entries name each page, 0: free;
 *   lengths      device, int32 [sequences]: tokens of each place's sequence, 0: none there;
 *   table        device, int32 [sequences][table_width]: block b of a sequence (tokens
 *                b * page_tokens on) is page table[s][b]; entries past a length mean nothing.
 * New books are zeros in refs and lengths; the calls below keep them in step. A csa_kv_batch over
 * all places uses the same lengths and table (places without rows in a call have equal offsets).
 * Whole pages may be shared, a page that is written to never is. Who names pages beside the
 * tables (a store of prompts) adds to their refs. refs, lengths and table do not overlap.
 *
 * All of these run on the device, asynchronous on `stream`, and may be captured; none allocates.
 * Lists of entries are device int32 arrays of n >= 1. An entry that breaks a rule is left out and
 * csa_get_status reports CSA_ERR_INDEX: a place outside [0, sequences), a length outside
 * [0, table_width * page_tokens] or past 2^31 - 1 before or after, a page outside [0, pages) (skipped), a place
 * that an earlier entry of the call extends or forks into. Free pages are given out lowest number
 * first, in the order of the entries; an entry for which too few are left, as if all entries before
 * it had got theirs, is left as it was and reported as CSA_ERR_PAGES.
 *
 * kv_pages_extend -- room for more[i] >= 0 more tokens of sequences[i]: its length grows by them
 * and pages are given to the blocks that it had none for (a place of length 0 begins a sequence).
 * What the pages hold is for kv_cache_write to write.
 *
 * kv_cache_fork -- children[i], a place of length 0, becomes a sequence of the first tokens[i]
 * tokens of parents[i] (tokens NULL: of all of them). Whole pages are shared, their refs grow; where
 * the last one is whole only in part, its written slots and its scales are copied to a page of the
 * child's own. A parent may have any number of children; a place is not both in one call. (A
 * sequence is shortened by forking its first tokens and ending it: a length alone must not be
 * lowered into a page that others share.)
 *
 * kv_pages_free -- sequences[i] ends: its length becomes 0 and the refs of its pages go down by
 * one each; those that reach 0 are free. A place named twice, or of length 0, has nothing to end.
 *
 * kv_cache_copy -- page to_pages[i] of `to` becomes a copy of page from_pages[i] of `from` (codes
 * of all slots, scales). Caches of the same heads, page_tokens, head_size and format, or one
 * cache; no page may be named twice in to_pages, nor in both lists of one cache (which of the
 * contents it has then is not said).
 *
 * kv_cache_compact -- with n pages in use (refs above 0), those from n on move to the free ones
 * below n, both in ascending order: codes, scales and refs, and every sequence's table entries.
 * Afterwards pages 0 .. n - 1 are in use and the rest free.
 *   moves    device, int32 [pages]: each page's new number, -1 for those that were free;
 *   in_use   device, int32 [1]: n. They overlap neither the books nor each other.
 *
 * kv_pages_workspace_size -- bytes of workspace that kv_pages_extend and kv_cache_fork with up to
 * n entries and kv_cache_compact need, into *bytes (host only; n >= 0). The workspace: device,
 * 16-byte aligned, needs no clearing, in use until the call's kernels complete: calls that may
 * overlap on the GPU, replays of captured ones too, need separate ones.
 */
typedef struct csa_kv_pages {
  int32_t* refs;
  int32_t* lengths;
  int32_t* table;
  int pages, sequences, table_width, page_tokens;
} csa_kv_pages;

csa_status kv_pages_workspace_size(const csa_kv_pages* pages, int n, size_t* bytes);
csa_status kv_pages_extend(const csa_kv_pages* pages, const int32_t* sequences,
                           const int32_t* more, int n, void* workspace, size_t workspace_bytes,
                           void* stream);
csa_status kv_cache_fork(const csa_kv_cache* cache, const csa_kv_pages* pages,
                         const int32_t* parents, const int32_t* children, const int32_t* tokens,
                         int n, void* workspace, size_t workspace_bytes, void* stream);
csa_status kv_pages_free(const csa_kv_pages* pages, const int32_t* sequences, int n, void* stream);
csa_status kv_cache_copy(const csa_kv_cache* to, const csa_kv_cache* from,
                         const int32_t* to_pages, const int32_t* from_pages, int n, void* stream);
csa_status kv_cache_compact(const csa_kv_cache* cache, const csa_kv_pages* pages, int32_t* moves,
                            int32_t* in_use, void* workspace, size_t workspace_bytes,
                            void* stream);

/*
 * token_logprobs_forward -- for each row x of logits (a dense layer's outputs) and its token,
 * with p = softmax(scale x):
 *   logprob[r]    log p[tokens[r]];
 *   entropy[r]    -sum_j p_j log p_j;
 *   stats[r]      (m, log sum_j exp(scale (x_j - m))), m the largest x: what the backward call
 *                 needs; their log-sum-exp is scale m + stats[r][1];
 *   top_token[r][0 .. top - 1], top_logprob[r][...]   the tokens of the largest x in falling
 *                 order, of equal ones the lowest number first (-0 equals 0), and their log p.
 *   logits       device, CSA_BF16, CSA_F16 or CSA_F32, [rows][vocab], rows `stride` elements
 *                apart (>= vocab; any alignment of the type);
 *   tokens       device, int32 [rows]; a negative one leaves its row out: its logits do not
 *                matter, its results are 0 and its top tokens -1. So does one from vocab on, which
 *                csa_get_status reports as CSA_ERR_INDEX;
 *   scale        1 / temperature: > 0, at most 2^64;
 *   logprob, entropy   device, fp32 [rows]; stats device, fp32 [rows][2], 8-byte aligned;
 *   top          0 .. min(32, vocab); top_logprob fp32 and top_token int32, [rows][top] (unused
 *                and may be NULL with top = 0).
 * Computed in fp32 (the difference to m first, so that log p near 0 is exact to fp32's
 * 2^-24 of the sum, not of m; the sums in runs of at most 512 16-byte groups of words and a sum of
 * such runs, whatever the vocabulary: their roundings are below 2^-14 of them at 2^27 words). A logit of -inf is a forbidden token: p = 0, nothing added to the
 * entropy. Where every logit of a row is -inf, log p is -inf, the entropy 0 and stats (-inf, 0).
 * A NaN or +inf makes its row's logprob, entropy and top_logprob NaN; among the top tokens a NaN
 * counts as -inf. Outputs must not overlap the inputs or each other (CSA_ERR_UNSUPPORTED; that
 * logprob and the alternatives' two are apart is not checked). Asynchronous on `stream`;
 * results do not depend on an SM limit beyond the order in which fp32 sums are taken.
 *
 * token_logprobs_backward -- the gradient of sum_r d_logprob[r] logprob[r] + d_entropy[r]
 * entropy[r] + sum_i d_top[r][i] top_logprob[r][i] by the logits, rounded once to their type:
 *   dlogits[r][j] = scale (g 1{j = token} - d_entropy p_j (log p_j + entropy)
 *                          + sum_i d_top[i] 1{j = top_token[i]} - (d_logprob + sum_i d_top[i]) p_j).
 *   stats, entropy     as the forward call left them (same logits, tokens and scale);
 *   d_logprob, d_entropy [rows], d_top [rows][top]   device, fp32; any may be NULL (no such
 *                term; top_token is read with d_top only);
 *   dlogits      device, of the logits' type, rows d_stride apart; the logits themselves with
 *                equal strides (in place), or apart from them (CSA_ERR_UNSUPPORTED otherwise);
 *                apart from the other arrays (the same).
 * Every element of dlogits is written: 0 in rows left out and in rows with every logit -inf.
 * The choice of the alternatives has no gradient. Asynchronous on `stream`.
 */
csa_status token_logprobs_forward(float* logprob, float* entropy, float* stats, const void* logits,
                                  int dtype, int64_t rows, int vocab, int64_t stride,
                                  const int32_t* tokens, float scale, int top, float* top_logprob,
                                  int32_t* top_token, void* stream);
csa_status token_logprobs_backward(void* dlogits, const void* logits, int dtype, int64_t rows,
                                   int vocab, int64_t d_stride, int64_t stride,
                                   const int32_t* tokens, float scale, const float* stats,
                                   const float* entropy, const float* d_logprob,
                                   const float* d_entropy, int top, const float* d_top,
                                   const int32_t* top_token, void* stream);

/*
 * csa_get_status -- synchronises `stream`, then returns and clears the current
 * device's status word: CSA_OK, or CSA_ERR_TIMEOUT if a kernel's bounded wait
 * ran out since the last call, or CSA_ERR_INDEX if a kernel met an index out of range
 * (see csa_kv_batch, csa_kv_pages), or CSA_ERR_PAGES if one found too few free pages: the first
 * of them since. Returns CSA_ERR_CUDA if synchronisation fails.
 */
csa_status csa_get_status(void* stream);

/* csa_status_string -- static description of a status code (never NULL). */
const char* csa_status_string(csa_status s);

/* csa_last_error -- text of the last failure on this host thread ("" if none). */
const char* csa_last_error(void);

/* csa_version -- library version string, e.g. "0.1.0 sm_103a". */
const char* csa_version(void);

/*
 * Watchdog controls, for tests of the failure path (no GPU fault involved).
 *
 * csa_set_wait_limit_ns -- upper bound, in nanoseconds of %globaltimer, on
 *   every spin-wait inside the kernels (0 restores the default: 2e9 = 2 s, or
 *   the environment variable CSA_WAIT_LIMIT_NS when it holds a positive integer,
 *   read once at the first launch or query).
 * csa_get_wait_limit_ns -- the bound the next launch will use.
 * csa_debug_inject -- when nonzero, the next kernel launch (any entry point)
 *   withholds one hand-off in every CTA: the first operand load (score
 *   products, the softmax's first Q tile, the dense layer's TMA form, the first codes of
 *   attention over prompts and over a shared part) or the first stage arrival (the dense layer's loader-warp
 *   forms), so a bounded wait
 *   downstream runs out; the kernel records CSA_ERR_TIMEOUT and returns with its
 *   output incomplete. Consumed by that launch (kernels without such waits, those of
 *   the rotary, cache, pages and logits calls and of attention for few rows, leave it set).
 */
void csa_set_wait_limit_ns(uint64_t ns);
uint64_t csa_get_wait_limit_ns(void);
void csa_debug_inject(int enable);

/*
 * Stream holds, for tests of launches that wait on the host (no GPU wait involved).
 *
 * csa_debug_hold_stream -- enqueues on `stream` a host function that returns once
 *   csa_debug_release_streams is called (or after 10 s): work enqueued behind it
 *   starts only then. CSA_ERR_CUDA if the host function cannot be enqueued.
 * csa_debug_release_streams -- releases every hold enqueued so far.
 */
csa_status csa_debug_hold_stream(void* stream);
void csa_debug_release_streams(void);

#ifdef __cplusplus
}
#endif

#endif /* CSA_GB300_H */
