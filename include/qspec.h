/*
 * qspec.h -- C ABI of libqspec.so, the GB300 (sm_103a) hot path of QSpec-style quantized
 * speculative decoding.
 *
 * The method (QSpec, as described in "QSpec実行時の2つの量子化による推論の一致率を調べる",
 * qiita.com/joule, sections "W4A4 と W4A16 量子化" and "QSpec の W4A4 モードと W4A16 モード"):
 * one set of 4-bit weights serves two modes.  The draft mode (W4A4) also quantises activations
 * to 4 bits; the verify mode (W4A16) keeps 16-bit activations and converts the 4-bit weights while
 * multiplying.  Drafted tokens are then checked against the verify-mode distribution with the
 * standard speculative-decoding rules ("Speculative Decodingとは？LLM生成を速くする方法",
 * kasblo.com, sections "greedy decodingでは一致するprefixを採用する" and
 * "samplingでもtargetの確率分布を保つ", eqs. a(x) and p'(x)).
 *
 * Conventions for every entry point:
 *  - All tensor pointers are DEVICE pointers owned by the caller, row-major and contiguous.
 *    bfloat16 and float16 tensors are passed as uint16_t bit patterns.
 *  - Every base pointer must be 16-byte aligned (QSPEC_ERR_MISALIGNED otherwise).
 *  - Work is enqueued asynchronously on `stream` (NULL = legacy default stream).  No entry point
 *    synchronises except qspec_check_status, and none allocates or frees device memory.
 *  - Argument checks happen on the host before anything is enqueued; on failure nothing is
 *    enqueued and the status says why.  Launch failures return QSPEC_ERR_CUDA.
 *  - Outputs must not alias inputs.
 *  - Calls are thread-safe.  Calls that share a verify workspace must not overlap on the GPU.
 */
#ifndef QSPEC_H_
#define QSPEC_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

struct CUstream_st;                       /* same type as cudaStream_t */
typedef struct CUstream_st* qspec_stream_t;

typedef enum {
  QSPEC_OK = 0,
  QSPEC_ERR_INVALID_ARG = 1,        /* null pointer, negative or zero size, bad token id        */
  QSPEC_ERR_UNSUPPORTED_SHAPE = 2,  /* size outside the documented limits                        */
  QSPEC_ERR_MISALIGNED = 3,         /* a base pointer is not 16-byte aligned                     */
  QSPEC_ERR_WORKSPACE = 4,          /* workspace missing, too small, or laid out for another shape */
  QSPEC_ERR_CUDA = 5,               /* a CUDA runtime/driver call or a launch failed             */
  QSPEC_ERR_TIMEOUT = 6             /* a kernel gave up a bounded wait and returned early        */
} qspec_status;

/* Limits checked by every call. */
#define QSPEC_GROUP 128             /* input channels per weight scale                           */
#define QSPEC_MAX_M 4096            /* tokens per linear call                                    */
#define QSPEC_MAX_GAMMA 16          /* draft length                                              */
#define QSPEC_MAX_V (1 << 24)       /* vocabulary                                                */
#define QSPEC_MAX_TREE 64           /* candidate nodes of a verification tree                    */

/*
 * qspec_pack_weights -- symmetric per-group INT4 weight quantiser and packer (step a1).
 *
 * The pages fix only "4-bit weights shared by both modes" (QSpec article, section
 * "QSpec の W4A4 モードと W4A16 モード"); the quantiser is the plain symmetric one:
 * for each row n and group g of 128 consecutive input channels,
 *     s[n,g]    = fp16( amax_g |W| / 7 )                   (fp32 IEEE division, round to fp16)
 *     code[n,k] = clamp( rint( W[n,k] / float(s[n,g]) ), -8, 7 )   (fp32 IEEE division, ties even)
 * with all codes 0 when s == 0.  Codes are two's complement nibbles; the 32-bit little-endian word
 * t of row n (bytes Wp[n, 4t..4t+3]) holds channels k = 8t..8t+7 with the even channels
 * 8t+0, 2, 4, 6 in nibbles 0..3 (bits 0..15) and the odd channels 8t+1, 3, 5, 7 in nibbles 4..7
 * (bits 16..31).  This packed format is the format both linear calls read.
 *
 *   W   [N, K] bf16 (input), K % 128 == 0, 1 <= N, N*K < 2^40
 *   Wp  [N, K/2] uint8 (output)
 *   S   [N, K/128] fp16 (output)
 * The result is bit-exact (independent of launch configuration).
 */
qspec_status qspec_pack_weights(const uint16_t* W, int64_t N, int64_t K, uint8_t* Wp, uint16_t* S,
                                qspec_stream_t stream);

/*
 * qspec_linear_w4a16 -- verify-mode linear (step a2): y = x . dequant(Wp, S)^T.
 *
 * QSpec article, section "W4A16: 重みのみを 4-bit に量子化": 4-bit weights are converted to
 * 16-bit values during the product with 16-bit activations.
 *     y[m,n] = sum_k x[m,k] * code[n,k] * s[n, k/128]
 * The codes are converted to bf16 exactly, products of each 128-channel group are summed in fp32
 * and scaled by s[n,g]; y is rounded to bf16 once.
 *
 *   x  [M, K] bf16, Wp [N, K/2] uint8, S [N, K/128] fp16 (from qspec_pack_weights)
 *   y  [M, N] bf16 (output)
 *   ws, ws_bytes  device workspace, >= qspec_linear_workspace_size(M, N, K), zero-filled before its
 *                 first use; it holds the per-tile tickets and partial sums of output tiles whose K
 *                 range is split between SMs, and the W4A4 activation codes.  A call leaves the
 *                 workspace ready for the next call OF THE SAME (M, N, K); its layout depends on the
 *                 shape, so calls of different shapes (for instance the layers of a model) need
 *                 workspaces of their own, or a zero-fill in between.  The workspace's header records
 *                 the (M, N, K) of the first call that uses its regions; a later call of another shape
 *                 that would use them touches neither the workspace nor y and makes the next
 *                 qspec_check_status return QSPEC_ERR_WORKSPACE.  (Calls whose kernels use no region,
 *                 such as one to three tokens on the decode-size path when K fits on chip, run on
 *                 any large-enough workspace.)
 *   1 <= M <= 4096, N % 8 == 0, K % 128 == 0; QSPEC_ERR_UNSUPPORTED_SHAPE for the (very large)
 *   shapes whose tensor-core work units would not fit 32-bit counters, and QSPEC_ERR_CUDA if the
 *   driver offers no tensor-map encoder (there is no other path).
 * The fp32 summation order depends on the device's SM count, so results are reproducible on one
 * device but may differ in the last bits between devices.
 */
qspec_status qspec_linear_w4a16(const uint16_t* x, const uint8_t* Wp, const uint16_t* S, int64_t M,
                                int64_t N, int64_t K, uint16_t* y, void* ws, size_t ws_bytes,
                                qspec_stream_t stream);

/*
 * qspec_linear_w4a4 -- draft-mode linear (steps a3 + a4) with the activation quantiser fused.
 *
 * QSpec article, section "W4A4 : 重みと活性値の両方を 4-bit に量子化": activations are also
 * quantised to 4 bits, so the product runs on 4-bit operands.  Per token m (all of K):
 *     s_a[m]    = amax_k |x[m,k]| / 7                     (fp32 IEEE division, kept in fp32)
 *     qa[m,k]   = clamp( rint( x[m,k] / s_a[m] ), -8, 7 ) (fp32 IEEE division, ties even; 0 if s_a==0)
 *     acc[m,n,g]= sum_{k in group g} qa[m,k] * code[n,k]  (exact integer)
 *     y[m,n]    = s_a[m] * sum_g float(s[n,g]) * acc[m,n,g]   (fp32, rounded to bf16 once)
 *
 *   x, Wp, S, y, M, N, K, ws, ws_bytes as for qspec_linear_w4a16 (the SAME Wp and S serve both modes).
 *   xq_out  [M, K] int8 codes qa, or NULL              (bit-exact)
 *   xs_out  [M] fp32 scales s_a, or NULL               (bit-exact)
 *   acc_out [M, N, K/128] int32 group sums, or NULL    (bit-exact; debugging aid)
 */
qspec_status qspec_linear_w4a4(const uint16_t* x, const uint8_t* Wp, const uint16_t* S, int64_t M,
                               int64_t N, int64_t K, uint16_t* y, int8_t* xq_out, float* xs_out,
                               int32_t* acc_out, void* ws, size_t ws_bytes, qspec_stream_t stream);

/*
 * qspec_linear_w4a8 -- the W4A8 configuration (step f3): qspec_linear_w4a4 with 8-bit activations.
 *
 * The speculative-decoding-with-quantisation summary (aibr.jp), section "中核となる技術的要素",
 * names W4A8 beside W4A16 as a weight/activation configuration; it gives no quantiser, so this one
 * is the W4A4 quantiser at 8 bits, on the same packed 4-bit weights:
 *     s_a[m]    = amax_k |x[m,k]| / 127                     (fp32 IEEE division, kept in fp32)
 *     qa[m,k]   = clamp( rint( x[m,k] / s_a[m] ), -128, 127 ) (fp32 IEEE division, ties even)
 *     acc, y    as for qspec_linear_w4a4 (|acc| <= 131072: exact)
 *   Arguments, outputs and limits as qspec_linear_w4a4.
 */
qspec_status qspec_linear_w4a8(const uint16_t* x, const uint8_t* Wp, const uint16_t* S, int64_t M,
                               int64_t N, int64_t K, uint16_t* y, int8_t* xq_out, float* xs_out,
                               int32_t* acc_out, void* ws, size_t ws_bytes, qspec_stream_t stream);

/*
 * qspec_linear_group -- several linears that read the same activations, in one launch and one mode
 * (steps a2, a3 + a4, or the W4A8 configuration of f3): e.g. the q, k and v projections of a
 * decoder layer, or its gate and up projections.
 *
 * QSpec article, section "QSpec の W4A4 モードと W4A16 モード": both modes read the same packed weights.
 * Part i computes exactly what qspec_linear_w4a16 / _w4a4 / _w4a8 compute for (x, Wp_i, S_i):
 *     y_i = x . dequant(Wp_i, S_i)^T          (abits = 16)
 *     y_i = s_a . sum_g s . acc               (abits = 4 or 8, x quantised once per token)
 * with the same definitions and tolerances (the fp32 summation order may differ in the last bits).
 * The parts' rows stream as one run of 16-row tiles, so the launch, the activation staging and the
 * per-token quantisation are paid once for the group.
 *
 *   abits     16 (W4A16), 4 (W4A4) or 8 (W4A8)
 *   x         [M, K] bf16, 1 <= M <= QSPEC_GROUP_MAX_M, K % 128 == 0
 *   parts     HOST array of n_parts descriptors, 1 <= n_parts <= QSPEC_GROUP_MAX_PARTS; each:
 *               Wp [N, K/2] uint8, S [N, K/128] fp16 (from qspec_pack_weights), y [M, N] bf16
 *               (output), N % 8 == 0; read during the call
 *   ws, ws_bytes  device workspace, >= qspec_linear_group_workspace_size(M, parts, n_parts, K),
 *             zero-filled before its first use; its header records the layout as (M, R, K), R = 16
 *             x the parts' 16-row tiles (QSPEC_ERR_WORKSPACE for a workspace laid out otherwise)
 * Shapes the decode-size kernel does not serve return QSPEC_ERR_UNSUPPORTED_SHAPE (call the parts
 * one by one then).
 */
#define QSPEC_GROUP_MAX_PARTS 4
#define QSPEC_GROUP_MAX_M 4
typedef struct {
  const uint8_t* Wp;
  const uint16_t* S;
  uint16_t* y;
  int64_t N;
} qspec_linear_part;
size_t qspec_linear_group_workspace_size(int64_t M, const qspec_linear_part* parts, int32_t n_parts, int64_t K);
qspec_status qspec_linear_group(int32_t abits, const uint16_t* x, int64_t M, int64_t K, const qspec_linear_part* parts,
                                int32_t n_parts, void* ws, size_t ws_bytes, qspec_stream_t stream);

/*
 * qspec_linear_pass -- one launch for a pass of decode-size linears in one mode (steps a2, a3 + a4,
 * or the W4A8 configuration of f3), e.g. every linear of a decoder layer and the lm_head.
 *
 * QSpec article, section "QSpec の W4A4 モードと W4A16 モード": a draft pass runs every linear of
 * the model in W4A4 mode and a verify pass runs them in W4A16 mode, over the same packed weights.
 * Each layer l of the pass computes exactly what qspec_linear_w4a16 / _w4a4 / _w4a8 compute for it
 * (same definitions, same tolerances; the fp32 summation order may differ in the last bits):
 *     y_l = x_l . dequant(Wp_l, S_l)^T          (abits = 16)
 *     y_l = s_a . sum_g s . acc                  (abits = 4 or 8, x_l quantised per token)
 * The layers run in order on one persistent grid (one CTA per SM): the weight stream continues
 * across layer boundaries and the next layer's activations are copied on chip while the current
 * layer streams.  A layer with `after` set reads what earlier layers of the pass wrote: every CTA
 * finishes the earlier layers and waits for all others (a grid-wide barrier with an iteration limit;
 * if it expires, the pass stops and qspec_check_status returns QSPEC_ERR_TIMEOUT).  Without `after`,
 * a layer's x must not be the y of an earlier layer of the same pass.
 *
 *   abits     16 (W4A16), 4 (W4A4) or 8 (W4A8)
 *   M         tokens, 1 <= M <= QSPEC_PASS_MAX_M (the same for every layer)
 *   layers    HOST array of n_layers descriptors, 1 <= n_layers <= QSPEC_PASS_MAX_LAYERS; each:
 *               x [M, K] bf16, Wp [N, K/2] uint8, S [N, K/128] fp16 (from qspec_pack_weights),
 *               y [M, N] bf16 (output); N % 8 == 0, K % 128 == 0, and the staged activations must
 *               fit on chip: slots(M) * K <= 102400 with slots(M) = 1, 2, 4 for M = 1, 2, 3..4
 *               (K <= 25600 at M = 4); `reserved` must be 0
 *   ws, ws_bytes  device workspace of >= qspec_linear_pass_workspace_size() bytes, zero-filled
 *             before its first use (it holds the grid barrier's counters, which every pass leaves
 *             ready for the next); passes that share a workspace must not overlap on the GPU
 * The descriptors are read during the call (they may be reused or freed when it returns).
 */
#define QSPEC_PASS_MAX_LAYERS 16
#define QSPEC_PASS_MAX_M 4
typedef struct {
  const uint16_t* x;
  const uint8_t* Wp;
  const uint16_t* S;
  uint16_t* y;
  int64_t N, K;
  int32_t after;     /* nonzero: this layer reads outputs of earlier layers of the pass */
  int32_t reserved;  /* must be 0 */
} qspec_pass_layer;
size_t qspec_linear_pass_workspace_size(void);
qspec_status qspec_linear_pass(int32_t abits, int64_t M, const qspec_pass_layer* layers, int32_t n_layers,
                               void* ws, size_t ws_bytes, qspec_stream_t stream);

/*
 * qspec_linear_workspace_size -- bytes of device workspace the linear calls need for an [M, K] x
 * [N, K] product on the CURRENT device (the size depends on its SM count).  0 for invalid sizes.
 */
size_t qspec_linear_workspace_size(int64_t M, int64_t N, int64_t K);

/*
 * qspec_verify_workspace_size -- bytes of device workspace that the verify calls need for the
 * given shape.  The workspace must be zero-filled before its first use (e.g. one cudaMemset
 * after allocation); every call leaves it ready for the next call.  Returns 0 for invalid sizes.
 */
size_t qspec_verify_workspace_size(int32_t B, int32_t gamma, int32_t V);

/*
 * qspec_verify_greedy -- greedy verification (steps a5 + a6).
 *
 * Tutorial, section "greedy decodingでは一致するprefixを採用する": draft tokens are compared left
 * to right with the target's most likely token; the matching prefix is accepted, the first
 * mismatching position takes the target's token instead, and when every draft token matches the
 * target's token for the following position is added (at most gamma+1 tokens per call).
 *     t[b,i] = argmax_j tgt_logits[b,i,j]    (lowest index among equal maxima; +0 == -0)
 *     n[b]   = largest k <= gamma with d[b,i] == t[b,i] for all i < k
 *     out[b] = (d[b,0..n-1], t[b,n], -1, ...)
 *
 *   tgt_logits [B, gamma+1, V] bf16   target logits at the gamma draft positions and the next one
 *   draft_tok  [B, gamma] int32       draft tokens; ids outside [0, V) never match and raise
 *                                     QSPEC_ERR_INVALID_ARG at the next qspec_check_status
 *   accept_len [B] int32 (output)     n
 *   out_tok    [B, gamma+1] int32 (output)
 *   tgt_argmax [B, gamma+1] int32 (output) or NULL
 *   ws, ws_bytes                      device workspace, >= qspec_verify_workspace_size(B,gamma,V)
 *   1 <= B, 1 <= gamma <= 16, 2 <= V <= 2^24, B*(gamma+1)*V < 2^40.  Bit-exact.
 */
qspec_status qspec_verify_greedy(const uint16_t* tgt_logits, const int32_t* draft_tok, int32_t B,
                                 int32_t gamma, int32_t V, int32_t* accept_len, int32_t* out_tok,
                                 int32_t* tgt_argmax, void* ws, size_t ws_bytes,
                                 qspec_stream_t stream);

/*
 * qspec_verify_sample -- sampling verification (steps a5, a7, a8).
 *
 * Tutorial, section "samplingでもtargetの確率分布を保つ": with p the target distribution and q the
 * draft distribution (softmax of the logits, temperature 1, computed in fp32), draft token x at
 * position i is accepted with probability a(x) = min(1, p(x)/q(x)) (eq. a(x)); at the first
 * rejection n the emitted token is drawn from the residual max(0, p - q) / sum(...) (eq. p'(x));
 * when all gamma are accepted a bonus token is drawn from the target distribution at position
 * gamma.  The library draws no random numbers; the uniforms are inputs:
 *     accept position i      iff  u_accept[b,i] < a_i          (a_i = 1 when q(x) == 0)
 *     n[b]                   = first rejected position, or gamma
 *     j*                     = smallest j with sum_{i<=j} r_i > u_resample[b,n] * sum(r)
 *                              (r = residual of row n, or p of row gamma; r = p if sum is 0)
 *     out[b]                 = (d[b,0..n-1], j*, -1, ...)
 *
 *   tgt_logits   [B, gamma+1, V] bf16;  draft_logits [B, gamma, V] bf16;  draft_tok [B, gamma]
 *   u_accept     [B, gamma] fp32 in [0,1);  u_resample [B, gamma+1] fp32 in [0,1)
 *   accept_len [B], out_tok [B, gamma+1] int32 (outputs)
 *   accept_prob, p_tok, q_tok  [B, gamma] fp32 (outputs) or NULL: a_i, p_i(d_i), q_i(d_i) at every
 *                              draft position (also those after the first rejection)
 *   ws, ws_bytes as for qspec_verify_greedy.  Same size limits.
 */
qspec_status qspec_verify_sample(const uint16_t* tgt_logits, const uint16_t* draft_logits,
                                 const int32_t* draft_tok, const float* u_accept,
                                 const float* u_resample, int32_t B, int32_t gamma, int32_t V,
                                 int32_t* accept_len, int32_t* out_tok, float* accept_prob,
                                 float* p_tok, float* q_tok, void* ws, size_t ws_bytes,
                                 qspec_stream_t stream);

/*
 * qspec_verify_top1 -- top-1 statistics of the two modes at every draft position (step f2).
 *
 * Article "QSpec実行時の2つの量子化による推論の一致率を調べる", sections "実験：W4A4 と W4A16 の
 * Top-1 一致率を調べる" and "結果": at each draft position the W4A4 (draft) and W4A16 (target) modes
 * each have a most likely token and a probability for it (their own top-1; the two may differ).
 * The article reports how often the two tokens agree, each mode's mean top-1 probability, and the
 * agreement inside the region where both probabilities exceed 0.8 and where both are at most 0.8.
 *     tgt_top1[b,i]   = argmax_j tgt_logits[b,i,j]     (i < gamma; lowest index among equal maxima)
 *     draft_top1[b,i] = argmax_j draft_logits[b,i,j]
 *     tgt_p1[b,i]     = 1 / sum_j exp(tgt_logits[b,i,j] - max_j tgt_logits[b,i,j])   (fp32 softmax)
 *     draft_p1[b,i]   likewise for the draft row
 *
 *   tgt_logits   [B, gamma+1, V] bf16 (row gamma is not read);  draft_logits [B, gamma, V] bf16
 *   tgt_top1, draft_top1 [B, gamma] int32 (outputs)
 *   tgt_p1, draft_p1     [B, gamma] fp32 (outputs) or NULL
 *   high                 threshold of the high-confidence region (the article uses 0.8); not NaN
 *   tally                [8] fp64 or NULL: ACCUMULATED (added to, never cleared) over calls, so a
 *                        decode loop can keep one running tally on the device:
 *                        [0] positions, [1] agreeing positions, [2] positions with both p1 > high,
 *                        [3] agreeing among [2], [4] positions with both p1 <= high, [5] agreeing
 *                        among [4], [6] sum of tgt_p1, [7] sum of draft_p1.  Counts are exact; the
 *                        sums are fp64 sums of the fp32 probabilities in an unspecified order.
 *   ws, ws_bytes as for qspec_verify_greedy.  Same size limits.  Token ids are bit-exact;
 *   probabilities carry the fp32 softmax's rounding (within 1e-5 absolute of the exact value).
 */
qspec_status qspec_verify_top1(const uint16_t* tgt_logits, const uint16_t* draft_logits, int32_t B,
                               int32_t gamma, int32_t V, int32_t* tgt_top1, int32_t* draft_top1,
                               float* tgt_p1, float* draft_p1, float high, double* tally, void* ws,
                               size_t ws_bytes, qspec_stream_t stream);

/*
 * qspec_verify_tree_greedy -- greedy verification of a tree of candidates (step f4).
 *
 * The speculative-decoding-with-quantisation summary (aibr.jp), sections "先行研究との差別化
 * ポイント" and "中核となる技術的要素", names tree-style verification (candidates expanded as a tree;
 * its cost grows exponentially with the tree) without giving an algorithm.  This is the greedy rule
 * of qspec_verify_greedy carried over from a chain to a tree: node j (j < T) holds token
 * tree_tok[b,j] and parent tree_parent[b,j] (-1: the committed prefix; otherwise an earlier node,
 * parent < j).  Target row 0 scores the token after the prefix, row j + 1 the token after node j.
 *     t[r]  = argmax_v tgt_logits[b,r,v]                 (lowest index among equal maxima)
 *     walk: cur = prefix (row 0); while some child j of cur has tree_tok[b,j] == t[row of cur]:
 *           accept the lowest-index such j, cur = j (row j + 1)
 *     out[b] = (tokens of the accepted path, t[row where the walk stopped], -1, ...)
 * A chain (parent j - 1) reproduces qspec_verify_greedy.
 *
 *   tgt_logits   [B, T+1, V] bf16;  tree_tok, tree_parent [B, T] int32
 *   accept_len   [B] int32 (output) -- accepted nodes (depth of the path)
 *   out_tok      [B, T+1] int32 (output);  accept_nodes [B, T] int32 (output, node ids, -1 fill) or NULL
 *   ws, ws_bytes device workspace, >= qspec_verify_tree_workspace_size(B, T, V), zero-filled once;
 *                qspec_check_status(ws) reports invalid nodes (token outside [0, V) or a parent not in
 *                [-1, j-1]) as QSPEC_ERR_INVALID_ARG; such nodes never match.
 *   1 <= B, 1 <= T <= QSPEC_MAX_TREE, 2 <= V <= 2^24, B*(T+1)*V < 2^40.  Bit-exact.
 */
size_t qspec_verify_tree_workspace_size(int32_t B, int32_t T, int32_t V);
qspec_status qspec_verify_tree_greedy(const uint16_t* tgt_logits, const int32_t* tree_tok,
                                      const int32_t* tree_parent, int32_t B, int32_t T, int32_t V,
                                      int32_t* accept_len, int32_t* out_tok, int32_t* accept_nodes,
                                      void* ws, size_t ws_bytes, qspec_stream_t stream);

/*
 * qspec_verify_greedy_noalloc -- qspec_verify_greedy for callers that cannot allocate device memory.
 *
 * The pages have no counterpart of this entry point.  Some callers cannot call cudaMalloc where they
 * verify: plug-ins executing inside another runtime's fixed memory plan (a serving engine that
 * forbids allocation during a decode step), or C hosts with no allocator at hand.  This variant takes
 * no workspace: its scratch (error word, per-sequence tickets, per-chunk partial argmaxes) is a fixed
 * array of QSPEC_NOALLOC_SCRATCH_BYTES of device memory inside the library, which every GPU that
 * loads the library holds until the process exits.  It allocates nothing and calls no allocating
 * routine.
 *
 *   Arguments and results as qspec_verify_greedy (bit-identical outputs), without ws / ws_bytes.
 *   Size limit: with R = B*(gamma+1) rows and C chunks per row (C = 1 once R >= 1216, otherwise at
 *   most ceil(1216 / R) and at most ceil(V / 2048)), the call needs
 *       256 + round_up_256(4*B) + 8*R*C  <=  QSPEC_NOALLOC_SCRATCH_BYTES
 *   bytes; that is up to about 26 000 rows at gamma = 1 and 31 700 at gamma = 15.  Larger shapes are
 *   rejected with QSPEC_ERR_UNSUPPORTED_SHAPE before anything is enqueued.
 *   The first call in a CUDA context (normally once per device, in its primary context) looks up the
 *   array's device address with that context current and caches it for the context; make that first
 *   call before any stream capture.
 *   Every call shares the one array and clears its error word and tickets on `stream` first, so
 *   calls that overlap on the GPU (different streams, or concurrent graphs) race and must not be
 *   issued.  Draft-token range errors are not reported by qspec_check_status for this variant;
 *   out-of-range tokens simply never match.
 */
#define QSPEC_NOALLOC_SCRATCH_BYTES (256 * 1024)
qspec_status qspec_verify_greedy_noalloc(const uint16_t* tgt_logits, const int32_t* draft_tok,
                                         int32_t B, int32_t gamma, int32_t V, int32_t* accept_len,
                                         int32_t* out_tok, int32_t* tgt_argmax, qspec_stream_t stream);

/*
 * qspec_gather_rows -- dst[m, :] = src[idx[m], :] for m < n (step f1: embedding lookup of the tokens
 * a decode step feeds the model, and reordering of logits rows between [gamma, B] and [B, gamma]).
 *
 * Tutorial "Speculative Decodingとは？LLM生成を速くする方法", section "draft modelとtarget modelの
 * 処理フロー": each draft step feeds the token just chosen back into the model.
 *   src  [n_src, row_bytes] device;  idx [n] int32 device;  dst [n, row_bytes] device (no overlap
 *   with src).  row_bytes a multiple of 4; src, dst and idx 4-byte aligned, and src and dst 16-byte
 *   aligned when row_bytes is a multiple of 16 and at least 1024 (one CTA per row, 16-byte copies;
 *   shorter rows such as token ids take one thread per row); n <= 2^31 - 1.
 *   An id outside [0, n_src) writes a zero row and makes the next qspec_check_status return
 *   QSPEC_ERR_INVALID_ARG.
 */
qspec_status qspec_gather_rows(const void* src, int64_t n_src, int64_t row_bytes, const int32_t* idx,
                               int64_t n, void* dst, qspec_stream_t stream);

/*
 * qspec_select_tokens -- the next token of each of R logits rows (step f1: how a draft step, or a
 * plain target-only decode step, picks its token).
 *
 * Same section: the draft proposes its most likely token when decoding greedily and a draw from its
 * distribution q when sampling (temperature 1, fp32 softmax, inverse CDF in index order as in the
 * sampling verify):
 *     u == NULL:  tok[r] = argmax_j logits[r, j]    (lowest index among equal maxima; bit-exact)
 *     otherwise:  tok[r] = smallest j with sum_{i<=j} exp(l_i - m) > u[r] * sum_i exp(l_i - m)
 *                 (m = max_j l_j; if rounding leaves no such j, the last j with a nonzero term)
 *   logits [R, V] bf16 (16-byte aligned);  u [R] fp32 in [0,1) or NULL;  tok [R] int32 (output);
 *   u and tok 4-byte aligned.  One CTA per row.  2 <= V <= 2^24.  A row of only -inf gives token 0.
 */
qspec_status qspec_select_tokens(const uint16_t* logits, int32_t R, int32_t V, const float* u, int32_t* tok,
                                 qspec_stream_t stream);

/*
 * qspec_copy -- move `bytes` from src to dst with one kernel on the SMs (no copy engine).
 *
 * For a decode step's small per-step transfers (a few tokens' activations in, the verify results
 * out), where a copy-engine transfer is mostly fixed latency and the kernel after it cannot begin
 * until it ends.  Either pointer may be device memory or pinned (page-locked, host-allocated or
 * registered) host memory, which the kernel reads or writes through its device mapping over the
 * host link; pageable host memory is refused.  Launched with programmatic dependent launch: the
 * next kernel's prologue overlaps the copy; the copy writes dst only after the previous kernel in
 * the stream has finished, and reads a device-memory src only then too (a host src earlier).
 *
 *   dst, src  16-byte aligned, not overlapping; bytes > 0, a multiple of 16.
 * Returns QSPEC_ERR_INVALID_ARG for a null pointer, zero bytes or memory the GPU cannot address,
 * QSPEC_ERR_MISALIGNED for an address or size that is not a multiple of 16.
 */
qspec_status qspec_copy(void* dst, const void* src, size_t bytes, qspec_stream_t stream);

/*
 * ---------------------------------------------------------------------------------------------------
 * Around the linears: rotary positions, a paged 8-bit key/value cache, attention over it, and the
 * adjustment of the logits that a verify call reads.  The pages have no counterpart of these; they are
 * what a decoder layer and a serving loop put between the two linear modes and the verify step: in
 * one iteration every sequence adds gamma + 1 positions (or the nodes of a tree) to its cache, attends
 * over it at each of them, and shortens it again to what was accepted.
 */

/*
 * qspec_rotary_turns -- the frequencies of a rotary embedding, for qspec_rotary and qspec_kv_append.
 * A HOST function: writes rot/2 words and one float to host memory; the caller copies the words to the
 * device.  Word i is the rotation of pair i per position as a 64-bit fraction of a full turn, so
 * position * word modulo 2^64 is the angle with no error from range reduction, at any position.  (A word has the few
 * fp64 roundings of its frequency, 2^-53 each, which the position multiplies.)
 *     w_i = base^(-2 i / rot) radians per position, scaled for long contexts:
 *     QSPEC_ROTARY_PLAIN   w_i
 *     QSPEC_ROTARY_LINEAR  w_i / factor
 *     QSPEC_ROTARY_BASE    base replaced by base * factor^(rot / (rot - 2))
 *     QSPEC_ROTARY_BANDS   t_i = original w_i / (2 pi) turns over the trained context:
 *                          w_i / factor below `low` turns, w_i above `high`, linear in t_i between
 *     QSPEC_ROTARY_YARN    pairs that turn more than `high` times over the trained context keep w_i, those
 *                          that turn less than `low` times take w_i / factor, with a linear ramp over
 *                          the pair index between (edges rounded outwards to whole indices; the ramp
 *                          begins at pair 0 at the earliest, which keeps w_0 therefore);
 *                          *mult = 0.1 ln(factor) + 1
 *   rot even, 2 <= rot <= 1024 (rot >= 4 for QSPEC_ROTARY_BASE); base > 1; factor >= 1; original > 0;
 *   0 < low < high (BANDS and YARN; ignored otherwise)
 *   turns [rot/2] uint64 HOST (output);  mult HOST (output): factor on the rotated values, 1 unless YARN
 */
#define QSPEC_ROTARY_PLAIN 0
#define QSPEC_ROTARY_LINEAR 1
#define QSPEC_ROTARY_BASE 2
#define QSPEC_ROTARY_BANDS 3
#define QSPEC_ROTARY_YARN 4
qspec_status qspec_rotary_turns(int32_t rot, double base, int32_t scaling, double factor, double original,
                                double low, double high, uint64_t* turns, float* mult);

/* A rotary embedding on the device. */
typedef struct {
  const uint64_t* turns;  /* [rot/2] DEVICE, from qspec_rotary_turns                              */
  int32_t rot;            /* leading values of each head that rotate, even                        */
  int32_t interleaved;    /* 0: pairs (i, i + rot/2); 1: pairs (2i, 2i + 1)                       */
  float mult;             /* factor on the rotated values                                         */
  int32_t reserved;       /* must be 0                                                            */
} qspec_rotary_plan;

/*
 * qspec_rotary -- rotary positions: for every token, head and pair (a, b) with angle t = pos * w_i,
 *     (a, b) -> mult * (a cos t - b sin t, a sin t + b cos t);   values from rot on are copied.
 * With `inverse` the angle is negated (mult stays): the transpose of the forward rotation, which is its
 * backward pass.  Computed in fp32, rounded to bf16 once.
 *
 *   x    bf16, value d of head h of token t at x[t * x_token + h * x_head + d]
 *   pos  [T] int32 device, 4-byte aligned; any value, negative ones included
 *   out  as x with its own strides; out may be x itself with the same strides, else no overlap
 *        (no two of its rows may share memory: QSPEC_ERR_UNSUPPORTED_SHAPE; rows of x may)
 *   dim a multiple of 8, 8 <= dim <= 1024, rot <= dim; 1 <= heads <= 65535; strides non-negative multiples
 *   of 8 (QSPEC_ERR_MISALIGNED otherwise); T <= 2^31 - 1, every offset below 2^40
 */
qspec_status qspec_rotary(const uint16_t* x, int64_t x_token, int64_t x_head, const int32_t* pos, int64_t T,
                          int32_t heads, int32_t dim, const qspec_rotary_plan* plan, int32_t inverse,
                          uint16_t* out, int64_t out_token, int64_t out_head, qspec_stream_t stream);

/*
 * A paged key/value cache of 8-bit codes.  A page holds `page` consecutive tokens of one sequence; keys
 * and values of each (page, head) share one power-of-two scale each: value = e4m3(code) * 2^exp.
 *     k, v          [n_pages, heads, page, dim] uint8, e4m3 codes (finite ones: 0x7F and 0xFF do not occur)
 *     k_exp, v_exp  [n_pages, heads] int8, -40 .. 40 (QSPEC_KV_MIN_EXP .. QSPEC_KV_MAX_EXP)
 * page is 16, 32, 64 or 128; dim is 64 or 128.  Contents need no initialisation.
 */
#define QSPEC_KV_MIN_EXP (-40)
#define QSPEC_KV_MAX_EXP 40
#define QSPEC_KV_MAX_B 1024
typedef struct {
  uint8_t* k;
  uint8_t* v;
  int8_t* k_exp;
  int8_t* v_exp;
  int64_t n_pages;
  int32_t heads, page, dim;
  int32_t reserved;  /* must be 0 */
} qspec_kv_cache;

/*
 * The sequences of one step.  Sequence b owns the tokens cu_tok[b] .. cu_tok[b+1] - 1 of the step's T
 * new ones; they are the last ones of its kv_len[b] cached positions, in order.  Its cache position p lies
 * in page pages[b, p / page], slot p mod page.
 *     cu_tok  [B+1] int32, from 0 non-decreasing to at most T;  kv_len [B] int32;  pages [B, max_pages] int32
 * (all three DEVICE, 4-byte aligned; only the entries of pages that kv_len reaches are read).
 * max_tok: at least the largest number of new tokens of one sequence.  1 <= B <= QSPEC_KV_MAX_B,
 * 1 <= T < 2^31, 1 <= max_tok <= T, max_pages * page <= 2^30.
 * A sequence whose numbers are out of range, and a page id outside [0, n_pages), touch no memory outside
 * the arrays: the call leaves the sequence out (a bad page: its tokens), and the next
 * qspec_check_status returns QSPEC_ERR_INVALID_ARG.
 */
typedef struct {
  const int32_t* cu_tok;
  const int32_t* kv_len;
  const int32_t* pages;
  int32_t B, max_pages, max_tok;
  int32_t reserved;  /* must be 0 */
  int64_t T;
} qspec_kv_batch;

/*
 * qspec_kv_append -- write the step's keys and values into the cache; rotate keys and queries on the way.
 *     e(a)   the smallest exponent with a <= 448 * 2^e, limited to [-40, 40]
 *     per (page, head) that receives tokens, amax over the tokens that this call writes there:
 *       page begun by this call (its slot 0 is written):  exp = e(amax)
 *       otherwise:  exp = max(exp, e(amax)); where that raises it, the codes of the page's other slots are
 *                   quantised again: code = e4m3(code * 2^(old - new))
 *     code = e4m3(x * 2^-exp), round to nearest even, saturating
 * Dropping rejected tokens of a chain needs no call: use a smaller kv_len next time.  The accepted path of a tree is no
 * prefix of what was appended: qspec_kv_compact moves it there (or append its tokens' keys and values again).  A page's scale does
 * not shrink until the page is begun again, so tokens that were dropped leave a mark: where they raised the scale, the
 * codes of the page's other tokens have been rounded again (those alone that fell below e4m3's normal range change).
 * A non-finite key or value is stored as 0 and makes the next
 * qspec_check_status return QSPEC_ERR_INVALID_ARG.
 *
 *   k, v   bf16, value d of head h of token t at k[t * k_token + h * dim + d]
 *   plan   rotary embedding of the keys and queries (keys are rounded to bf16 before they are
 *          quantised), or NULL: none.  Its rot is a multiple of 16 unless pairs are interleaved
 *          (QSPEC_ERR_UNSUPPORTED_SHAPE otherwise)
 *   pos    [T] int32 device: each token's rotary position, or NULL: its cache position
 *   q      bf16 [T] tokens of heads_q * dim values, stride q_token, rotated into q_out (stride
 *          q_out_token; q_out may be q itself with the same stride), or NULL: no queries
 *          (heads_q is then ignored)
 * Token strides are multiples of 8 and at least heads * dim.  No other call may read or write the pages
 * at the same time; the pages written must belong to one sequence only.  Given rotated keys, bit-exact.
 */
qspec_status qspec_kv_append(const qspec_kv_cache* cache, const qspec_kv_batch* batch, const uint16_t* k,
                             int64_t k_token, const uint16_t* v, int64_t v_token, const qspec_rotary_plan* plan,
                             const int32_t* pos, const uint16_t* q, int64_t q_token, int32_t heads_q,
                             uint16_t* q_out, int64_t q_out_token, qspec_stream_t stream);

/*
 * qspec_kv_attention -- causal attention of the step's tokens over the cache (the step's own keys and
 * values included: append first).  For token i of a sequence with n new tokens and query head h, which
 * reads key head h / (heads_q / heads):
 *     p = kv_len - n + i                                   (its cache position)
 *     s_j = scale * q . k_j  for the visible j;   out = sum_j softmax(s)_j v_j;   lse = ln sum_j exp(s_j)
 *     visible:  j <= p, and j > p - window when window > 0;
 *     with a tree:  j < kv_len - n, or bit (j - (kv_len - n)) of the token's tree word is set (j < kv_len)
 * A token that sees nothing gets out = 0 and lse = -inf; a query with a NaN or an infinity that sees
 * anything gets out = lse = NaN.  Scores and softmax statistics are fp32; the
 * probabilities are rounded to fp16 for the product with the (exactly converted) codes, where a weight p_j 2^exp counts
 * down to 2^-33 of the largest that came with it; out is rounded to bf16 once.
 *
 *   q      bf16, value d of head h of token t at q[t * q_token + h * dim + d]
 *   window 0: none
 *   tree   [T] uint64 device, or NULL; needs max_tok <= 64 and window == 0
 *   out    bf16 as q with stride out_token; tokens beyond cu_tok[B] are not written
 *   lse    [T, heads_q] fp32 or NULL
 *   ws, ws_bytes  device workspace of >= qspec_kv_attention_workspace_size() bytes, zero-filled before
 *          its first use; it serves every shape and is left ready for the next call (after a wait that
 *          ran out, QSPEC_ERR_TIMEOUT, too: only the outputs are void then).  Calls that can overlap, on two
 *          streams, need one each
 *   heads_q a multiple of the cache's heads, at most 128 times them; |scale| <= 2^127; token strides multiples of
 *   8 and at least heads_q * dim
 */
size_t qspec_kv_attention_workspace_size(void);
qspec_status qspec_kv_attention(const qspec_kv_cache* cache, const qspec_kv_batch* batch, const uint16_t* q,
                                int64_t q_token, int32_t heads_q, float scale, int32_t window, const uint64_t* tree,
                                uint16_t* out, int64_t out_token, float* lse, void* ws, size_t ws_bytes,
                                qspec_stream_t stream);

/*
 * ---------------------------------------------------------------------------------------------------
 * Several continuations of one prompt: beams, samples, candidate trees.  The pages name tree-style candidates alone; these
 * calls choose continuations, let their sequences share pages of the cache, and read what they share once.
 */

/*
 * qspec_beam_select -- the n best continuations of each sequence's beams, by summed log probability:
 *     S(k, v) = scores[b,k] + (logit[b,k,v] - ln sum_v exp(logit[b,k,v]))     for every beam k and token v
 *     done[b,k] != 0: the beam offers itself alone, S = scores[b,k] with token end_tok
 * The n largest S(k, v) * weights[b,k], largest first; equal ones in the order of the beams, a beam's own offers in the order of
 * its logits, equal logits in the order of the tokens.  (weights: 1 / length penalty, for beams of different lengths.)
 *     parent = b * beams + k (a row of logits, and of what qspec_kv_pages and qspec_gather_rows reorder),  tok = v,  score = S
 * Where fewer than n are possible the rest are parent = tok = -1, score = -inf.  Logits of -inf and beams whose score is -inf
 * offer nothing (the logits of such a beam and of a finished one are not read).
 *
 *   logits [B, beams, V] bf16 (16-byte aligned);  scores [B, beams] fp32;  done [B, beams] int32 or NULL: none;
 *   weights [B, beams] fp32 or NULL: 1;  parent, tok [B, n] int32, score [B, n] fp32 (outputs;
 *          none of them over another array)
 *   ws, ws_bytes  device workspace, >= qspec_beam_workspace_size(B, beams, V, n), zero-filled before its first use and left ready for
 *          the next call, of any shape that it is large enough for: of every one that is no larger in any of B, beams, V and n.
 *          Calls that can overlap need one each
 *   1 <= beams <= QSPEC_BEAM_MAX_BEAMS, 1 <= n <= min(QSPEC_BEAM_MAX_N, beams * V), 2 <= V <= 2^24, B <= 65535,
 *   B*beams*V < 2^40; the other arrays 4-byte aligned
 * Sums of exponentials are fp32, of approximate powers: by trees within 8192 logits and one addition for each 8192 more.  In units of
 * 2^-24 of a sum the additions are within 25 + V / 8192; the terms' exponents within 3 ln V (a term's is off by three of its own
 * size, which under the weights of a softmax averages ln V at most); their powers, of a relative error below 2^-22, within 20 with
 * the three joinings, and 5 more for each time that the largest logit that a thread has seen rises (V / 8192 times at most).
 * Logarithms are within 2^-24, log probabilities and comparisons are fp64 and score is rounded to fp32 once.  Together S is within
 * 2^-16 for V = 152064, whatever the logits; two candidates of different beams can change places only where their S differ by less
 * than the two errors, those of one beam never.
 * A beam with a NaN or +inf among its logits, a score that is NaN or +inf, or a weight that is not positive and finite offers
 * nothing and makes the next qspec_check_status return QSPEC_ERR_INVALID_ARG.
 */
#define QSPEC_BEAM_MAX_BEAMS 32
#define QSPEC_BEAM_MAX_N 64
size_t qspec_beam_workspace_size(int32_t B, int32_t beams, int32_t V, int32_t n);
qspec_status qspec_beam_select(const uint16_t* logits, const float* scores, const int32_t* done, int32_t end_tok,
                               const float* weights, int32_t B, int32_t beams, int32_t V, int32_t n, int32_t* parent,
                               int32_t* tok, float* score, void* ws, size_t ws_bytes, qspec_stream_t stream);

/*
 * qspec_kv_pages -- the page tables of the next step: rows fork, move, shorten, grow, end or begin, in one call.
 * Row b of the old table holds ceil(room[b] / page) pages, pages[b, 0 ...].  Row r of the new one keeps the first keep[r]
 * positions of row parent[r] and has room for need[r] positions.  refs[p] counts who holds page p: each row that has it
 * in its table, and anyone else for whom the caller raised the count (kept prefixes).  A page of count 0 is free.
 *   - Kept pages are shared: their counts rise by one for each new row that has them; then all old rows are released.
 *   - Where keep[r] ends inside a page and need[r] > keep[r], row r will write in that page.  If all that hold it are such rows,
 *     the lowest of them keeps it; every other row gets a page of its own in its place, and (copy_src[r], copy_dst[r],
 *     copy_len[r]) = (page, its own page, keep[r] mod page) for qspec_kv_copy_pages.  Rows without a copy get (-1, -1, 0).
 *   - Fresh pages (copies first, then those up to need[r]) go to the rows in order, the free page of the lowest id first; pages
 *     that this call released count as free.
 *   - left = free pages that remain.  If they do not suffice, left is minus the number that lacks, the counts stay as they were,
 *     no copies are asked for and new_pages is of no use.
 *
 *   pages [rows, max_pages], room [rows]: rows may be 0 (both NULL then);  parent [new_rows], or NULL: row r comes from row r
 *   (negative: from none, with keep[r] = 0);  keep, need [new_rows]: 0 <= keep[r] <= room[parent[r]], keep[r] <= need[r];
 *   new_pages [new_rows, new_max_pages] (not the old table: entries beyond need[r] are left as they are);  refs, new_refs
 *   [n_pages], which may be the same array;  copy_src, copy_dst, copy_len [new_rows];  left [1].  new_rows may be 0 (its arrays
 *   NULL then: all rows end).  All int32, DEVICE, 4-byte aligned (refs and new_refs 16); but for refs in place no output
 *   overlaps another array.
 *   page is 16, 32, 64 or 128; rows and new_rows at most QSPEC_KV_MAX_B; max_pages * page <= 2^30
 * A row whose numbers are out of range gets no pages (an old one: releases none), an id outside [0, n_pages) is passed on without
 * being counted, and either of them or a count below zero makes the next qspec_check_status return QSPEC_ERR_INVALID_ARG.
 * Bit-exact.
 */
qspec_status qspec_kv_pages(const int32_t* pages, const int32_t* room, int32_t rows, int32_t max_pages, const int32_t* parent,
                            const int32_t* keep, const int32_t* need, int32_t new_rows, int32_t new_max_pages,
                            const int32_t* refs, int64_t n_pages, int32_t page, int32_t* new_pages, int32_t* new_refs,
                            int32_t* copy_src, int32_t* copy_dst, int32_t* copy_len, int32_t* left, qspec_stream_t stream);

/*
 * qspec_kv_copy_pages -- page src[i] -> page dst[i] in each of n_caches caches (the layers of a model, which share page tables):
 * the scales, and the codes of the first len[i] slots of every head (len NULL: of all).
 *   caches HOST array of n_caches descriptors of one shape, 1 <= n_caches <= QSPEC_KV_MAX_LAYERS (read during the call; deeper
 *          models take a call for each 64 of their layers)
 *   src, dst, len [n] int32 DEVICE, 4-byte aligned (n may be 0, all three NULL then); pairs with src[i] < 0 are skipped.  No
 *   dst[i] may be any other pair's src or dst
 * A pair with an id outside [0, n_pages) or a len[i] outside [0, page] copies nothing and makes the next qspec_check_status return
 * QSPEC_ERR_INVALID_ARG.
 */
#define QSPEC_KV_MAX_LAYERS 64
qspec_status qspec_kv_copy_pages(const qspec_kv_cache* caches, int32_t n_caches, const int32_t* src, const int32_t* dst,
                                 const int32_t* len, int32_t n, qspec_stream_t stream);

/*
 * qspec_kv_compact -- the accepted path of a tree becomes a prefix of what was appended, without its keys and values at hand.
 * The last n new tokens of sequence b (n = cu_tok[b+1] - cu_tok[b]) were appended as a tree: node j lies at position
 * kv_len - n + first + j (first = 1 where the token before the tree was appended with it).  For t < count[b] the cached keys and
 * values of node nodes[b, t] move to position kv_len - n + first + t, as if qspec_kv_append wrote their (dequantised) values there:
 * a page whose slot 0 is written takes the smallest scale that holds what it receives, another page's scale grows where it
 * must.  The sequence's length after it is kv_len - n + first + count[b].
 *   caches, n_caches  as for qspec_kv_copy_pages, none of them twice;  batch: as it was for the append
 *   nodes [B, T] int32, count [B] int32 DEVICE, 4-byte aligned: what qspec_verify_tree_greedy returns.  1 <= T <=
 *   QSPEC_MAX_TREE;  first >= 0;  nodes rising in [0, n - first), n - first <= QSPEC_MAX_TREE, count[b] <= min(T, n - first)
 * A sequence whose numbers, nodes or pages are out of range is left as it is and makes the next qspec_check_status return
 * QSPEC_ERR_INVALID_ARG.  The pages of the tree must belong to one sequence only.  Bit-exact.
 */
qspec_status qspec_kv_compact(const qspec_kv_cache* caches, int32_t n_caches, const qspec_kv_batch* batch, const int32_t* nodes,
                              const int32_t* count, int32_t T, int32_t first, qspec_stream_t stream);

/*
 * qspec_kv_attention_shared -- qspec_kv_attention for sequences that share a prefix, which is read and multiplied once for all of
 * them.  Group g is the sequences cu_seq[g] .. cu_seq[g+1] - 1; the first len[g] cache positions of all of them hold the same
 * tokens, and are read through the page table of the group's first sequence that has new tokens: entries of pages that lie wholly in the
 * prefix are not read in the others' tables.  (A group of one sequence, or of any sequences with len = 0, is plain attention.)
 * len[g] may exceed what its sequences have in common with their new tokens taken off: the prefix ends where the new tokens of one
 * of them begin, at the latest.
 * It pays for prefixes of some thousand positions that are longer than what the sequences have alone: its start takes longer than
 * qspec_kv_attention's, and keys of one sequence take twice as long in groups of more than 32 rows.  With 32 query heads on 8 of 128
 * it was the quicker one for 128 single tokens with 512 / 4000 positions of their own from 1500 / 4500 shared ones on, for 16 groups of
 * four single tokens from 1000 and of 16 tokens from 6000, for one group of four from 4000.
 *   cu_seq [n_groups+1] int32, non-decreasing within [0, B];  len [n_groups] int32 (both DEVICE, 4-byte aligned)
 *   max_tok: at least the largest number of new tokens of one group, at most T.  1 <= n_groups <= QSPEC_KV_MAX_GROUPS
 * Arguments, masks, outputs and limits otherwise as for qspec_kv_attention, whose workspace serves both calls.  Sequences of
 * no group are not computed, their outputs not written.  A group with a sequence whose numbers are out of range (or more than max_tok
 * new tokens, or a len outside [0, max_pages * page]) is left out, all groups if cu_seq is out of order, and the next
 * qspec_check_status returns QSPEC_ERR_INVALID_ARG.
 */
#define QSPEC_KV_MAX_GROUPS 512
typedef struct {
  const int32_t* cu_seq;
  const int32_t* len;
  int32_t n_groups, max_tok;
} qspec_kv_prefixes;
qspec_status qspec_kv_attention_shared(const qspec_kv_cache* cache, const qspec_kv_batch* batch, const qspec_kv_prefixes* prefixes,
                                       const uint16_t* q, int64_t q_token, int32_t heads_q, float scale, int32_t window,
                                       const uint64_t* tree, uint16_t* out, int64_t out_token, float* lse, void* ws,
                                       size_t ws_bytes, qspec_stream_t stream);

/*
 * qspec_logits_adjust -- penalties for repeated tokens, biases and a grammar mask on the logits of a verify
 * call (or of plain decoding: rows = 1).  Row i of sequence b scores the token after its history and its
 * first i draft tokens, so those count as history there:
 *     c[v]    occurrences of v in hist[b, prompt_len .. hist_len - 1] and draft_tok[b, 0 .. i-1]
 *     seen[v] v occurs there or in the prompt, hist[b, 0 .. prompt_len - 1]
 *     z = logit;  if seen: z = z > 0 ? z / repetition : z * repetition
 *     z = z - frequency * c - (c > 0 ? presence : 0) + bias[v];   masked out: z = -inf
 * (The bias comes last.  Where it is added before the penalties, as many servers do, a token that is both seen and biased
 * comes out differently, as the repetition penalty goes by the logit's sign.)
 * computed in fp32 (the quotient as the product with 1 / repetition) and rounded to bf16 once; a logit that nothing
 * touches keeps its bits.
 *
 *   logits     [B, rows, V] bf16;  out [B, rows, V] bf16, may be logits itself
 *   draft_tok  [B, rows-1] int32, or NULL: none
 *   hist       [B, hist_stride] int32, hist_len [B] int32, or both NULL: no history
 *   prompt_len [B] int32, or NULL: 0
 *   penalties  [B, 3] fp32 (repetition > 0, frequency, presence), or NULL: 1, 0, 0
 *   bias_ids   [B, n_bias] int32 (negative: unused entry; the last entry of an id that is repeated counts) and
 *              bias [B, n_bias] fp32, or both NULL
 *   mask       [B, rows, ceil(V/32)] uint32: bit v mod 32 of word v / 32 allows token v, or NULL
 *   1 <= rows <= QSPEC_MAX_GAMMA + 1, 2 <= V <= 2^24, B*rows*V < 2^40, B <= 65535, n_bias <= 65535; logits and out 16-byte
 *   aligned, the other arrays 4-byte aligned.
 * Ids outside [0, V), lengths outside [0, hist_stride] (limited to it), prompt_len > hist_len and a repetition
 * penalty that is not > 0 (taken as 1) make the next qspec_check_status return QSPEC_ERR_INVALID_ARG; such
 * ids count for nothing.
 */
qspec_status qspec_logits_adjust(const uint16_t* logits, int32_t B, int32_t rows, int32_t V,
                                 const int32_t* draft_tok, const int32_t* hist, int64_t hist_stride,
                                 const int32_t* hist_len, const int32_t* prompt_len, const float* penalties,
                                 const int32_t* bias_ids, const float* bias, int32_t n_bias, const uint32_t* mask,
                                 uint16_t* out, qspec_stream_t stream);

/*
 * qspec_check_status -- synchronises `stream`, then reports (and clears) the error words that the
 * kernels set on the device: the verify workspace's word when `ws` is not NULL, and the library's
 * own words for the linear and decode-loop kernels of the current device.  QSPEC_ERR_TIMEOUT if a
 * kernel gave up a bounded wait, QSPEC_ERR_WORKSPACE if a linear call found its workspace laid out
 * for another shape, QSPEC_ERR_INVALID_ARG if a draft token id or a gather id was out of range
 * (or a kernel of the cache and logits calls met a bad value), QSPEC_ERR_CUDA if the stream reported an
 * error, QSPEC_OK otherwise.
 */
qspec_status qspec_check_status(void* ws, qspec_stream_t stream);

/* qspec_status_string -- a static, human-readable name for a status code. */
const char* qspec_status_string(qspec_status status);

#ifdef __cplusplus
}
#endif

#endif /* QSPEC_H_ */
