// Attention of a step's tokens over the paged cache of e4m3 codes: the entry point and its choice of kernel.
#include "kv_decode.cuh"
#include "kv_prefill.cuh"

namespace qspec {
namespace att {
namespace {

// The workspace: tickets, then two partial items per CTA, then the items that runs have cut.  Its layout does not depend on the call's shape.
constexpr size_t kTicketBytes = 24576;  // three a CTA
constexpr int kMaxGrid = 2048;
constexpr size_t kCutBytes = sizeof(CutItem) * kMaxGrid;
constexpr size_t slot_bytes(int rows) { return sizeof(float) * 2 * rows * (128 + 2); }  // of a CTA, heads of 128

int max_grid(int ctas_per_sm) {
  const int n = ctas_per_sm * num_sms();
  return n < kMaxGrid ? n : kMaxGrid;
}

// kShared: `a` has groups of sequences, otherwise their items are the sequences'.
template <int D, int RG, bool kShared>
qspec_status launch_decode(AttArgs& a, int64_t rows, cudaStream_t s) {
  using C = DecodeCfg<D, RG, kShared>;
  a.max_tiles = static_cast<int>((rows + C::kRows - 1) / C::kRows);
  const int owners = kShared ? a.groups : a.b.B, most = kShared ? QSPEC_KV_MAX_GROUPS : QSPEC_KV_MAX_B;
  if (cudaFuncSetAttribute(decode_kernel<D, RG, kShared>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::smem(most)) != cudaSuccess)
    return QSPEC_ERR_CUDA;
  return launch_pdl(decode_kernel<D, RG, kShared>, dim3(max_grid(C::ctas(owners))), dim3(C::kThreads), C::smem(owners), s, a);
}

template <int D, bool kBigPages, bool kShared>
qspec_status launch_prefill(AttArgs& a, int64_t rows, cudaStream_t s) {
  using C = PrefillCfg<D>;
  a.max_tiles = static_cast<int>((rows + C::kRows - 1) / C::kRows);
  const int owners = kShared ? a.groups : a.b.B, most = kShared ? QSPEC_KV_MAX_GROUPS : QSPEC_KV_MAX_B;
  const int fixed = kShared ? C::kSmemShared : C::kSmem, each = sizeof(int2);
  if (cudaFuncSetAttribute(prefill_kernel<D, kBigPages, kShared>, cudaFuncAttributeMaxDynamicSharedMemorySize, fixed + each * (most + 1)) !=
      cudaSuccess)
    return QSPEC_ERR_CUDA;
  const qspec_status st =
      launch_pdl(prefill_kernel<D, kBigPages, kShared>, dim3(max_grid(1)), dim3(C::kThreads), fixed + each * (owners + 1), s, a);
  if (!kShared || st != QSPEC_OK) return st;
  return launch_pdl(merge_kernel<D>, dim3(max_grid(1), kMergeSplit), dim3(C::kRows), 0, s, a);
}

template <bool kShared>
qspec_status launch(AttArgs& a, int64_t rows, cudaStream_t s) {
  const bool d128 = a.c.dim == 128;
  // Up to 64 rows a key head the decode kernel reads a sequence's keys twice at most and wins everywhere (16
  // sequences of 4096, 64 rows: 71 against 77 us; one of 32768: 51 against 94); with 96 rows and more it reads them three
  // times and computes on the legacy tensor path (128 rows: 119 against 78 us).
  // With shared prefixes the prefill kernel takes key tiles in turn with its two query tiles, and wins from 33 rows on (16 groups
  // over 6001 + 300 positions, 32 rows: 103 us in either; 64 rows: 182 here, 141 there; one group over 32768, 32 rows: 45 here, 49 there).
  if (rows > (kShared ? 32 : 64)) {
    if (a.c.page >= 64) return d128 ? launch_prefill<128, true, kShared>(a, rows, s) : launch_prefill<64, true, kShared>(a, rows, s);
    return d128 ? launch_prefill<128, false, kShared>(a, rows, s) : launch_prefill<64, false, kShared>(a, rows, s);
  }
  if (d128) return rows <= 16 ? launch_decode<128, 1, kShared>(a, rows, s) : launch_decode<128, 2, kShared>(a, rows, s);
  return rows <= 16 ? launch_decode<64, 1, kShared>(a, rows, s) : launch_decode<64, 2, kShared>(a, rows, s);
}

}  // namespace
}  // namespace att
}  // namespace qspec

using namespace qspec;
using namespace qspec::att;

extern "C" size_t qspec_kv_attention_workspace_size(void) {
  const size_t few = max_grid(4) * slot_bytes(DecodeCfg<128, 1>::kRows), many = max_grid(1) * slot_bytes(PrefillCfg<128>::kRows);
  return kTicketBytes + (few > many ? few : many) + kCutBytes;
}

namespace {

// Checks that both calls share; fills `a`.  rows: query rows a key head of `owners` sequences or groups of most_tok tokens at most.
qspec_status prepare(const qspec_kv_cache* cache, const qspec_kv_batch* batch, const uint16_t* q, int64_t q_token, int32_t heads_q,
                     float scale, int32_t window, const uint64_t* tree, uint16_t* out, int64_t out_token, float* lse, void* ws,
                     size_t ws_bytes, int64_t owners, int64_t most_tok, AttArgs& a, int64_t& rows) {
  const float scale_log2 = scale * 1.44269504088896f;
  if (!q || !out || heads_q <= 0 || !isfinite(scale_log2) || window < 0) return QSPEC_ERR_INVALID_ARG;
  qspec_status st = check_kv(cache, batch);
  if (st != QSPEC_OK) return st;
  if (heads_q % cache->heads != 0 || heads_q / cache->heads > 128) return QSPEC_ERR_UNSUPPORTED_SHAPE;
  if (tree && (batch->max_tok > 64 || window != 0)) return QSPEC_ERR_UNSUPPORTED_SHAPE;
  const int64_t row = static_cast<int64_t>(heads_q) * cache->dim;
  if ((st = check_rows(q, batch->T, row, q_token)) != QSPEC_OK) return st;
  if ((st = check_rows(out, batch->T, row, out_token)) != QSPEC_OK) return st;
  if ((tree && (reinterpret_cast<uintptr_t>(tree) & 7u)) || !aligned4(lse) || !aligned16(ws)) return QSPEC_ERR_MISALIGNED;
  if (!ws || ws_bytes < qspec_kv_attention_workspace_size()) return QSPEC_ERR_WORKSPACE;
  rows = most_tok * (heads_q / cache->heads);
  if (rows > 0x7FFFFF00 || owners * ((rows + 15) / 16) >= (int64_t(1) << 30)) return QSPEC_ERR_UNSUPPORTED_SHAPE;
  a = AttArgs{*cache, *batch, q, out, lse, reinterpret_cast<const unsigned long long*>(tree), linear_error_word()};
  if (!a.err) return QSPEC_ERR_CUDA;
  a.tickets = static_cast<unsigned int*>(ws);
  a.partial = reinterpret_cast<float*>(static_cast<char*>(ws) + kTicketBytes);
  a.cuts = reinterpret_cast<CutItem*>(static_cast<char*>(ws) + qspec_kv_attention_workspace_size() - kCutBytes);
  a.q_token = q_token;
  a.out_token = out_token;
  a.heads_q = heads_q;
  a.group = heads_q / cache->heads;
  a.window = window;
  int shift = 0;
  while ((1 << shift) < a.group) ++shift;
  a.group_shift = 31 + shift;
  a.group_mul = static_cast<uint32_t>(((uint64_t(1) << a.group_shift) + a.group - 1) / a.group);
  a.scale_log2 = scale_log2;
  return QSPEC_OK;
}

}  // namespace

extern "C" qspec_status qspec_kv_attention(const qspec_kv_cache* cache, const qspec_kv_batch* batch, const uint16_t* q,
                                           int64_t q_token, int32_t heads_q, float scale, int32_t window,
                                           const uint64_t* tree, uint16_t* out, int64_t out_token, float* lse, void* ws,
                                           size_t ws_bytes, qspec_stream_t stream) {
  AttArgs a;
  int64_t rows;
  const qspec_status st = prepare(cache, batch, q, q_token, heads_q, scale, window, tree, out, out_token, lse, ws, ws_bytes,
                                  batch ? batch->B : 0, batch ? batch->max_tok : 0, a, rows);
  if (st != QSPEC_OK) return st;
  return launch<false>(a, rows, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" qspec_status qspec_kv_attention_shared(const qspec_kv_cache* cache, const qspec_kv_batch* batch,
                                                  const qspec_kv_prefixes* prefixes, const uint16_t* q, int64_t q_token,
                                                  int32_t heads_q, float scale, int32_t window, const uint64_t* tree, uint16_t* out,
                                                  int64_t out_token, float* lse, void* ws, size_t ws_bytes, qspec_stream_t stream) {
  if (!prefixes || !prefixes->cu_seq || !prefixes->len || prefixes->n_groups <= 0 || prefixes->max_tok <= 0) return QSPEC_ERR_INVALID_ARG;
  AttArgs a;
  int64_t rows;
  const qspec_status st = prepare(cache, batch, q, q_token, heads_q, scale, window, tree, out, out_token, lse, ws, ws_bytes,
                                  prefixes->n_groups, prefixes->max_tok, a, rows);
  if (st != QSPEC_OK) return st;
  if (prefixes->n_groups > QSPEC_KV_MAX_GROUPS || prefixes->max_tok > batch->T) return QSPEC_ERR_UNSUPPORTED_SHAPE;
  if (!aligned4(prefixes->cu_seq) || !aligned4(prefixes->len)) return QSPEC_ERR_MISALIGNED;
  a.cu_seq = prefixes->cu_seq;
  a.prefix = prefixes->len;
  a.groups = prefixes->n_groups;
  a.group_tok = prefixes->max_tok;
  return launch<true>(a, rows, reinterpret_cast<cudaStream_t>(stream));
}
