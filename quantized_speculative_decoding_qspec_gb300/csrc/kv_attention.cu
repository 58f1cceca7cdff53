// Attention of a step's tokens over the paged cache of e4m3 codes: the entry point and its choice of kernel.
#include "kv_decode.cuh"
#include "kv_prefill.cuh"

namespace qspec {
namespace att {
namespace {

// The workspace: tickets, then two partial items per CTA.  Its layout does not depend on the call's shape.
constexpr size_t kTicketBytes = 24576;  // three a CTA
constexpr int kMaxGrid = 2048;
constexpr size_t slot_bytes(int rows) { return sizeof(float) * 2 * rows * (128 + 2); }  // of a CTA, heads of 128

int max_grid(int ctas_per_sm) {
  const int n = ctas_per_sm * num_sms();
  return n < kMaxGrid ? n : kMaxGrid;
}

template <int D, int RG>
qspec_status launch_decode(AttArgs& a, int64_t rows, cudaStream_t s) {
  using C = DecodeCfg<D, RG>;
  a.max_tiles = static_cast<int>((rows + C::kRows - 1) / C::kRows);
  if (cudaFuncSetAttribute(decode_kernel<D, RG>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::smem(QSPEC_KV_MAX_B)) != cudaSuccess)
    return QSPEC_ERR_CUDA;
  return launch_pdl(decode_kernel<D, RG>, dim3(max_grid(C::ctas(a.b.B))), dim3(C::kThreads), C::smem(a.b.B), s, a);
}

template <int D, bool kBigPages>
qspec_status launch_prefill(AttArgs& a, int64_t rows, cudaStream_t s) {
  using C = PrefillCfg<D>;
  a.max_tiles = static_cast<int>((rows + C::kRows - 1) / C::kRows);
  const size_t smem = C::kSmem + sizeof(int2) * (a.b.B + 1);
  if (cudaFuncSetAttribute(prefill_kernel<D, kBigPages>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           C::kSmem + static_cast<int>(sizeof(int2)) * (QSPEC_KV_MAX_B + 1)) != cudaSuccess)
    return QSPEC_ERR_CUDA;
  return launch_pdl(prefill_kernel<D, kBigPages>, dim3(max_grid(1)), dim3(C::kThreads), smem, s, a);
}

}  // namespace
}  // namespace att
}  // namespace qspec

using namespace qspec;
using namespace qspec::att;

extern "C" size_t qspec_kv_attention_workspace_size(void) {
  const size_t few = max_grid(4) * slot_bytes(DecodeCfg<128, 1>::kRows), many = max_grid(1) * slot_bytes(PrefillCfg<128>::kRows);
  return kTicketBytes + (few > many ? few : many);
}

extern "C" qspec_status qspec_kv_attention(const qspec_kv_cache* cache, const qspec_kv_batch* batch, const uint16_t* q,
                                           int64_t q_token, int32_t heads_q, float scale, int32_t window,
                                           const uint64_t* tree, uint16_t* out, int64_t out_token, float* lse, void* ws,
                                           size_t ws_bytes, qspec_stream_t stream) {
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
  const int64_t rows = static_cast<int64_t>(batch->max_tok) * (heads_q / cache->heads);
  if (rows > 0x7FFFFF00 || batch->B * ((rows + 15) / 16) >= (int64_t(1) << 30)) return QSPEC_ERR_UNSUPPORTED_SHAPE;
  AttArgs a{*cache, *batch, q, out, lse, reinterpret_cast<const unsigned long long*>(tree), linear_error_word()};
  if (!a.err) return QSPEC_ERR_CUDA;
  a.tickets = static_cast<unsigned int*>(ws);
  a.partial = reinterpret_cast<float*>(static_cast<char*>(ws) + kTicketBytes);
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
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  // Up to 64 rows a key head the decode kernel reads a sequence's keys twice at most and wins everywhere (16
  // sequences of 4096, 64 rows: 71 against 77 us; one of 32768: 51 against 94); with 96 rows and more it reads them three
  // times and computes on the legacy tensor path (128 rows: 119 against 78 us).
  if (rows > 64) {
    if (cache->page >= 64) return cache->dim == 128 ? launch_prefill<128, true>(a, rows, s) : launch_prefill<64, true>(a, rows, s);
    return cache->dim == 128 ? launch_prefill<128, false>(a, rows, s) : launch_prefill<64, false>(a, rows, s);
  }
  if (cache->dim == 128) return rows <= 16 ? launch_decode<128, 1>(a, rows, s) : launch_decode<128, 2>(a, rows, s);
  return rows <= 16 ? launch_decode<64, 1>(a, rows, s) : launch_decode<64, 2>(a, rows, s);
}
