// Attention of a step's tokens over the paged cache of e4m3 codes.
//
// out = sum_j softmax(scale q . k_j) v_j over the visible cache positions j, in one pass: a running
// maximum m, the sum l of exp(s_j - m) and the weighted sum of the values are rescaled when m grows.
// This is the plain kernel: a warp owns one (token, query head); in a step of 32 positions each lane
// scores one key, and each lane then adds its D / 32 channels of the 32 values.
#include "kv_internal.h"

namespace qspec {
namespace {

constexpr int kWarps = 4;

struct AttArgs {
  qspec_kv_cache c;
  qspec_kv_batch b;
  const uint16_t* q;
  uint16_t* out;
  float* lse;
  const unsigned long long* tree;
  unsigned int* err;
  int64_t q_token, out_token;
  int heads_q, group, window;
  float scale;
};

template <int D>
__global__ void __launch_bounds__(kWarps * 32) attention_kernel(const AttArgs a) {
  __shared__ float qs[kWarps][D];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int b = blockIdx.z, i = blockIdx.x, h = blockIdx.y * kWarps + warp;
  const int P = a.c.page;
  const SeqSpan sp = seq_span(a.b, P, b);
  if (!sp.ok && threadIdx.x == 0) atomicOr(a.err, kErrInvalid);
  if (i >= sp.n || h >= a.heads_q) return;
  const int64_t t = sp.tok0 + i;
  const uint16_t* q = a.q + t * a.q_token + static_cast<int64_t>(h) * D;
  bool odd = false;  // a NaN or an infinity in the query
  for (int d = lane; d < D; d += 32) {
    odd |= (q[d] & 0x7F80u) == 0x7F80u;
    qs[warp][d] = odd ? 0.0f : bf16_lo(q[d]) * a.scale;
  }
  odd = __any_sync(0xFFFFFFFFu, odd);
  const int base = sp.kv - sp.n;
  const int hi = a.tree ? sp.kv : min(base + i + 1, sp.kv);
  const int lo = a.window > 0 ? max(base + i + 1 - a.window, 0) : 0;
  const unsigned long long bits = a.tree ? a.tree[t] : 0ull;
  const int hk = h / a.group;
  const int32_t* pages = a.b.pages + static_cast<int64_t>(b) * a.b.max_pages;

  constexpr int kPer = D / 32;
  float m = -INFINITY, l = 0.0f, acc[kPer] = {};
  for (int j0 = lo; j0 < hi; j0 += 32) {
    const int j = j0 + lane;
    bool see = j < hi;
    if (a.tree && see && j >= base) see = (bits >> (j - base)) & 1ull;
    int page = 0;
    if (see) {
      page = pages[j / P];
      if (page < 0 || page >= a.c.n_pages) {
        atomicOr(a.err, kErrInvalid);
        see = false;
        page = 0;
      }
    }
    const int64_t ph = static_cast<int64_t>(page) * a.c.heads + hk;
    const int64_t at = (ph * P + (see ? j % P : 0)) * D;
    float s = -INFINITY;
    if (see) {
      s = 0.0f;
      const uint4* kp = reinterpret_cast<const uint4*>(a.c.k + at);
      for (int d = 0; d < D / 16; ++d) {
        const uint4 w = kp[d];
        const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 x = e4m3x2_to_f32(ww[e] & 0xFFFFu), y = e4m3x2_to_f32(ww[e] >> 16);
          const float* qd = qs[warp] + 16 * d + 4 * e;
          s += qd[0] * x.x + qd[1] * x.y + qd[2] * y.x + qd[3] * y.y;
        }
      }
      s *= exp2_int(a.c.k_exp[ph]);
    }
    float mx = s;
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, off));
    const float m1 = fmaxf(m, mx);
    if (m1 == -INFINITY) continue;
    const float keep = expf(m - m1), p = see ? expf(s - m1) : 0.0f;
    m = m1;
    l = l * keep + p;
#pragma unroll
    for (int e = 0; e < kPer; ++e) acc[e] *= keep;
    const float pv = see ? p * exp2_int(a.c.v_exp[ph]) : 0.0f;
    for (int n = 0; n < 32; ++n) {
      const float w = __shfl_sync(0xFFFFFFFFu, pv, n);
      const long long vat = __shfl_sync(0xFFFFFFFFu, static_cast<long long>(at), n);
      if (!__shfl_sync(0xFFFFFFFFu, see ? 1 : 0, n)) continue;
#pragma unroll
      for (int e = 0; e < kPer; e += 2) {
        const float2 x = e4m3x2_to_f32(*reinterpret_cast<const uint16_t*>(a.c.v + vat + lane * kPer + e));
        acc[e] += w * x.x;
        acc[e + 1] += w * x.y;
      }
    }
  }
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, off);
  const float inv = l > 0.0f ? (odd ? NAN : 1.0f / l) : 0.0f;
  uint16_t* o = a.out + t * a.out_token + static_cast<int64_t>(h) * D + lane * kPer;
#pragma unroll
  for (int e = 0; e < kPer; e += 2) *reinterpret_cast<uint32_t*>(o + e) = pack_bf16(acc[e] * inv, acc[e + 1] * inv);
  if (a.lse && lane == 0) a.lse[t * a.heads_q + h] = l > 0.0f ? (odd ? NAN : m + logf(l)) : -INFINITY;
}

}  // namespace
}  // namespace qspec

using namespace qspec;

extern "C" size_t qspec_kv_attention_workspace_size(void) { return 256; }

extern "C" qspec_status qspec_kv_attention(const qspec_kv_cache* cache, const qspec_kv_batch* batch, const uint16_t* q,
                                           int64_t q_token, int32_t heads_q, float scale, int32_t window,
                                           const uint64_t* tree, uint16_t* out, int64_t out_token, float* lse, void* ws,
                                           size_t ws_bytes, qspec_stream_t stream) {
  if (!q || !out || heads_q <= 0 || !isfinite(scale) || window < 0) return QSPEC_ERR_INVALID_ARG;
  qspec_status st = check_kv(cache, batch);
  if (st != QSPEC_OK) return st;
  if (heads_q % cache->heads != 0 || heads_q / cache->heads > 128) return QSPEC_ERR_UNSUPPORTED_SHAPE;
  if (tree && (batch->max_tok > 64 || window != 0)) return QSPEC_ERR_UNSUPPORTED_SHAPE;
  const int64_t row = static_cast<int64_t>(heads_q) * cache->dim;
  if ((st = check_rows(q, batch->T, row, q_token)) != QSPEC_OK) return st;
  if ((st = check_rows(out, batch->T, row, out_token)) != QSPEC_OK) return st;
  if ((tree && (reinterpret_cast<uintptr_t>(tree) & 7u)) || !aligned4(lse) || !aligned16(ws)) return QSPEC_ERR_MISALIGNED;
  if (!ws || ws_bytes < qspec_kv_attention_workspace_size()) return QSPEC_ERR_WORKSPACE;
  AttArgs a{*cache, *batch, q, out, lse, reinterpret_cast<const unsigned long long*>(tree), linear_error_word(),
            q_token, out_token, heads_q, heads_q / cache->heads, window, scale};
  if (!a.err) return QSPEC_ERR_CUDA;
  const dim3 grid(batch->max_tok, (heads_q + kWarps - 1) / kWarps, batch->B);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (cache->dim == 128) return launch_pdl(attention_kernel<128>, grid, dim3(kWarps * 32), 0, s, a);
  return launch_pdl(attention_kernel<64>, grid, dim3(kWarps * 32), 0, s, a);
}
