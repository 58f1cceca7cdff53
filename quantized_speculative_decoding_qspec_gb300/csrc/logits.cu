// Penalties for repeated tokens, biases and a grammar mask on the logits that a verify call reads.
//
// z = logit; seen: z > 0 ? z / rep : z * rep; then - freq * count - presence * (count > 0) + bias; masked out:
// -inf.  Row i of a sequence counts its history and its first i draft tokens.  Each logit is read and
// written once (2 + 2 bytes, and a mask bit), which bounds it.  A block owns a range of the vocabulary of one
// sequence for all its rows: it counts the history's tokens of that range in shared memory (integer
// atomics, so the order does not matter; history and bias list come from L2 once per range), and every
// thread then walks the rows of its 8 tokens, adding the draft tokens in registers as it goes.  Logits that
// nothing touches keep their bits.
#include "kv_internal.h"

namespace qspec {
namespace {

constexpr int kThreads = 256;
constexpr uint32_t kSeen = 0x80000000u;

struct LogitsArgs {
  const uint16_t* logits;
  uint16_t* out;
  const int32_t* draft;
  const int32_t* hist;
  const int32_t* hist_len;
  const int32_t* prompt_len;
  const float* pen;
  const int32_t* bias_ids;
  const float* bias;
  const uint32_t* mask;
  unsigned int* err;
  int64_t hist_stride;
  int rows, V, n_bias, range;  // range: tokens per block
};

struct Penalty {
  float rep, freq, pres;
};

__device__ __forceinline__ float adjust(float z, uint32_t count, float bias, const Penalty& p) {
  if (count & kSeen) z = z > 0.0f ? z / p.rep : z * p.rep;
  const uint32_t c = count & ~kSeen;
  if (c) z -= p.freq * static_cast<float>(c) + p.pres;
  return z + bias;
}

// kVec tokens per thread and step: 8 (V a multiple of 8, 16-byte accesses) or 1.
template <int kVec>
__global__ void __launch_bounds__(kThreads) logits_kernel(const LogitsArgs a) {
  extern __shared__ uint32_t count[];  // [range] kSeen | occurrences, then [range] 1 + bias entry
  uint32_t* entry = count + a.range;
  __shared__ int32_t sdraft[QSPEC_MAX_GAMMA];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int b = blockIdx.y;
  const int v0 = blockIdx.x * a.range;
  const int nv = min(a.V - v0, a.range);
  bool bad = false;

  for (int i = threadIdx.x; i < nv; i += kThreads) {
    count[i] = 0;
    if (a.n_bias) entry[i] = 0;
  }
  const int n_draft = a.draft ? a.rows - 1 : 0;
  if (threadIdx.x < n_draft) {
    const int32_t t = a.draft[static_cast<int64_t>(b) * n_draft + threadIdx.x];
    bad |= t < 0 || t >= a.V;
    sdraft[threadIdx.x] = t;
  }
  Penalty p{1.0f, 0.0f, 0.0f};
  if (a.pen) {
    p = Penalty{a.pen[3 * b], a.pen[3 * b + 1], a.pen[3 * b + 2]};
    if (!(p.rep > 0.0f)) {
      bad = true;
      p.rep = 1.0f;
    }
  }
  __syncthreads();
  if (a.hist && a.pen) {
    int len = a.hist_len[b], prompt = a.prompt_len ? a.prompt_len[b] : 0;
    bad |= len < 0 || len > a.hist_stride || prompt < 0 || prompt > len;
    len = static_cast<int>(min(static_cast<int64_t>(max(len, 0)), a.hist_stride));
    const int32_t* h = a.hist + static_cast<int64_t>(b) * a.hist_stride;
    auto add = [&](int i, int32_t t) {
      bad |= t < 0 || t >= a.V;
      const uint32_t at = static_cast<uint32_t>(t) - static_cast<uint32_t>(v0);
      if (at < static_cast<uint32_t>(nv)) {
        atomicOr(count + at, kSeen);
        if (i >= prompt) atomicAdd(count + at, 1u);
      }
    };
    int i = threadIdx.x;
    for (; i + 3 * kThreads < len; i += 4 * kThreads) {
      const int32_t t0 = h[i], t1 = h[i + kThreads], t2 = h[i + 2 * kThreads], t3 = h[i + 3 * kThreads];
      add(i, t0);
      add(i + kThreads, t1);
      add(i + 2 * kThreads, t2);
      add(i + 3 * kThreads, t3);
    }
    for (; i < len; i += kThreads) add(i, h[i]);
  }
  const float* bias = a.bias + static_cast<int64_t>(b) * a.n_bias;
  for (int i = threadIdx.x; i < a.n_bias; i += kThreads) {
    const int32_t t = a.bias_ids[static_cast<int64_t>(b) * a.n_bias + i];
    bad |= t >= a.V;
    const uint32_t at = static_cast<uint32_t>(t) - static_cast<uint32_t>(v0);
    if (t >= 0 && at < static_cast<uint32_t>(nv)) atomicMax(entry + at, static_cast<uint32_t>(i) + 1u);
  }
  if (bad && blockIdx.x == 0) atomicOr(a.err, kErrInvalid);  // (every block of the sequence sees the same lists)
  __syncthreads();

  const int words = (a.V + 31) / 32;
  const bool pen = a.pen != nullptr;
  for (int i = threadIdx.x * kVec; i < nv; i += kThreads * kVec) {
    uint32_t c[kVec];
    float bs[kVec];
    bool touched = false;
#pragma unroll
    for (int e = 0; e < kVec; ++e) {
      c[e] = count[i + e];
      const uint32_t at = a.n_bias ? entry[i + e] : 0u;
      bs[e] = at ? bias[at - 1] : 0.0f;
      touched |= c[e] != 0 || at != 0;
    }
    const int64_t row0 = static_cast<int64_t>(b) * a.rows;
    for (int r = 0; r < a.rows; ++r) {
      if (pen && r > 0 && r <= n_draft) {
        const uint32_t at = static_cast<uint32_t>(sdraft[r - 1]) - static_cast<uint32_t>(v0 + i);
        if (at < kVec) {
          touched = true;
#pragma unroll
          for (int e = 0; e < kVec; ++e)
            if (at == e) c[e] = (c[e] | kSeen) + 1u;
        }
      }
      const int64_t off = (row0 + r) * a.V + v0 + i;
      uint32_t allowed = 0xFFu;
      if (a.mask) {
        const uint8_t* m = reinterpret_cast<const uint8_t*>(a.mask + (row0 + r) * words);
        allowed = kVec == 8 ? m[(v0 + i) >> 3] : (m[(v0 + i) >> 3] >> ((v0 + i) & 7)) & 1u;
      }
      if (kVec == 8) {
        uint4 w = *reinterpret_cast<const uint4*>(a.logits + off);
        uint32_t* u = reinterpret_cast<uint32_t*>(&w);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (touched) {
            const int l = 2 * e, h = l + 1;
            if (c[l] || bs[l] != 0.0f)
              u[e] = (u[e] & 0xFFFF0000u) | f32_to_bf16_bits(adjust(bf16_lo(u[e]), c[l], bs[l], p));
            if (c[h] || bs[h] != 0.0f)
              u[e] = (u[e] & 0xFFFFu) | static_cast<uint32_t>(f32_to_bf16_bits(adjust(bf16_hi(u[e]), c[h], bs[h], p))) << 16;
          }
          if (!(allowed >> (2 * e) & 1u)) u[e] = (u[e] & 0xFFFF0000u) | 0xFF80u;
          if (!(allowed >> (2 * e + 1) & 1u)) u[e] = (u[e] & 0xFFFFu) | 0xFF800000u;
        }
        *reinterpret_cast<uint4*>(a.out + off) = w;
      } else {
        uint16_t w = a.logits[off];
        if (c[0] || bs[0] != 0.0f) w = f32_to_bf16_bits(adjust(bf16_lo(w), c[0], bs[0], p));
        if (!(allowed & 1u)) w = 0xFF80u;
        a.out[off] = w;
      }
    }
  }
}

}  // namespace
}  // namespace qspec

using namespace qspec;

extern "C" qspec_status qspec_logits_adjust(const uint16_t* logits, int32_t B, int32_t rows, int32_t V,
                                            const int32_t* draft_tok, const int32_t* hist, int64_t hist_stride,
                                            const int32_t* hist_len, const int32_t* prompt_len, const float* penalties,
                                            const int32_t* bias_ids, const float* bias, int32_t n_bias,
                                            const uint32_t* mask, uint16_t* out, qspec_stream_t stream) {
  if (!logits || !out || B <= 0 || rows <= 0 || V <= 0) return QSPEC_ERR_INVALID_ARG;
  if (!hist != !hist_len || (hist && hist_stride <= 0) || (prompt_len && !hist)) return QSPEC_ERR_INVALID_ARG;
  if (!bias_ids != !bias || (bias && n_bias <= 0)) return QSPEC_ERR_INVALID_ARG;
  if (rows > QSPEC_MAX_GAMMA + 1 || V < 2 || V > QSPEC_MAX_V || B > 65535 ||
      int64_t(B) * rows * int64_t(V) >= (int64_t(1) << 40) || hist_stride > 0x7FFFFFFF)
    return QSPEC_ERR_UNSUPPORTED_SHAPE;
  if (!aligned16(logits) || !aligned16(out) || !aligned4(draft_tok) || !aligned4(hist) || !aligned4(hist_len) ||
      !aligned4(prompt_len) || !aligned4(penalties) || !aligned4(bias_ids) || !aligned4(bias) || !aligned4(mask))
    return QSPEC_ERR_MISALIGNED;
  LogitsArgs a{logits, out, draft_tok, hist, hist_len, prompt_len, penalties, bias_ids, bias, mask,
               linear_error_word(), hist_stride, rows, V, bias ? n_bias : 0};
  if (!a.err) return QSPEC_ERR_CUDA;
  a.range = 2048;
  const dim3 grid((V + a.range - 1) / a.range, B);
  const size_t smem = sizeof(uint32_t) * a.range * (a.n_bias ? 2 : 1);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (V % 8 == 0) return launch_pdl(logits_kernel<8>, grid, dim3(kThreads), smem, s, a);
  return launch_pdl(logits_kernel<1>, grid, dim3(kThreads), smem, s, a);
}
