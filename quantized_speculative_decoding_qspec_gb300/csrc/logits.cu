// Penalties for repeated tokens, biases and a grammar mask on the logits that a verify call reads.
//
// z = logit; seen: z > 0 ? z / rep : z * rep; then - freq * count - presence * (count > 0) + bias; masked out:
// -inf.  Row i of a sequence counts its history and its first i draft tokens.  Each logit is read and
// written once (2 + 2 bytes, and a mask bit), which bounds it.  A block owns a range of the vocabulary of one
// sequence for all its rows: it counts the history's tokens of that range in shared memory (integer
// atomics, so the order does not matter; history and bias list come from L2 once per range), and every
// thread then walks the rows of its 8 tokens, adding the draft tokens in registers as it goes.  Few tokens
// are touched but most warps have some, so the arithmetic runs only for those of the 8 places that some
// lane of the warp needs, with what history and bias do to a token worked out once for all rows.  Logits
// that nothing touches keep their bits.  A block asks for its rows' bytes in L2 before it counts (without lists 60 -> 55
// us).  [64, 8, 152064]: 55 us without penalties (5.7 TB/s), 80 with histories of 8192, 300 biases and masks, where the
// schedulers issue in 61% of the cycles and warps wait on L2 or on the arithmetic's results for the rest; listing the
// touched tokens and doing them after the copy, a lane each, took 105, the adjustment in paired FMAs 84.
#include "kv_internal.h"

namespace qspec {
namespace {

constexpr int kThreads = 256;
constexpr uint32_t kSeen = 0x80000000u;
constexpr uint32_t kEntry = 0xFFFF0000u;  // + entry of the bias list: a NaN that no bias is stored as

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

// What a token's history and bias do to its logit: z > 0 ? z / rep : z * rep where it was seen, then - sub.  The quotient
// is the product with the reciprocal, one fp32 rounding more before the one to bf16 ([64, 8, 152064] with divisions: 96
// us against 80).  Where the reciprocal is no normal number (`divide`) the sequence's blocks walk token by token and
// divide: a choice for each logit cost 9 us of the 80, too.
struct Penalty {
  float rep, inv, freq, pres;
  bool divide;
  __device__ float sub(uint32_t count, float bias) const {
    const uint32_t c = count & ~kSeen;
    return (c ? fmaf(freq, static_cast<float>(c), pres) : 0.0f) - bias;
  }
  __device__ float adjust(float z, bool seen, float sub) const {
    if (seen) z *= z > 0.0f ? inv : rep;
    return z - sub;
  }
  __device__ float adjust_dividing(float z, bool seen, float sub) const {
    if (seen) z = z > 0.0f ? z / rep : z * rep;
    return z - sub;
  }
};

// A count and one draft token more.  (A count of 2^31 - 1 stays: it has no bit left, and fp32 rounds it to 2^31.)
__device__ __forceinline__ uint32_t one_more(uint32_t count) { return (count | kSeen) == 0xFFFFFFFFu ? count | kSeen : (count | kSeen) + 1u; }

// 16 bytes read once (not through the read-only path: `out` may be the same memory).
__device__ __forceinline__ uint4 load_once(const void* p) {
  uint4 r;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p) : "memory");
  return r;
}

// Bits 0 .. 7 of `bits` -> masks of the halves of four words of two logits each.
__device__ __forceinline__ void spread(uint32_t bits, uint32_t (&m)[4]) {
#pragma unroll
  for (int n = 0; n < 2; ++n) {
    const uint32_t x = (bits >> (4 * n) & 15u) * (0x00204081u << 7) & 0x80808080u;  // bit k to the top of byte k
    asm("prmt.b32 %0, %1, 0, 0x9988;" : "=r"(m[2 * n]) : "r"(x));                // which fills its half
    asm("prmt.b32 %0, %1, 0, 0xBBAA;" : "=r"(m[2 * n + 1]) : "r"(x));
  }
}
__device__ __forceinline__ uint32_t choose(uint32_t m, uint32_t x, uint32_t y) { return (x & m) | (y & ~m); }

// kVec tokens per thread and step: 8 (V a multiple of 8, 16-byte accesses) or 1.
template <int kVec>
__global__ void __launch_bounds__(kThreads, 4) logits_kernel(const LogitsArgs a) {
  extern __shared__ __align__(16) uint32_t count[];  // [range] occurrences, kSeen for those of the prompt; [range] bias
  uint32_t* biased = count + a.range;
  __shared__ int32_t sdraft[QSPEC_MAX_GAMMA];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int b = blockIdx.y;
  const int v0 = blockIdx.x * a.range;
  const int nv = min(a.V - v0, a.range);
  bool bad = false;

  // the rows come to L2 while the lists are counted (V and nv: multiples of 8)
  if (kVec == 8 && threadIdx.x < a.rows)
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(a.logits + (static_cast<int64_t>(b) * a.rows + threadIdx.x) * a.V + v0),
                 "r"(nv * 2)
                 : "memory");
  const int words = a.range / 4 * (a.n_bias ? 2 : 1);  // of 16 bytes
  for (int i = threadIdx.x; i < words; i += kThreads) reinterpret_cast<uint4*>(count)[i] = make_uint4(0, 0, 0, 0);
  const int n_draft = a.draft ? a.rows - 1 : 0;
  if (threadIdx.x < n_draft) {
    const int32_t t = a.draft[static_cast<int64_t>(b) * n_draft + threadIdx.x];
    bad |= t < 0 || t >= a.V;
    sdraft[threadIdx.x] = t;
  }
  Penalty p{1.0f, 1.0f, 0.0f, 0.0f, false};
  if (a.pen) {
    p = Penalty{a.pen[3 * b], 1.0f, a.pen[3 * b + 1], a.pen[3 * b + 2], false};
    if (!(p.rep > 0.0f)) {
      bad = true;
      p.rep = 1.0f;
    }
    p.inv = 1.0f / p.rep;
    p.divide = !(p.rep >= 0x1p-126f && p.rep <= 0x1p126f);
  }
  __syncthreads();
  if (a.hist && a.pen) {
    const int len = a.hist_len[b], prompt = a.prompt_len ? a.prompt_len[b] : 0;
    bad |= len < 0 || len > a.hist_stride || prompt < 0 || prompt > len;
    // (unsigned indices: a history of almost 2^31 tokens and the 2048 of a step stay below 2^32)
    const uint32_t n = static_cast<uint32_t>(min(static_cast<int64_t>(max(len, 0)), a.hist_stride));
    const uint32_t n_prompt = static_cast<uint32_t>(max(prompt, 0));
    const int32_t* h = a.hist + static_cast<int64_t>(b) * a.hist_stride;
    constexpr int kAtOnce = 8;
    for (uint32_t i0 = threadIdx.x; i0 < n; i0 += kAtOnce * kThreads) {
      int32_t t[kAtOnce];
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) t[k] = i0 + k * kThreads < n ? h[i0 + k * kThreads] : v0 + nv;  // (of another block)
      if (blockIdx.x == 0) {  // (one block's check is enough)
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) bad |= i0 + k * kThreads < n && (t[k] < 0 || t[k] >= a.V);
      }
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) {
        const uint32_t at = static_cast<uint32_t>(t[k]) - static_cast<uint32_t>(v0);
        if (at < static_cast<uint32_t>(nv)) {
          if (i0 + k * kThreads < n_prompt)
            atomicOr(count + at, kSeen);
          else
            atomicAdd(count + at, 1u);
        }
      }
    }
  }
  const float* bias = a.bias + static_cast<int64_t>(b) * a.n_bias;
  for (int i = threadIdx.x; i < a.n_bias; i += kThreads) {
    const int32_t t = a.bias_ids[static_cast<int64_t>(b) * a.n_bias + i];
    bad |= t >= a.V;
    const uint32_t at = static_cast<uint32_t>(t) - static_cast<uint32_t>(v0);
    if (t >= 0 && at < static_cast<uint32_t>(nv)) atomicMax(biased + at, kEntry + i);
  }
  if (bad && blockIdx.x == 0) atomicOr(a.err, kErrInvalid);  // (every block of the sequence sees the same lists)
  __syncthreads();
  if (a.n_bias) {  // the last entry of an id puts its bias in place
    for (int i = threadIdx.x; i < a.n_bias; i += kThreads) {
      const int32_t t = a.bias_ids[static_cast<int64_t>(b) * a.n_bias + i];
      const uint32_t at = static_cast<uint32_t>(t) - static_cast<uint32_t>(v0);
      if (t >= 0 && at < static_cast<uint32_t>(nv) && biased[at] == kEntry + i) {
        const float x = bias[i];
        biased[at] = x != x ? 0x7FFFFFFFu : __float_as_uint(x);
      }
    }
    __syncthreads();
  }

  const int mask_words = (a.V + 31) / 32;
  uint32_t drafted = 0;  // bit r: row r is the first to count a draft token of this block's range
  if (a.pen)
    for (int r = 1; r <= n_draft; ++r)
      if (static_cast<uint32_t>(sdraft[r - 1]) - static_cast<uint32_t>(v0) < static_cast<uint32_t>(nv)) drafted |= 1u << r;
  const int64_t row0 = static_cast<int64_t>(b) * a.rows;
  if (kVec == 8 && !p.divide) {
    for (int i0 = (threadIdx.x & ~31) * 8; i0 < nv; i0 += kThreads * 8) {  // 256 tokens of a warp
      const int lane = threadIdx.x & 31, i = i0 + 8 * lane;
      const bool in = i < nv;
      uint32_t seen = 0, touched = 0;  // bit e: token i + e
      float sub[8];
      auto bias_of = [&](int e) {
        return a.n_bias ? __uint_as_float(biased[i + e]) : 0.0f;
      };
#pragma unroll
      for (int e = 0; e < 8; ++e) sub[e] = 0.0f;
      if (in) {
        const uint4 lo = *reinterpret_cast<const uint4*>(count + i), hi = *reinterpret_cast<const uint4*>(count + i + 4);
        uint4 blo = make_uint4(0, 0, 0, 0), bhi = blo;
        if (a.n_bias) {
          blo = *reinterpret_cast<const uint4*>(biased + i);
          bhi = *reinterpret_cast<const uint4*>(biased + i + 4);
        }
        const uint32_t c[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
        const uint32_t bs[8] = {blo.x, blo.y, blo.z, blo.w, bhi.x, bhi.y, bhi.z, bhi.w};
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          if (c[e]) seen |= 1u << e;
          if (c[e] | bs[e]) {
            touched |= 1u << e;
            sub[e] = p.sub(c[e], __uint_as_float(bs[e]));
          }
        }
      }
      uint32_t any = __reduce_or_sync(0xFFFFFFFFu, touched);  // the places that some lane of the warp has touched
      uint32_t tm[4];
      spread(touched, tm);
      const uint16_t* src = a.logits + row0 * a.V + v0 + i;
      uint16_t* dst = a.out + row0 * a.V + v0 + i;
      const uint8_t* bits = reinterpret_cast<const uint8_t*>(a.mask) + row0 * mask_words * 4 + ((v0 + i) >> 3);
      constexpr int kAtOnce = 2;  // rows whose loads are in flight together ([64, 8, 152064]: 80 us; one: 85, four: 87)
      for (int r0 = 0; r0 < a.rows; r0 += kAtOnce) {
        uint4 w[kAtOnce];
        uint32_t allowed[kAtOnce];
#pragma unroll
        for (int q = 0; q < kAtOnce; ++q)
          if (in && r0 + q < a.rows) {
            w[q] = load_once(src + static_cast<int64_t>(r0 + q) * a.V);
            if (a.mask) allowed[q] = bits[static_cast<int64_t>(r0 + q) * mask_words * 4];
          }
#pragma unroll
        for (int q = 0; q < kAtOnce; ++q) {
          const int r = r0 + q;
          if (r >= a.rows) break;
          if (drafted >> r & 1u) {
            const uint32_t at = static_cast<uint32_t>(sdraft[r - 1]) - static_cast<uint32_t>(v0 + i0);
            if (at < 256u) {  // the row before drafted one of the warp's tokens
#pragma unroll
              for (int e = 0; e < 8; ++e)
                if (at == static_cast<uint32_t>(8 * lane + e)) {
                  const uint32_t c = one_more(count[i + e]);  // (the entry is this thread's)
                  count[i + e] = c;
                  sub[e] = p.sub(c, bias_of(e));
                  seen |= 1u << e;
                  touched |= 1u << e;
                }
              any = __reduce_or_sync(0xFFFFFFFFu, touched);
              spread(touched, tm);
            }
          }
          uint32_t u[4] = {w[q].x, w[q].y, w[q].z, w[q].w};
          if (any) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (any >> (2 * e) & 3u) {
                const float lo = p.adjust(bf16_lo(u[e]), seen >> (2 * e) & 1u, sub[2 * e]);
                const float hi = p.adjust(bf16_hi(u[e]), seen >> (2 * e + 1) & 1u, sub[2 * e + 1]);
                u[e] = choose(tm[e], pack_bf16(lo, hi), u[e]);  // (untouched ones keep their bits)
              }
          }
          if (a.mask) {
            uint32_t m[4];
            spread(allowed[q], m);
#pragma unroll
            for (int e = 0; e < 4; ++e) u[e] = choose(m[e], u[e], 0xFF80FF80u);
          }
          if (in) *reinterpret_cast<uint4*>(dst + static_cast<int64_t>(r) * a.V) = make_uint4(u[0], u[1], u[2], u[3]);
        }
      }
    }
  } else {
    for (int i = threadIdx.x; i < nv; i += kThreads) {
      uint32_t c = count[i];
      const uint32_t bs = a.n_bias ? biased[i] : 0u;
      for (int r0 = 0; r0 < a.rows; r0 += 4) {
        uint16_t w[4];
        uint32_t allowed[4];
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (r0 + q < a.rows) {
            const int64_t row = row0 + r0 + q;
            w[q] = a.logits[row * a.V + v0 + i];
            allowed[q] = a.mask ? reinterpret_cast<const uint8_t*>(a.mask + row * mask_words)[(v0 + i) >> 3] >> ((v0 + i) & 7) : 1u;
          }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int r = r0 + q;
          if (r >= a.rows) break;
          if ((drafted >> r & 1u) && sdraft[r - 1] == v0 + i) c = one_more(c);
          uint16_t x = w[q];
          if (c | bs) {
            const float sub = p.sub(c, __uint_as_float(bs));
            x = f32_to_bf16_bits(p.divide ? p.adjust_dividing(bf16_lo(x), c != 0, sub) : p.adjust(bf16_lo(x), c != 0, sub));
          }
          if (!(allowed[q] & 1u)) x = 0xFF80u;
          a.out[(row0 + r) * a.V + v0 + i] = x;
        }
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
  if (!bias) n_bias = 0;
  if (rows > QSPEC_MAX_GAMMA + 1 || n_bias > 65535 || V < 2 || V > QSPEC_MAX_V || B > 65535 ||
      int64_t(B) * rows * int64_t(V) >= (int64_t(1) << 40) || hist_stride > 0x7FFFFFFF)
    return QSPEC_ERR_UNSUPPORTED_SHAPE;
  if (!aligned16(logits) || !aligned16(out) || !aligned4(draft_tok) || !aligned4(hist) || !aligned4(hist_len) ||
      !aligned4(prompt_len) || !aligned4(penalties) || !aligned4(bias_ids) || !aligned4(bias) || !aligned4(mask))
    return QSPEC_ERR_MISALIGNED;
  LogitsArgs a{logits, out, draft_tok, hist, hist_len, prompt_len, penalties, bias_ids, bias, mask,
               linear_error_word(), hist_stride, rows, V, n_bias};
  if (!a.err) return QSPEC_ERR_CUDA;
  // Every block reads its sequence's whole history, so ranges are as long as leaves four blocks an SM ([64, 8, 152064]
  // with histories of 8192: 80 us with ranges of 4096, 81 with 8192); one sequence's rows take the shortest.
  a.range = 1024;
  while (a.range < 4096 && static_cast<int64_t>(B) * ((V + 2 * a.range - 1) / (2 * a.range)) >= 4 * num_sms()) a.range *= 2;
  const dim3 grid((V + a.range - 1) / a.range, B);
  const size_t smem = static_cast<size_t>(a.range) * (a.n_bias ? 8 : 4);  // at most 32 KB
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  auto kernel = V % 8 == 0 ? logits_kernel<8> : logits_kernel<1>;
  return launch_pdl(kernel, grid, dim3(kThreads), smem, s, a);
}
