// Appends a step's keys and values to the paged cache of e4m3 codes, rotating keys and queries on the way.
//
// value = code * 2^exp with one exponent per (page, head) for the keys and one for the values: the
// smallest e with amax <= 448 * 2^e.  Power-of-two scales make both directions exact but for the one
// rounding to e4m3.  A page that has to grow is quantised again by a shift: codes that stay in e4m3's normal range keep
// their values, those that fall below it are rounded once more.  Each value is read
// once (2 bytes) and its code written once (1 byte); memory bounds long appends, launch latency short
// ones.  A block owns one side (keys or values) of one (sequence, touched page) and up to four heads: it holds the page's new
// values in registers (at most 8 items of 16 a thread), so the maximum, the rounding and the writes need one
// pass over memory and no block waits for another.  Further blocks of the same launch rotate the queries
// of the page's tokens, up to 8 heads each, with the cosines of a token computed once for them.
#include "kv_internal.h"

namespace qspec {
namespace {

constexpr int kThreads = 256;
constexpr int kHeadsPerQ = 8;  // in passes of 4

struct AppendArgs {
  qspec_kv_cache c;
  qspec_kv_batch b;
  const uint16_t* k;
  const uint16_t* v;
  const uint16_t* q;
  uint16_t* q_out;
  const int32_t* pos;
  const uint64_t* turns;  // null: no rotation
  unsigned int* err;
  int64_t k_token, v_token, q_token, q_out_token;
  int rot, interleaved, group, pages_per_seq;  // group: query heads per key head
  float mult;
};

// Item j of a head of D values: two chunks of 8 values.  In the half layout the chunks of rotating items
// are rot / 2 apart (rot a multiple of 16), else they follow one another.
__device__ __forceinline__ void item_chunks(int j, int rot, bool half, int& d0, int& d1) {
  if (half && 16 * j < rot) {
    d0 = 8 * j;
    d1 = rot / 2 + 8 * j;
  } else {
    d0 = 16 * j;
    d1 = 16 * j + 8;
  }
}

// cos and sin (times mult) of the item's 8 pairs; pairs beyond rot / 2 do not rotate.
__device__ __forceinline__ void item_angles(const AppendArgs& a, int j, int32_t pos, float2 (&cs)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int p = 8 * j + i;
    if (p < a.rot / 2) {
      cs[i] = rotary_cos_sin(__ldg(a.turns + p), pos);
      cs[i].x *= a.mult;
      cs[i].y *= a.mult;
    } else {
      cs[i] = make_float2(1.0f, 0.0f);
    }
  }
}

__device__ __forceinline__ void item_rotate(const float2 (&cs)[8], bool half, int rot, int j, uint4& c0, uint4& c1) {
  uint32_t* w0 = reinterpret_cast<uint32_t*>(&c0);
  uint32_t* w1 = reinterpret_cast<uint32_t*>(&c1);
  if (half) {
    if (16 * j >= rot) return;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float a0 = bf16_lo(w0[i]), a1 = bf16_hi(w0[i]), b0 = bf16_lo(w1[i]), b1 = bf16_hi(w1[i]);
      const float2 p = cs[2 * i], q = cs[2 * i + 1];
      w0[i] = pack_bf16(a0 * p.x - b0 * p.y, a1 * q.x - b1 * q.y);
      w1[i] = pack_bf16(a0 * p.y + b0 * p.x, a1 * q.y + b1 * q.x);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint32_t& w = i < 4 ? w0[i] : w1[i - 4];
      if (8 * j + i < rot / 2) {
        const float a = bf16_lo(w), b = bf16_hi(w);
        w = pack_bf16(a * cs[i].x - b * cs[i].y, a * cs[i].y + b * cs[i].x);
      }
    }
  }
}

// Largest |value| of a bf16 pair as bf16 bits; non-finite values are replaced by 0.
__device__ __forceinline__ uint32_t amax_finite(uint32_t& w, bool& bad) {
  uint32_t lo = w & 0x7FFFu, hi = (w >> 16) & 0x7FFFu;
  if (lo >= 0x7F80u) {
    bad = true;
    lo = 0;
    w &= 0xFFFF0000u;
  }
  if (hi >= 0x7F80u) {
    bad = true;
    hi = 0;
    w &= 0x0000FFFFu;
  }
  return max(lo, hi);
}

// The smallest e with amax <= 448 * 2^e = 1.75 * 2^(e + 8), limited to the stored range.
__device__ __forceinline__ int exp_of_amax(uint32_t bits) {
  const int e = static_cast<int>(bits >> 7) - 127 - ((bits & 0x7Fu) <= 0x60u ? 8 : 7);
  return min(max(e, kKvMinExp), kKvMaxExp);
}

// NI: items of a head per thread at most (page * D / 16 values over 256 threads); HB: heads of a block, whose tokens' cosines
// are computed once for all of them.
template <int D, int NI, int HB>
__global__ void __launch_bounds__(kThreads) append_kernel(const AppendArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  constexpr int kPerTok = D / 16;  // items of a token and head
  const int b = blockIdx.x / a.pages_per_seq, jp = blockIdx.x - b * a.pages_per_seq;
  const int head0 = blockIdx.y * HB, heads = min(HB, a.c.heads - head0), role = blockIdx.z;
  const SeqSpan sp = seq_span(a.b, a.c.page, b);
  if (!sp.ok || sp.n > sp.kv) {
    if (threadIdx.x == 0) atomicOr(a.err, kErrInvalid);
    return;
  }
  const int P = a.c.page;
  const int start = sp.kv - sp.n;
  const int pg = start / P + jp;
  const int first = max(start, pg * P), last = min(sp.kv, pg * P + P);  // positions written in this page
  const int n = last - first;
  if (n <= 0) return;
  const int tok = sp.tok0 + (first - start);  // the step's index of the first of them
  const bool half = !a.interleaved;

  if (role >= 2) {
    // ------------------------------------------------------------------ queries
    const int h0 = head0 * a.group + (role - 2) * kHeadsPerQ;
    const int nh = min(kHeadsPerQ, (head0 + heads) * a.group - h0);
    for (int i = threadIdx.x; i < n * kPerTok; i += kThreads) {
      const int t = i / kPerTok, j = i - t * kPerTok;
      int d0, d1;
      item_chunks(j, a.rot, half, d0, d1);
      const uint16_t* src = a.q + static_cast<int64_t>(tok + t) * a.q_token + static_cast<int64_t>(h0) * D;
      uint16_t* dst = a.q_out + static_cast<int64_t>(tok + t) * a.q_out_token + static_cast<int64_t>(h0) * D;
      float2 cs[8];
      if (a.turns) item_angles(a, j, a.pos ? a.pos[tok + t] : first + t, cs);
#pragma unroll 1
      for (int g = 0; g < nh; g += 4) {
        uint4 v[4][2];
#pragma unroll
        for (int h = 0; h < 4; ++h)
          if (g + h < nh) {
            v[h][0] = *reinterpret_cast<const uint4*>(src + (g + h) * D + d0);
            v[h][1] = *reinterpret_cast<const uint4*>(src + (g + h) * D + d1);
          }
#pragma unroll
        for (int h = 0; h < 4; ++h)
          if (g + h < nh) {
            if (a.turns) item_rotate(cs, half, a.rot, j, v[h][0], v[h][1]);
            *reinterpret_cast<uint4*>(dst + (g + h) * D + d0) = v[h][0];
            *reinterpret_cast<uint4*>(dst + (g + h) * D + d1) = v[h][1];
          }
      }
    }
    return;
  }

  // -------------------------------------------------------------------- keys (role 0) or values (role 1)
  const int page = a.b.pages[static_cast<int64_t>(b) * a.b.max_pages + pg];
  if (page < 0 || page >= a.c.n_pages) {
    if (threadIdx.x == 0) atomicOr(a.err, kErrInvalid);
    return;
  }
  const int64_t ph = static_cast<int64_t>(page) * a.c.heads + head0;
  uint8_t* codes = (role == 0 ? a.c.k : a.c.v) + ph * P * D;  // of the block's first head; P * D to the next
  int8_t* exp_at = (role == 0 ? a.c.k_exp : a.c.v_exp) + ph;
  const uint16_t* src = (role == 0 ? a.k : a.v) + static_cast<int64_t>(head0) * D;
  const int64_t stride = role == 0 ? a.k_token : a.v_token;
  const bool rotate = role == 0 && a.turns != nullptr;
  const int items = n * kPerTok;

  uint4 v[NI][HB][2];
#pragma unroll
  for (int it = 0; it < NI; ++it) {
    const int i = it * kThreads + threadIdx.x;
    if (i < items) {
      const int t = i / kPerTok, j = i - t * kPerTok;
      int d0, d1;
      item_chunks(j, a.rot, half && rotate, d0, d1);
      const uint16_t* s = src + static_cast<int64_t>(tok + t) * stride;
#pragma unroll
      for (int h = 0; h < HB; ++h)
        if (h < heads) {
          v[it][h][0] = *reinterpret_cast<const uint4*>(s + h * D + d0);
          v[it][h][1] = *reinterpret_cast<const uint4*>(s + h * D + d1);
        }
    }
  }
  const bool begun = first == pg * P;  // slot 0 is among the new ones
  int old[HB];
#pragma unroll
  for (int h = 0; h < HB; ++h)
    old[h] = begun || h >= heads ? kKvMinExp : min(max(static_cast<int>(exp_at[h]), kKvMinExp), kKvMaxExp);
  uint32_t amax[HB] = {};
  bool bad = false;
#pragma unroll
  for (int it = 0; it < NI; ++it) {
    const int i = it * kThreads + threadIdx.x;
    if (i < items) {
      float2 cs[8];
      const int t = i / kPerTok, j = i - t * kPerTok;
      if (rotate) item_angles(a, j, a.pos ? a.pos[tok + t] : first + t, cs);
#pragma unroll
      for (int h = 0; h < HB; ++h)
        if (h < heads) {
          if (rotate) item_rotate(cs, half, a.rot, j, v[it][h][0], v[it][h][1]);
          uint32_t* w = reinterpret_cast<uint32_t*>(&v[it][h][0]);
#pragma unroll
          for (int e = 0; e < 8; ++e) amax[h] = max(amax[h], amax_finite(w[e], bad));
        }
    }
  }
  __shared__ uint32_t sh[HB][kThreads / 32];
#pragma unroll
  for (int h = 0; h < HB; ++h) {
    amax[h] = __reduce_max_sync(0xFFFFFFFFu, amax[h]);
    if ((threadIdx.x & 31) == 0) sh[h][threadIdx.x >> 5] = amax[h];
  }
  if (bad) atomicOr(a.err, kErrInvalid);
  __syncthreads();
#pragma unroll
  for (int h = 0; h < HB; ++h) {
    if (h >= heads) break;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) amax[h] = max(amax[h], sh[h][w]);
    const int e = max(old[h], exp_of_amax(amax[h]));
    uint8_t* at_head = codes + h * P * D;

    if (!begun && e > old[h]) {  // the page grows: its other slots again
      const float shrink = exp2_int(old[h] - e);
      for (int i = threadIdx.x; i < P * kPerTok; i += kThreads) {
        const int slot = i / kPerTok + pg * P;
        if (slot >= first && slot < last) continue;
        uint4* at = reinterpret_cast<uint4*>(at_head) + i;
        uint4 c = *at;
        uint32_t* w = reinterpret_cast<uint32_t*>(&c);
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          const float2 lo = e4m3x2_to_f32(w[m] & 0xFFFFu), hi = e4m3x2_to_f32(w[m] >> 16);
          w[m] = f32_to_e4m3x2(lo.x * shrink, lo.y * shrink) | f32_to_e4m3x2(hi.x * shrink, hi.y * shrink) << 16;
        }
        *at = c;
      }
    }
    const float inv = exp2_int(-e);
#pragma unroll
    for (int it = 0; it < NI; ++it) {
      const int i = it * kThreads + threadIdx.x;
      if (i < items) {
        const int t = i / kPerTok, j = i - t * kPerTok;
        int d0, d1;
        item_chunks(j, a.rot, half && rotate, d0, d1);
        uint8_t* dst = at_head + (first - pg * P + t) * D;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const uint32_t* w = reinterpret_cast<const uint32_t*>(&v[it][h][c]);
          uint2 o;
          o.x = f32_to_e4m3x2(bf16_lo(w[0]) * inv, bf16_hi(w[0]) * inv) |
                f32_to_e4m3x2(bf16_lo(w[1]) * inv, bf16_hi(w[1]) * inv) << 16;
          o.y = f32_to_e4m3x2(bf16_lo(w[2]) * inv, bf16_hi(w[2]) * inv) |
                f32_to_e4m3x2(bf16_lo(w[3]) * inv, bf16_hi(w[3]) * inv) << 16;
          *reinterpret_cast<uint2*>(dst + (c == 0 ? d0 : d1)) = o;
        }
      }
    }
    if (threadIdx.x == 0) exp_at[h] = static_cast<int8_t>(e);
  }
}

template <int D, int NI, int HB>
qspec_status launch_append(const AppendArgs& a, unsigned int blocks, cudaStream_t s) {
  const dim3 grid(blocks, (a.c.heads + HB - 1) / HB, 2 + (HB * a.group + kHeadsPerQ - 1) / kHeadsPerQ);
  return launch_pdl(append_kernel<D, NI, HB>, grid, dim3(kThreads), 0, s, a);
}

}  // namespace
}  // namespace qspec

using namespace qspec;

extern "C" qspec_status qspec_kv_append(const qspec_kv_cache* cache, const qspec_kv_batch* batch, const uint16_t* k,
                                        int64_t k_token, const uint16_t* v, int64_t v_token,
                                        const qspec_rotary_plan* plan, const int32_t* pos, const uint16_t* q,
                                        int64_t q_token, int32_t heads_q, uint16_t* q_out, int64_t q_out_token,
                                        qspec_stream_t stream) {
  if (!k || !v || (q && !q_out)) return QSPEC_ERR_INVALID_ARG;
  qspec_status st = check_kv(cache, batch);
  if (st != QSPEC_OK) return st;
  const int64_t row = static_cast<int64_t>(cache->heads) * cache->dim;
  if ((st = check_rows(k, batch->T, row, k_token)) != QSPEC_OK) return st;
  if ((st = check_rows(v, batch->T, row, v_token)) != QSPEC_OK) return st;
  if (plan) {
    if ((st = check_rotary_plan(plan, cache->dim)) != QSPEC_OK) return st;
    if (!plan->interleaved && plan->rot % 16 != 0) return QSPEC_ERR_UNSUPPORTED_SHAPE;
  }
  if (pos && !aligned4(pos)) return QSPEC_ERR_MISALIGNED;
  if (q) {
    if (heads_q <= 0) return QSPEC_ERR_INVALID_ARG;
    if (heads_q % cache->heads != 0 || heads_q / cache->heads > 128) return QSPEC_ERR_UNSUPPORTED_SHAPE;
    const int64_t q_row = static_cast<int64_t>(heads_q) * cache->dim;
    if ((st = check_rows(q, batch->T, q_row, q_token)) != QSPEC_OK) return st;
    if ((st = check_rows(q_out, batch->T, q_row, q_out_token)) != QSPEC_OK) return st;
  }
  AppendArgs a{*cache, *batch, k, v, q, q_out, pos, plan ? plan->turns : nullptr, linear_error_word(),
               k_token, v_token, q_token, q_out_token};
  if (!a.err) return QSPEC_ERR_CUDA;
  a.rot = plan ? plan->rot : 0;
  a.interleaved = plan ? plan->interleaved : 1;
  a.mult = plan ? plan->mult : 1.0f;
  a.group = q ? heads_q / cache->heads : 0;
  a.pages_per_seq = (batch->max_tok + cache->page - 2) / cache->page + 1;  // a span of max_tok tokens touches at most
  const int64_t blocks = static_cast<int64_t>(batch->B) * a.pages_per_seq;
  if (blocks > 0x7FFFFFFF) return QSPEC_ERR_UNSUPPORTED_SHAPE;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  // Heads to a block: as many (4 at most) as 64 registers of values a thread hold; the cosines of a token are
  // computed once for them (about 10000 tokens, 32 + 8 + 8 heads: 46 us with one head to a block, 43 with four).
  const unsigned int n = static_cast<unsigned int>(blocks);
  if (cache->dim == 128)
    return cache->page == 128 ? launch_append<128, 4, 2>(a, n, s) : cache->page == 64 ? launch_append<128, 2, 4>(a, n, s)
                                                                                      : launch_append<128, 1, 4>(a, n, s);
  return cache->page == 128 ? launch_append<64, 2, 4>(a, n, s) : launch_append<64, 1, 4>(a, n, s);
}
