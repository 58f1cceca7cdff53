// Shared by the rotary, cache, attention and logits kernels: the angle of a rotary pair, the checks of
// the cache and batch descriptors.  Bad values on the device set kErrInvalid in the library's error word.
#pragma once

#include <math.h>

#include "common.cuh"
#include "linear_internal.h"

namespace qspec {

constexpr int kKvMinExp = QSPEC_KV_MIN_EXP, kKvMaxExp = QSPEC_KV_MAX_EXP;

// cos and sin of pos * (turns / 2^64) full turns.  The product modulo 2^64 is the exact fraction of a
// turn; its top 32 bits, read as signed, are the angle in [-pi, pi).  Rounded to fp32 it is off by about 2^-26 turns at most.
__device__ __forceinline__ float2 rotary_cos_sin(uint64_t turns, int32_t pos) {
  const uint64_t phase = static_cast<uint64_t>(static_cast<int64_t>(pos)) * turns;
  const float half_turns = static_cast<float>(static_cast<int32_t>(phase >> 32)) * 0x1p-31f;
  float2 cs;
  sincospif(half_turns, &cs.y, &cs.x);
  return cs;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Where sequence b's new tokens lie; `ok` false (and the error bit set) if its numbers are out of range.
struct SeqSpan {
  int tok0, n, kv;
  bool ok;
};
__device__ __forceinline__ SeqSpan seq_span(const qspec_kv_batch& bt, int page, int b) {
  SeqSpan s;
  s.tok0 = bt.cu_tok[b];
  const int t1 = bt.cu_tok[b + 1];
  s.kv = bt.kv_len[b];
  s.n = t1 - s.tok0;
  s.ok = s.tok0 >= 0 && t1 >= s.tok0 && t1 <= bt.T && s.n <= bt.max_tok && s.kv >= 0 &&
         static_cast<int64_t>(s.kv) <= static_cast<int64_t>(bt.max_pages) * page;
  if (!s.ok) s.n = 0;
  return s;
}

// e4m3 code pairs (low byte first) <-> fp16 pairs (exact) and from fp32 pairs (nearest even, saturating).
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t two) {
  uint32_t r;
  asm("{\n\t.reg .b16 t;\n\tcvt.u16.u32 t, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}" : "=r"(r) : "r"(two));
  return r;
}
// Four codes -> two fp16 pairs.
__device__ __forceinline__ void e4m3x4_to_f16x4(uint32_t four, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 l, h;\n\t"
      "mov.b32 {l, h}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(four));
}
__device__ __forceinline__ float2 e4m3x2_to_f32(uint32_t two) {
  const uint32_t h = e4m3x2_to_f16x2(two);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
__device__ __forceinline__ uint32_t f32_to_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// 2^e for |e| <= 126.
__device__ __forceinline__ float exp2_int(int e) { return __int_as_float((127 + e) << 23); }

// n 32-bit words of memory (p null: none).
struct Words {
  const void* p;
  int64_t n;
};
// An output shares a word with an input or another output.
inline bool outputs_overlap(const Words* out, int n_out, const Words* in, int n_in) {
  auto meet = [](const Words& x, const Words& y) {
    const char *a = static_cast<const char*>(x.p), *b = static_cast<const char*>(y.p);
    return a && b && a < b + 4 * y.n && b < a + 4 * x.n;
  };
  for (int i = 0; i < n_out; ++i) {
    for (int j = 0; j < i; ++j)
      if (meet(out[i], out[j])) return true;
    for (int j = 0; j < n_in; ++j)
      if (meet(out[i], in[j])) return true;
  }
  return false;
}

inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

inline qspec_status check_rotary_plan(const qspec_rotary_plan* p, int32_t dim) {
  if (!p->turns || p->reserved != 0 || !isfinite(p->mult)) return QSPEC_ERR_INVALID_ARG;
  if (p->rot < 2 || p->rot % 2 != 0 || p->rot > dim) return QSPEC_ERR_UNSUPPORTED_SHAPE;
  if ((reinterpret_cast<uintptr_t>(p->turns) & 7u) != 0) return QSPEC_ERR_MISALIGNED;
  return QSPEC_OK;
}

// A strided [T, row] operand: rows of `row` values, `stride` apart.
inline qspec_status check_rows(const void* p, int64_t T, int64_t row, int64_t stride) {
  if (stride < row || stride > (int64_t(1) << 40) / T) return QSPEC_ERR_UNSUPPORTED_SHAPE;
  if (!aligned16(p) || stride % 8 != 0) return QSPEC_ERR_MISALIGNED;
  return QSPEC_OK;
}

inline qspec_status check_kv(const qspec_kv_cache* c, const qspec_kv_batch* b) {
  if (!c || !b || !c->k || !c->v || !c->k_exp || !c->v_exp || !b->cu_tok || !b->kv_len || !b->pages)
    return QSPEC_ERR_INVALID_ARG;
  if (c->reserved != 0 || b->reserved != 0 || c->n_pages <= 0 || c->heads <= 0 || b->B <= 0 || b->max_pages <= 0 ||
      b->max_tok <= 0 || b->T <= 0)
    return QSPEC_ERR_INVALID_ARG;
  if ((c->page != 16 && c->page != 32 && c->page != 64 && c->page != 128) || (c->dim != 64 && c->dim != 128) ||
      c->heads > 4096 || c->n_pages > 0x7FFFFFFF || b->B > QSPEC_KV_MAX_B || b->T > 0x7FFFFFFF || b->max_tok > b->T ||
      static_cast<int64_t>(b->max_pages) * c->page > (int64_t(1) << 30))
    return QSPEC_ERR_UNSUPPORTED_SHAPE;
  if (!aligned16(c->k) || !aligned16(c->v) || !aligned4(b->cu_tok) || !aligned4(b->kv_len) || !aligned4(b->pages))
    return QSPEC_ERR_MISALIGNED;
  return QSPEC_OK;
}

}  // namespace qspec
