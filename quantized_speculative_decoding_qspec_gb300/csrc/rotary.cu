// Rotary positions: rotates pairs of values of every head by an angle proportional to the token's position.
//
// (a, b) -> mult (a cos t - b sin t, a sin t + b cos t), t = pos * w_i.  The frequencies are held as
// 64-bit fractions of a turn, so the range reduction is one integer product (kv_internal.h) and far
// positions lose nothing.  The operator reads and writes each value once (2 + 2 bytes) and is bound by
// memory, or by launch latency for a few tokens.  A block takes a few tokens: its threads compute the
// tokens' cosines and sines once into shared memory (one pair each) and then rotate all heads with
// 16-byte accesses; a thread holds both halves of its pairs, so in-place calls are safe.
#include "kv_internal.h"

namespace qspec {
namespace {

constexpr int kRotThreads = 256;

struct RotaryArgs {
  const uint16_t* x;
  uint16_t* out;
  const int32_t* pos;
  const uint64_t* turns;
  int64_t x_token, x_head, out_token, out_head;
  int64_t T;
  int heads, rot, tokens, heads_per_block, items;  // items: work items of a head
  float mult, sign;
};

enum { kHalf = 0, kInter = 1, kAny = 2, kAnyInter = 3 };

__device__ __forceinline__ uint32_t rotate_lo_hi(uint32_t w, float2 cs) {
  const float a = bf16_lo(w), b = bf16_hi(w);
  return pack_bf16(a * cs.x - b * cs.y, a * cs.y + b * cs.x);
}

// kHalf: an item is two chunks of 8 values rot/2 apart (rot a multiple of 16); kInter: one chunk of 8
// (rot a multiple of 8); both have one further item for each chunk that is only copied.  kAny and
// kAnyInter: one pair, or one copied value.
template <int kMode>
__global__ void __launch_bounds__(kRotThreads) rotary_kernel(const RotaryArgs a) {
  extern __shared__ float2 cs[];  // [tokens][rot / 2]
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * a.tokens;
  const int nt = a.T - t0 < a.tokens ? static_cast<int>(a.T - t0) : a.tokens;
  const int h0 = blockIdx.y * a.heads_per_block;
  const int nh = min(a.heads - h0, a.heads_per_block);
  const int half = a.rot / 2;
  for (int i = threadIdx.x; i < nt * half; i += kRotThreads) {
    const int t = i / half;
    float2 v = rotary_cos_sin(__ldg(a.turns + (i - t * half)), a.pos[t0 + t]);
    v.x *= a.mult;
    v.y *= a.mult * a.sign;
    cs[i] = v;
  }
  __syncthreads();
  constexpr int kChunk = kMode == kHalf ? 16 : 8;
  const int rot_items = kMode >= kAny ? half : a.rot / kChunk;
  if (kMode >= kAny) {
    const unsigned int n = static_cast<unsigned int>(nt) * nh * a.items;
    for (unsigned int e = threadIdx.x; e < n; e += kRotThreads) {
      const unsigned int r = e / a.items, j = e - r * a.items;
      const unsigned int t = r / nh, h = r - t * nh;
      const uint16_t* x = a.x + (t0 + t) * a.x_token + static_cast<int64_t>(h0 + h) * a.x_head;
      uint16_t* o = a.out + (t0 + t) * a.out_token + static_cast<int64_t>(h0 + h) * a.out_head;
      if (j >= rot_items) {
        const int d = a.rot + (j - rot_items);
        o[d] = x[d];
        continue;
      }
      const int da = kMode == kAny ? j : 2 * j, db = kMode == kAny ? j + half : 2 * j + 1;
      const uint32_t w = rotate_lo_hi(x[da] | static_cast<uint32_t>(x[db]) << 16, cs[t * half + j]);
      o[da] = static_cast<uint16_t>(w);
      o[db] = static_cast<uint16_t>(w >> 16);
    }
    return;
  }
  // A thread keeps its item j of a head and walks the (token, head) rows, `rows` of them at a time over the block;
  // kAtOnce rows' loads are in flight before the first is rotated.
  const int rows = kRotThreads / a.items, lane_row = threadIdx.x / a.items, j = threadIdx.x - lane_row * a.items;
  if (lane_row >= rows) return;
  const bool rotates = j < rot_items;
  const int d0 = rotates ? 8 * j : a.rot + 8 * (j - rot_items), d1 = half + d0;  // (d1: kHalf)
  const int64_t pair = kMode == kHalf && rotates ? 1 : 0;
  constexpr int kAtOnce = kMode == kHalf ? 2 : 4;
  int t = 0, h = lane_row;
  while (h >= nh) {
    h -= nh;
    ++t;
  }
  while (t < nt) {
    uint4 va[kAtOnce], vb[kAtOnce];
    int tt[kAtOnce], hh[kAtOnce];
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      tt[k] = t;
      hh[k] = h;
      if (t < nt) {
        const uint16_t* x = a.x + (t0 + t) * a.x_token + static_cast<int64_t>(h0 + h) * a.x_head;
        va[k] = *reinterpret_cast<const uint4*>(x + d0);
        if (pair) vb[k] = *reinterpret_cast<const uint4*>(x + d1);
      }
      h += rows;
      while (h >= nh) {
        h -= nh;
        ++t;
      }
    }
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      if (tt[k] >= nt) break;
      uint16_t* o = a.out + (t0 + tt[k]) * a.out_token + static_cast<int64_t>(h0 + hh[k]) * a.out_head;
      if (!rotates) {
        *reinterpret_cast<uint4*>(o + d0) = va[k];
      } else if (kMode == kInter) {
        const float4* c = reinterpret_cast<const float4*>(cs + tt[k] * half + 4 * j);  // (rot / 2 is a multiple of 4)
        const float4 c0 = c[0], c1 = c[1];
        const uint4 v = va[k];
        *reinterpret_cast<uint4*>(o + d0) =
            make_uint4(rotate_lo_hi(v.x, make_float2(c0.x, c0.y)), rotate_lo_hi(v.y, make_float2(c0.z, c0.w)),
                       rotate_lo_hi(v.z, make_float2(c1.x, c1.y)), rotate_lo_hi(v.w, make_float2(c1.z, c1.w)));
      } else {
        const uint32_t wa[4] = {va[k].x, va[k].y, va[k].z, va[k].w}, wb[4] = {vb[k].x, vb[k].y, vb[k].z, vb[k].w};
        const float4* c = reinterpret_cast<const float4*>(cs + tt[k] * half + 8 * j);
        uint32_t ra[4], rb[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float4 q = c[i];
          const float a0 = bf16_lo(wa[i]), a1 = bf16_hi(wa[i]), b0 = bf16_lo(wb[i]), b1 = bf16_hi(wb[i]);
          ra[i] = pack_bf16(a0 * q.x - b0 * q.y, a1 * q.z - b1 * q.w);
          rb[i] = pack_bf16(a0 * q.y + b0 * q.x, a1 * q.w + b1 * q.z);
        }
        *reinterpret_cast<uint4*>(o + d0) = make_uint4(ra[0], ra[1], ra[2], ra[3]);
        *reinterpret_cast<uint4*>(o + d1) = make_uint4(rb[0], rb[1], rb[2], rb[3]);
      }
    }
  }
}

// Whether two rows (token, head) of `dim` values share memory.  Tokens within a stride of heads, or heads within a
// stride of tokens, are told apart at once; other layouts are looked at head by head.
bool rows_overlap(int64_t T, int64_t heads, int64_t dim, int64_t token, int64_t head) {
  if ((T > 1 && token < dim) || (heads > 1 && head < dim)) return true;
  if (T == 1 || heads == 1 || token >= (heads - 1) * head + dim || head >= (T - 1) * token + dim) return false;
  for (int64_t j = 1; j < heads; ++j) {  // head j of one token against head 0 of the k-th after it
    const int64_t at = j * head, k = at / token;
    if (k < T && at - k * token < dim) return true;
    if (k + 1 < T && (k + 1) * token - at < dim) return true;
  }
  return false;
}

}  // namespace

}  // namespace qspec

using namespace qspec;

extern "C" qspec_status qspec_rotary_turns(int32_t rot, double base, int32_t scaling, double factor, double original,
                                           double low, double high, uint64_t* turns, float* mult) {
  constexpr double kTwoPi = 6.283185307179586476925286766559;
  if (!turns || !mult || rot <= 0 || !(base > 1.0) || !isfinite(base) || scaling < QSPEC_ROTARY_PLAIN ||
      scaling > QSPEC_ROTARY_YARN)
    return QSPEC_ERR_INVALID_ARG;
  if (rot % 2 != 0 || rot > 1024 || (scaling == QSPEC_ROTARY_BASE && rot < 4)) return QSPEC_ERR_UNSUPPORTED_SHAPE;
  if (scaling != QSPEC_ROTARY_PLAIN && (!(factor >= 1.0) || !isfinite(factor))) return QSPEC_ERR_INVALID_ARG;
  const bool ranges = scaling == QSPEC_ROTARY_BANDS || scaling == QSPEC_ROTARY_YARN;
  if (ranges && (!(original > 0.0) || !isfinite(original) || !(low > 0.0) || !(high > low) || !isfinite(high)))
    return QSPEC_ERR_INVALID_ARG;
  const double n = rot;
  if (scaling == QSPEC_ROTARY_BASE) base *= pow(factor, n / (n - 2.0));
  double first = 0.0, last = 0.0;  // the ramp of YARN, in pair indices
  if (scaling == QSPEC_ROTARY_YARN) {
    const double per = n / (2.0 * log(base));
    first = fmax(floor(per * log(original / (high * kTwoPi))), 0.0);
    last = fmin(ceil(per * log(original / (low * kTwoPi))), n - 1.0);
  }
  for (int i = 0; i < rot / 2; ++i) {
    double w = pow(base, -2.0 * i / n);
    if (scaling == QSPEC_ROTARY_LINEAR) w /= factor;
    if (scaling == QSPEC_ROTARY_BANDS) {
      const double keep = fmin(fmax((original * w / kTwoPi - low) / (high - low), 0.0), 1.0);
      w = (1.0 - keep) * w / factor + keep * w;
    }
    if (scaling == QSPEC_ROTARY_YARN) {
      const double ramp = fmin(fmax((i - first) / fmax(last - first, 1e-3), 0.0), 1.0);
      w = w / factor * ramp + w * (1.0 - ramp);
    }
    turns[i] = static_cast<uint64_t>(w / kTwoPi * 0x1p64);  // w <= 1: below a sixth of a turn
  }
  *mult = scaling == QSPEC_ROTARY_YARN ? static_cast<float>(0.1 * log(factor) + 1.0) : 1.0f;
  return QSPEC_OK;
}

extern "C" qspec_status qspec_rotary(const uint16_t* x, int64_t x_token, int64_t x_head, const int32_t* pos, int64_t T,
                                     int32_t heads, int32_t dim, const qspec_rotary_plan* plan, int32_t inverse,
                                     uint16_t* out, int64_t out_token, int64_t out_head, qspec_stream_t stream) {
  if (!x || !pos || !plan || !out || T <= 0 || heads <= 0 || dim <= 0) return QSPEC_ERR_INVALID_ARG;
  if (dim % 8 != 0 || dim > 1024 || heads > 65535 || T > 0x7FFFFFFF) return QSPEC_ERR_UNSUPPORTED_SHAPE;
  const qspec_status st = check_rotary_plan(plan, dim);
  if (st != QSPEC_OK) return st;
  if (x_token < 0 || x_head < 0 || out_token < 0 || out_head < 0) return QSPEC_ERR_UNSUPPORTED_SHAPE;
  const int64_t most = int64_t(1) << 40;
  if (x_token > most / T || out_token > most / T || x_head > most / heads || out_head > most / heads)
    return QSPEC_ERR_UNSUPPORTED_SHAPE;
  if (x_token % 8 || x_head % 8 || out_token % 8 || out_head % 8) return QSPEC_ERR_MISALIGNED;
  if (rows_overlap(T, heads, dim, out_token, out_head)) return QSPEC_ERR_UNSUPPORTED_SHAPE;
  if (!aligned16(x) || !aligned16(out) || !aligned4(pos)) return QSPEC_ERR_MISALIGNED;
  RotaryArgs a{x, out, pos, plan->turns, x_token, x_head, out_token, out_head, T, heads, plan->rot};
  a.mult = plan->mult;
  a.sign = inverse ? -1.0f : 1.0f;
  const bool inter = plan->interleaved != 0;
  const int mode = inter ? (a.rot % 8 == 0 ? kInter : kAnyInter) : (a.rot % 16 == 0 ? kHalf : kAny);
  const bool in_place = out == x && x_token == out_token && x_head == out_head;
  const int copied = in_place ? 0 : dim - a.rot;
  a.items = mode == kHalf ? a.rot / 16 + copied / 8 : mode == kInter ? a.rot / 8 + copied / 8 : a.rot / 2 + copied;
  // Four tokens a block once that still gives every SM a full set of blocks; below that one token a
  // block, and the heads split so that a block has about one item a thread.
  const int64_t full = 8 * num_sms();
  a.tokens = T >= 4 * full ? 4 : 1;
  const int64_t blocks = (T + a.tokens - 1) / a.tokens;
  a.heads_per_block = blocks >= full ? heads : (kRotThreads + a.items - 1) / a.items;
  if (a.heads_per_block > heads) a.heads_per_block = heads;
  const dim3 grid(static_cast<unsigned int>(blocks), (heads + a.heads_per_block - 1) / a.heads_per_block);
  const size_t smem = sizeof(float2) * a.tokens * (a.rot / 2);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  switch (mode) {
    case kHalf: return launch_pdl(rotary_kernel<kHalf>, grid, dim3(kRotThreads), smem, s, a);
    case kInter: return launch_pdl(rotary_kernel<kInter>, grid, dim3(kRotThreads), smem, s, a);
    case kAny: return launch_pdl(rotary_kernel<kAny>, grid, dim3(kRotThreads), smem, s, a);
    default: return launch_pdl(rotary_kernel<kAnyInter>, grid, dim3(kRotThreads), smem, s, a);
  }
}
