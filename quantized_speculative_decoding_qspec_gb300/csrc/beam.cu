// Beam selection: the n best of a sequence's beams times vocabulary by summed log probability.
//
//     S(k, v) = score[k] + (logit[k, v] - lse[k]),   lse[k] = ln sum_v exp(logit[k, v])
// Within a beam the order is that of its logits (bf16: ties are common, and go to the lowest token), so each beam offers its n
// largest logits, and the beams' offers are ordered by S (times a weight).  One pass over the logits bounds it: a CTA
// holds a tile of a row in registers, reduces maximum and sum of exponentials, and collects the few logits that
// reach a lower bound of its n-th largest.  The last CTA of a sequence (atomic ticket) merges the offers.
#include <math.h>

#include "kv_internal.h"

namespace qspec {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kVecs = 8;                          // 16-byte loads in flight a thread: 32 registers, two CTAs an SM
constexpr int kTileVecs = kThreads * kVecs;       // 32768 logits
constexpr int kTile = kTileVecs * 8;
constexpr int kList = 1024;                       // logits collected at most; more: see exact_bound
constexpr int kMaxN = QSPEC_BEAM_MAX_N, kMaxBeams = QSPEC_BEAM_MAX_BEAMS;
constexpr int kMaxLists = kThreads;               // (beam, chunk) pairs of a sequence: a thread each in the merge
constexpr int kStage = 4096;                      // offers of a sequence that are merged from shared memory
constexpr uint32_t kLowest = 0xFF80FF80u;         // two bf16 -inf

struct BeamArgs {
  const uint16_t* logits;
  const float* scores;
  const int32_t* done;
  const float* weights;
  int32_t* parent;
  int32_t* tok;
  float* score;
  unsigned int* err;
  unsigned int* tickets;        // [B]
  float2* stats;                // [B, K, chunks]: maximum, sum of exponentials
  unsigned long long* offers;   // [B, K, chunks, n]: ordered logit << 32 | ~token; 0: none
  long long total;              // logits in all
  int B, K, V, n, chunks, chunk_len, end_tok;
};

// bf16 bits -> 16-bit keys in the order of the values; both zeros alike, -inf 0x7F, NaN above +inf or below -inf.
__device__ __forceinline__ uint32_t ordered(uint32_t bits) {
  if (bits == 0x8000u) bits = 0;
  return bits & 0x8000u ? 0xFFFFu - bits : bits + 0x8000u;
}
__device__ __forceinline__ float value_of(uint32_t key) {
  return __uint_as_float((key & 0x8000u ? key - 0x8000u : 0xFFFFu - key) << 16);
}
constexpr uint32_t kKeyLowest = 0x7Fu, kKeyInf = 0xFF80u;

__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ float pow2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
constexpr float kLog2e = 1.44269504088896341f;

// An order-preserving map of doubles (no NaN) to integers, 0 below all of them.
__device__ __forceinline__ unsigned long long ordered64(double x) {
  const long long b = __double_as_longlong(x == 0.0 ? 0.0 : x);
  return static_cast<unsigned long long>(b < 0 ? ~b : b | (1ll << 63));
}

struct BeamShared {
  union {
    unsigned long long list[kList];
    unsigned long long stage[kStage];
  };
  unsigned long long top[kMaxN];
  uint32_t group[64];
  float2 warp_stat[kWarps];
  unsigned int counts[2];
  unsigned long long best[2][kWarps];
  int best_at[2][kWarps];
  double lse[kMaxBeams];
  int n_list, last;
};

struct Best {
  unsigned long long key;
  int at;
};
// The largest key of the warp, the lowest lane among equal ones.
__device__ __forceinline__ Best warp_best(unsigned long long key, int at) {
  const uint32_t hi = __reduce_max_sync(0xFFFFFFFFu, static_cast<uint32_t>(key >> 32));
  const uint32_t lo = __reduce_max_sync(0xFFFFFFFFu, static_cast<uint32_t>(key >> 32) == hi ? static_cast<uint32_t>(key) : 0u);
  const unsigned long long top = static_cast<unsigned long long>(hi) << 32 | lo;
  const int first = __reduce_min_sync(0xFFFFFFFFu, key == top ? at : 0x7FFFFFFF);
  return {top, first};
}

// The last CTA of sequence b: the beams' sums, then n times the best of what the lists offer next.
__device__ __noinline__ void merge(const BeamArgs& a, BeamShared& sh, int b) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int lists = a.K * a.chunks, count = lists * a.n;
  const float2* stats = a.stats + static_cast<long long>(b) * lists;
  const unsigned long long* offers = a.offers + static_cast<long long>(b) * count;
  const bool staged = count <= kStage;
  if (staged)
    for (int i = tid; i < count; i += kThreads) sh.stage[i] = __ldcg(offers + i);
  // lse[k]: a warp to a beam; NaN where the beam offers nothing
  for (int k = warp; k < a.K; k += kWarps) {
    float m = -INFINITY;
    bool nan = false;
    for (int c = lane; c < a.chunks; c += 32) {
      const float x = __ldcg(&stats[k * a.chunks + c].x);
      nan = nan || x != x;
      m = fmaxf(m, x);
    }
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, off));
    nan = __any_sync(0xFFFFFFFFu, nan) || m == INFINITY;
    double sum = 0.0;
    if (!nan && m > -INFINITY)
      for (int c = lane; c < a.chunks; c += 32) {
        const float2 x = __ldcg(stats + k * a.chunks + c);
        if (x.x > -INFINITY) sum += static_cast<double>(x.y) * exp(static_cast<double>(x.x) - static_cast<double>(m));
      }
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, off);
    if (lane == 0) {
      const float s = a.scores[static_cast<long long>(b) * a.K + k], w = a.weights ? a.weights[static_cast<long long>(b) * a.K + k] : 1.0f;
      const bool done = a.done && a.done[static_cast<long long>(b) * a.K + k] != 0;
      const bool odd = !(s < INFINITY) || !(w > 0.0f && w < INFINITY) || (nan && !done);
      if (odd) atomicOr(a.err, kErrInvalid);
      const bool none = odd || s == -INFINITY || (!done && !(m > -INFINITY));
      sh.lse[k] = none ? NAN : done ? 0.0 : static_cast<double>(m) + log(sum);
    }
  }
  __syncthreads();

  // ---- a thread to a list
  const int k = tid / a.chunks, chunk = tid - k * a.chunks;
  int at = 0;                                    // of the list's next offer
  unsigned long long key = 0, offer = 0;
  double S = 0.0, score = 0.0, lse = 0.0, weight = 1.0;
  bool done = false;
  if (tid < lists) {
    lse = sh.lse[k];
    score = a.scores[static_cast<long long>(b) * a.K + k];
    if (a.weights) weight = a.weights[static_cast<long long>(b) * a.K + k];
    done = a.done && a.done[static_cast<long long>(b) * a.K + k] != 0;
    if (lse != lse || (done && chunk != 0)) at = a.n;
  } else {
    at = a.n;
  }
  auto look = [&]() {
    key = 0;
    if (at >= a.n) return;
    if (done) {
      S = score;
    } else {
      offer = staged ? sh.stage[tid * a.n + at] : __ldcg(offers + static_cast<long long>(tid) * a.n + at);
      if (offer == 0) return;
      S = score + (static_cast<double>(value_of(static_cast<uint32_t>(offer >> 32))) - lse);
    }
    key = ordered64(S * weight);
  };
  look();
  const int warps = (lists + 31) / 32;
  for (int i = 0; i < a.n; ++i) {
    Best best = warp_best(key, tid);
    if (warps > 1) {
      if (lane == 0) {
        sh.best[i & 1][warp] = best.key;
        sh.best_at[i & 1][warp] = best.at;
      }
      __syncthreads();
      best = lane < warps ? Best{sh.best[i & 1][lane], sh.best_at[i & 1][lane]} : Best{0, 0x7FFFFFFF};
      best = warp_best(best.key, best.at);
    }
    const long long out = static_cast<long long>(b) * a.n + i;
    if (best.key == 0) {
      if (tid == 0) {
        a.parent[out] = -1;
        a.tok[out] = -1;
        a.score[out] = -INFINITY;
      }
    } else if (best.at == tid) {
      a.parent[out] = b * a.K + k;
      a.tok[out] = done ? a.end_tok : static_cast<int>(~static_cast<uint32_t>(offer));
      a.score[out] = static_cast<float>(S);
      at = done ? a.n : at + 1;
      look();
    }
  }
}

__global__ void __launch_bounds__(kThreads, 2) beam_kernel(const BeamArgs a) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  BeamShared& sh = *reinterpret_cast<BeamShared*>(smem_raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int row = blockIdx.x / a.chunks, chunk = blockIdx.x - row * a.chunks, b = row / a.K;
  // the chunk's logits, and the aligned 16-byte vectors that hold them
  const long long row0 = static_cast<long long>(row) * a.V;
  const long long e0 = row0 + static_cast<long long>(chunk) * a.chunk_len, e1 = min(e0 + a.chunk_len, row0 + a.V);
  // (from here on all places count from the first of these vectors; a row has at most 2^24 logits)
  const uint16_t* const from = a.logits + (e0 & ~7ll);
  const int lo = static_cast<int>(e0 & 7), hi = lo + static_cast<int>(e1 - e0), vecs = (hi + 7) >> 3;
  const int there = static_cast<int>(min(a.total - (e0 & ~7ll), 1ll << 26));   // logits of the whole tensor
  const uint32_t first_token = static_cast<uint32_t>((e0 & ~7ll) - row0);      // (wraps below a row's first)
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // a beam that has ended, or that has no score, offers nothing of its logits: they are not read
  const bool idle = (a.done && a.done[row] != 0) || a.scores[row] == -INFINITY;
  bool bad = false;                        // a NaN or +inf among the logits
  float all_m = -INFINITY, all_s = 0.0f;   // (thread 0)
  int have = 0;                            // of the best so far, in top
  for (int t0 = idle ? vecs : 0; t0 < vecs; t0 += kTileVecs) {
    uint4 x[kVecs];
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      const int v = t0 + i * kThreads + tid;
      x[i] = make_uint4(kLowest, kLowest, kLowest, kLowest);
      if (v < vecs) {
        if (8 * v + 8 <= there) {
          x[i] = ld_stream_v4(from + 8 * v);
        } else {  // the tensor's last logits
          uint32_t* w = reinterpret_cast<uint32_t*>(&x[i]);
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (8 * v + e < there)
              w[e >> 1] = e & 1 ? (w[e >> 1] & 0xFFFFu) | static_cast<uint32_t>(from[8 * v + e]) << 16
                                : (w[e >> 1] & 0xFFFF0000u) | from[8 * v + e];
        }
      }
    }
    // what belongs to other rows or chunks
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      const int v = t0 + i * kThreads + tid;
      if (v < vecs && (8 * v < lo || 8 * v + 8 > hi)) {
        uint32_t* w = reinterpret_cast<uint32_t*>(&x[i]);
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (8 * v + e < lo || 8 * v + e >= hi)
            w[e >> 1] = e & 1 ? (w[e >> 1] & 0xFFFFu) | (kLowest & 0xFFFF0000u) : (w[e >> 1] & 0xFFFF0000u) | (kLowest & 0xFFFFu);
      }
    }
    uint32_t pair = kLowest;
#pragma unroll
    for (int i = 0; i < kVecs; ++i) pair = max2(pair, max2(max2(x[i].x, x[i].y), max2(x[i].z, x[i].w)));
    const uint32_t mine = max(ordered(pair & 0xFFFFu), ordered(pair >> 16));
    const float m = fmaxf(bf16_lo(pair), bf16_hi(pair));
    const bool odd = mine >= kKeyInf;      // +inf or a NaN (max.NaN's is positive)
    // ---- the sum of exponentials, by a tree: errors of few roundings
    float part[kVecs];
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
      float p[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) p[e] = pow2((bf16_lo(w[e]) - m) * kLog2e) + pow2((bf16_hi(w[e]) - m) * kLog2e);
      part[i] = (p[0] + p[1]) + (p[2] + p[3]);
    }
#pragma unroll
    for (int h = kVecs / 2; h >= 1; h >>= 1)
#pragma unroll
      for (int i = 0; i < h; ++i) part[i] += part[i + h];
    float s = part[0], top = m;
    if (!(m > -INFINITY)) s = 0.0f;        // (nothing, or a NaN, which `odd` says)
    {
      float wm = m > -INFINITY ? m : -INFINITY;
#pragma unroll
      for (int off = 16; off >= 1; off >>= 1) wm = fmaxf(wm, __shfl_xor_sync(0xFFFFFFFFu, wm, off));
      s = m > -INFINITY ? s * pow2((m - wm) * kLog2e) : 0.0f;
#pragma unroll
      for (int off = 16; off >= 1; off >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, off);
      top = wm;
    }
    // ---- groups of threads, at least n of them: the n-th largest of their maxima bounds the n-th largest logit from below
    const int size = a.n <= 16 ? 32 : a.n <= 32 ? 16 : 8, groups = kThreads / size;
    uint32_t g = mine;
    for (int off = size / 2; off >= 1; off >>= 1) g = max(g, __shfl_xor_sync(0xFFFFFFFFu, g, off));
    if (lane % size == 0) sh.group[tid / size] = g;
    if (lane == 0) sh.warp_stat[warp] = make_float2(top, s);
    if (tid == 0) sh.n_list = have;
    if (tid < have) sh.list[tid] = sh.top[tid];
    bad = __syncthreads_or(odd);
    if (bad) break;
    if (warp == 0) {
      const float2 w = lane < kWarps ? sh.warp_stat[lane] : make_float2(-INFINITY, 0.0f);
      float wm = w.x;
#pragma unroll
      for (int off = 16; off >= 1; off >>= 1) wm = fmaxf(wm, __shfl_xor_sync(0xFFFFFFFFu, wm, off));
      const float both = fmaxf(wm, all_m);
      float ws = w.x > -INFINITY ? w.y * pow2((w.x - both) * kLog2e) : 0.0f;
#pragma unroll
      for (int off = 16; off >= 1; off >>= 1) ws += __shfl_xor_sync(0xFFFFFFFFu, ws, off);
      all_s = (all_m > -INFINITY ? all_s * pow2((all_m - both) * kLog2e) : 0.0f) + ws;
      all_m = both;
    }
    uint32_t bound = 0;
    for (int i = lane; i < groups; i += 32) {
      const uint32_t v = sh.group[i];
      int before = 0;
      for (int j = 0; j < groups; ++j) before += sh.group[j] > v || (sh.group[j] == v && j < i);
      if (before == a.n - 1) bound = v;
    }
    bound = __reduce_max_sync(0xFFFFFFFFu, bound);
    if (have == a.n) bound = max(bound, static_cast<uint32_t>(sh.top[a.n - 1] >> 32));
    bound = max(bound, kKeyLowest + 1);
    auto token = [&](int i, int e) { return first_token + 8 * (t0 + i * kThreads + tid) + e; };
    auto key_of = [&](int i, int e) {
      const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
      return ordered(e & 1 ? w[e >> 1] >> 16 : w[e >> 1] & 0xFFFFu);
    };
    auto push = [&](uint32_t key, uint32_t t) {
      const int at = atomicAdd(&sh.n_list, 1);
      if (at < kList) sh.list[at] = static_cast<unsigned long long>(key) << 32 | (0xFFFFFFFFu - t);
    };
    if (mine >= bound) {
#pragma unroll
      for (int i = 0; i < kVecs; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const uint32_t key = key_of(i, e);
          if (key >= bound) push(key, token(i, e));
        }
    }
    __syncthreads();
    int n = sh.n_list;
    if (n > kList) {
      // ---- too many equal (or so) logits: the exact n-th largest (logit, lowest token) of the tile, bit by bit
      uint32_t exact = 0;
      for (int bit = 31; bit >= 0; --bit) {
        const uint32_t cand = exact | 1u << bit;
        int c = 0;
        if (mine >= cand >> 16) {
#pragma unroll
          for (int i = 0; i < kVecs; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e)
              c += (key_of(i, e) << 16 | (0xFFFFu - static_cast<uint32_t>((i * kThreads + tid) * 8 + e))) >= cand;
        }
        c = __reduce_add_sync(0xFFFFFFFFu, c);
        if (tid < 2) sh.counts[tid] = 0;
        __syncthreads();
        if (lane == 0 && c) atomicAdd(&sh.counts[0], c);
        __syncthreads();
        if (sh.counts[0] >= static_cast<unsigned int>(a.n)) exact = cand;
        __syncthreads();
      }
      if (tid == 0) sh.n_list = have;
      __syncthreads();
      if (mine >= exact >> 16) {
#pragma unroll
        for (int i = 0; i < kVecs; ++i)
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const uint32_t key = key_of(i, e);
            if (key > kKeyLowest && (key << 16 | (0xFFFFu - static_cast<uint32_t>((i * kThreads + tid) * 8 + e))) >= exact)
              push(key, token(i, e));
          }
      }
      __syncthreads();
      n = sh.n_list;
    }
    // ---- in order: a key's place is the number of larger ones
    for (int i = tid; i < n; i += kThreads) {
      const unsigned long long key = sh.list[i];
      int place = 0;
      for (int j = 0; j < n; ++j) place += sh.list[j] > key;
      if (place < a.n) sh.top[place] = key;
    }
    have = min(n, a.n);
    __syncthreads();
  }
  const long long list = static_cast<long long>(row) * a.chunks + chunk;
  if (tid < a.n) a.offers[list * a.n + tid] = tid < have && !bad ? sh.top[tid] : 0ull;
  if (tid == 0) a.stats[list] = bad ? make_float2(NAN, 0.0f) : make_float2(all_m, all_s);
  __syncthreads();
  if (tid == 0) {
    __threadfence();
    const bool last = atomicAdd(a.tickets + b, 1u) == static_cast<unsigned int>(a.K * a.chunks - 1);
    if (last) a.tickets[b] = 0;
    __threadfence();
    sh.last = last;
  }
  __syncthreads();
  if (sh.last) merge(a, sh, b);
}

struct BeamPlan {
  int chunks, chunk_len;
  size_t stats, offers, total;
};

// Chunks of a row: as many as keep two CTAs on every SM busy, of 4096 logits at least, and no larger than a tile; at most a
// list a thread in the merge (a larger vocabulary takes a chunk in several tiles).
bool beam_plan(int64_t B, int64_t K, int64_t V, int64_t n, BeamPlan& p) {
  if (B < 1 || K < 1 || K > kMaxBeams || V < 2 || V > QSPEC_MAX_V || n < 1 || n > kMaxN || n > K * V || B > 65535 ||
      B * K * V >= (int64_t(1) << 40))
    return false;
  int64_t c = 2 * num_sms() / (B * K);
  const int64_t most = (V + 4095) / 4096, least = (V + kTile - 9) / (kTile - 8);
  if (c > most) c = most;
  if (c < least) c = least;
  if (c > kMaxLists / K) c = kMaxLists / K;
  p.chunk_len = static_cast<int>((V + c - 1) / c);
  p.chunks = static_cast<int>((V + p.chunk_len - 1) / p.chunk_len);
  const size_t lists = static_cast<size_t>(B) * K * p.chunks;
  p.stats = (sizeof(unsigned int) * B + 255) & ~size_t(255);
  p.offers = (p.stats + sizeof(float2) * lists + 255) & ~size_t(255);
  p.total = p.offers + sizeof(unsigned long long) * lists * n;
  return true;
}

}  // namespace
}  // namespace qspec

using namespace qspec;

extern "C" size_t qspec_beam_workspace_size(int32_t B, int32_t beams, int32_t V, int32_t n) {
  BeamPlan p;
  return beam_plan(B, beams, V, n, p) ? p.total : 0;
}

extern "C" qspec_status qspec_beam_select(const uint16_t* logits, const float* scores, const int32_t* done, int32_t end_tok,
                                          const float* weights, int32_t B, int32_t beams, int32_t V, int32_t n, int32_t* parent,
                                          int32_t* tok, float* score, void* ws, size_t ws_bytes, qspec_stream_t stream) {
  if (!logits || !scores || !parent || !tok || !score || B <= 0 || beams <= 0 || V <= 0 || n <= 0) return QSPEC_ERR_INVALID_ARG;
  BeamPlan p;
  if (!beam_plan(B, beams, V, n, p)) return QSPEC_ERR_UNSUPPORTED_SHAPE;
  const int64_t blocks = static_cast<int64_t>(B) * beams * p.chunks;
  if (blocks > 0x7FFFFFFF) return QSPEC_ERR_UNSUPPORTED_SHAPE;
  if (!aligned16(logits) || !aligned4(scores) || !aligned4(done) || !aligned4(weights) || !aligned4(parent) || !aligned4(tok) ||
      !aligned4(score) || !aligned16(ws))
    return QSPEC_ERR_MISALIGNED;
  if (!ws || ws_bytes < p.total) return QSPEC_ERR_WORKSPACE;
  char* w = static_cast<char*>(ws);
  BeamArgs a{logits, scores, done, weights, parent, tok, score, linear_error_word(), reinterpret_cast<unsigned int*>(w),
             reinterpret_cast<float2*>(w + p.stats), reinterpret_cast<unsigned long long*>(w + p.offers),
             static_cast<long long>(B) * beams * V, B, beams, V, n, p.chunks, p.chunk_len, end_tok};
  if (!a.err) return QSPEC_ERR_CUDA;
  static_assert(sizeof(BeamShared) <= 48 * 1024, "no opt-in needed");
  return launch_pdl(beam_kernel, dim3(static_cast<unsigned int>(blocks)), dim3(kThreads), sizeof(BeamShared),
                    reinterpret_cast<cudaStream_t>(stream), a);
}
