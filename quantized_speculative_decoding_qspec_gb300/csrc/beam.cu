// Beam selection: the n best of a sequence's beams times vocabulary by summed log probability.
//
//     S(k, v) = score[k] + (logit[k, v] - lse[k]),   lse[k] = ln sum_v exp(logit[k, v])
// Within a beam the order is that of its logits (bf16: ties are common, and go to the lowest token), so each beam offers its n
// largest logits, and the beams' offers are ordered by S (times a weight).  One pass over the logits bounds it: a CTA
// streams a part of a row through registers, a tile of 8192 at a time, two tiles under way.  A thread keeps its own maximum and sum of
// exponentials; the maxima give a lower bound of the n-th largest logit, from the first tile on and better with every look, and the few
// vectors that reach it are collected in shared memory.  The last CTA of a sequence (atomic ticket) merges the offers.
// [64, 8, 152064]: 40 us for 156 MB, 3.9 TB/s (39 us with one beam in seven finished: 133 MB, 3.4 TB/s); [16, 4, 128256] 14,
// [1, 4, 32000] 7.9.  512 blocks of 256 threads are resident at once, three or four
// to an SM, and wait at their barriers in turn (two of 512 threads: 47 us; eight of 128: 57; a tile of 32768 to a CTA, selected and
// handed over before the next CTA began: 102).  The smaller ones are a chain of latencies: the first tile 2 us, its bound 0.5, the list 1.5,
// the ticket 1, the merge 4.
#include <math.h>

#include "kv_internal.h"

namespace qspec {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kVecs = 4;                          // 16-byte loads in flight a thread
constexpr int kTileVecs = kThreads * kVecs;       // 8192 logits
constexpr int kList = 1024;                       // logits collected at most; tiles that bring more: see below
constexpr int kListFull = 512;                    // from here on they are cut down to the n best
constexpr int kVecList = 512;                     // vectors collected between looks at them
constexpr int kCheck = 4;                         // tiles between looks
constexpr int kCtasPerSm = 4;                     // resident
constexpr int kMaxN = QSPEC_BEAM_MAX_N, kMaxBeams = QSPEC_BEAM_MAX_BEAMS;
constexpr int kMaxLists = kThreads;               // (beam, chunk) pairs of a sequence: a thread each in the merge
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
  unsigned int* tickets;        // [65536]
  float2* stats;                // [B, K, chunks]: maximum, sum of exponentials
  unsigned long long* offers;   // [B, K, chunks, n]: ordered logit << 32 | ~token; 0: none
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
// Pairs of fp32 numbers: 2^((x + a) s), and sums: half the instructions of the sum of exponentials ([64, 8, 152064] 65 -> 61 us).
__device__ __forceinline__ uint64_t pair_of(float x, float y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ uint64_t add_pair(uint64_t x, uint64_t y) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
  return r;
}
__device__ __forceinline__ uint64_t pow2_pair(uint64_t x, uint64_t a, uint64_t s) {
  float lo, hi;
  asm("{\n\t.reg .b64 v;\n\tadd.rn.f32x2 v, %2, %3;\n\tmul.rn.f32x2 v, v, %4;\n\tmov.b64 {%0, %1}, v;\n\t}"
      : "=f"(lo), "=f"(hi)
      : "l"(x), "l"(a), "l"(s));
  return pair_of(pow2(lo), pow2(hi));
}

// An order-preserving map of doubles (no NaN) to integers, 0 below all of them.
__device__ __forceinline__ unsigned long long ordered64(double x) {
  const long long b = __double_as_longlong(x == 0.0 ? 0.0 : x);
  return static_cast<unsigned long long>(b < 0 ? ~b : b | (1ll << 63));
}

struct BeamShared {
  union {
    unsigned long long list[kList + kMaxN];
    struct {
      unsigned long long head[kMaxLists];
      uint32_t head_order[kMaxLists];
    };
  };
  unsigned long long pair_key[kMaxN * (kMaxN + 1) / 2];
  uint32_t pair_order[kMaxN * (kMaxN + 1) / 2];
  int best_list[kMaxN];
  unsigned long long top[kMaxN];
  uint32_t group[64];
  float2 warp_stat[kWarps];
  int count;
  double lse[kMaxBeams];
  float row_score[kMaxBeams], row_weight[kMaxBeams];
  bool row_done[kMaxBeams];
  float2 row_stat[kMaxBeams];
  uint32_t bound;
  uint4 vec[kVecList];
  uint32_t token[kVecList];  // of a vector's first logit
  int n_vec, n_list, last;
};

struct Candidate {
  unsigned long long key;  // of S times the weight
  uint32_t order;          // among equal keys, lowest first: by beam, logit (largest first), place in the row
  double S;
  int row, tok;
};

// ln s for 1 <= s: the power of two apart, so that the error is that of logf near 1, 2^-24.  (fp64 runs at a fiftieth of fp32's rate:
// its logarithm took 1 us of the merge.)
__device__ __forceinline__ double ln_of_sum(float s) {
  int e = static_cast<int>(__float_as_uint(s) >> 23) - 127;
  float m = __uint_as_float((__float_as_uint(s) & 0x7FFFFFu) | 0x3F800000u);
  if (m > 1.41421356f) {
    m *= 0.5f;
    ++e;
  }
  return e * 0.69314718055994531 + static_cast<double>(logf(m));
}

// The last CTA of sequence b: the beams' sums, then the n best of what the lists offer.
__device__ __noinline__ void merge(const BeamArgs& a, BeamShared& sh, int b) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int lists = a.K * a.chunks, n = a.n;
  const float2* stats = a.stats + static_cast<long long>(b) * lists;
  const unsigned long long* offers = a.offers + static_cast<long long>(b) * lists * n;
  // (what comes from memory is asked for at once: each round of it takes 0.6 us)
  const unsigned long long first = tid < lists ? __ldcg(offers + static_cast<long long>(tid) * n) : 0;
  float score = 0.0f, weight = 1.0f;
  bool done = false;
  if (tid < a.K) {
    const long long at = static_cast<long long>(b) * a.K + tid;
    score = a.scores[at];
    if (a.weights) weight = a.weights[at];
    done = a.done && a.done[at] != 0;
  }
  // the beams' maxima and sums, a warp to a beam; NaN where the beam offers nothing
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
    float sum = 0.0f;
    if (!nan && m > -INFINITY)
      for (int c = lane; c < a.chunks; c += 32) {
        const float2 x = __ldcg(stats + k * a.chunks + c);
        if (x.x > -INFINITY) sum += x.y * pow2((x.x - m) * kLog2e);
      }
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, off);
    if (lane == 0) sh.row_stat[k] = nan ? make_float2(NAN, 0.0f) : make_float2(m, sum);
  }
  __syncthreads();
  if (tid < a.K) {
    const float2 x = sh.row_stat[tid];
    const bool odd = !(score < INFINITY) || !(weight > 0.0f && weight < INFINITY) || (x.x != x.x && !done);
    if (odd) atomicOr(a.err, kErrInvalid);
    const bool none = odd || score == -INFINITY || (!done && !(x.x > -INFINITY));
    sh.lse[tid] = none ? NAN : done ? 0.0 : static_cast<double>(x.x) + ln_of_sum(x.y);
    sh.row_score[tid] = score;
    sh.row_weight[tid] = weight;
    sh.row_done[tid] = done;
  }
  __syncthreads();

  // ---- the best n lists by their first offers, in order: the r-th can give n - r of the n best.  (Choosing the n best one after
  // the other by reductions over the lists took 5 to 7 us for eight.)
  // S is fp64, so different logits of a beam can have equal ones (far scores; logits much nearer than the logarithm's size): a chunk's
  // offers are in their order, those of different chunks are put in it by the logit.
  const int at_bits = 6 + (32 - __clz(a.chunks - 1));
  static_assert(kMaxN <= 1 << 6 && kMaxLists <= 1 << 8 && kMaxBeams <= 1 << 5, "beam and chunk have 9 bits, logit and place 22");
  auto candidate = [&](int list, int e, unsigned long long offer, Candidate& c) {  // false: no offer
    const int k = list / a.chunks;
    c.order = static_cast<uint32_t>(k) << (at_bits + 16) | (0xFFFFu - static_cast<uint32_t>(offer >> 32)) << at_bits |
              static_cast<uint32_t>(list - k * a.chunks) << 6 | e;
    const double lse = sh.lse[k];
    if (lse != lse) return false;
    c.S = sh.row_score[k];
    c.tok = a.end_tok;
    c.row = b * a.K + k;
    if (sh.row_done[k]) {
      if (e > 0 || list != k * a.chunks) return false;
    } else {
      if (offer == 0) return false;
      c.tok = static_cast<int>(~static_cast<uint32_t>(offer));
      c.S += static_cast<double>(value_of(static_cast<uint32_t>(offer >> 32))) - lse;
    }
    c.key = ordered64(a.weights ? c.S * sh.row_weight[k] : c.S);
    return true;
  };
  Candidate c{};
  const unsigned long long head = tid < lists && candidate(tid, 0, first, c) ? c.key : 0;
  const uint32_t head_order = c.order;
  sh.head[tid] = head;
  sh.head_order[tid] = head_order;
  if (tid < n) sh.best_list[tid] = -1;
  if (tid == 0) sh.count = 0;
  __syncthreads();
  if (head != 0) {
    int place = 0;
#pragma unroll 4
    for (int j = 0; j < lists; ++j) {
      const unsigned long long x = sh.head[j];
      const uint32_t o = sh.head_order[j];
      place += (x > head) | ((x == head) & (o < head_order));
    }
    if (place < n) sh.best_list[place] = tid;
  }
  __syncthreads();
  const int pairs = n * (n + 1) / 2;
  auto pair = [&](int p, int& list, int& e) {
    int r = 0;
    for (e = p; e >= n - r;) e -= n - r++;
    list = sh.best_list[r];
    return list >= 0 && candidate(list, e, __ldcg(offers + static_cast<long long>(list) * n + e), c);
  };
  Candidate mine;
  for (int p = tid; p < pairs; p += kThreads) {
    int list, e;
    const bool real = pair(p, list, e);
    if (p == tid) mine = c;
    sh.pair_key[p] = real ? c.key : 0;
    sh.pair_order[p] = c.order;
    if (real) atomicAdd(&sh.count, 1);
  }
  __syncthreads();
  for (int p = tid; p < pairs; p += kThreads) {
    const unsigned long long key = sh.pair_key[p];
    const uint32_t order = sh.pair_order[p];
    if (key == 0) continue;
    int place = 0;
#pragma unroll 4
    for (int j = 0; j < pairs; ++j) {  // (both reads of a step at once: with the second behind a branch a step took 120 cycles)
      const unsigned long long x = sh.pair_key[j];
      const uint32_t o = sh.pair_order[j];
      place += (x > key) | ((x == key) & (o < order));
    }
    if (place >= n) continue;
    c = mine;
    int list, e;
    if (p != tid) pair(p, list, e);
    const long long out = static_cast<long long>(b) * n + place;
    a.parent[out] = c.row;
    a.tok[out] = c.tok;
    a.score[out] = static_cast<float>(c.S);
  }
  if (tid < n && tid >= sh.count) {
    const long long out = static_cast<long long>(b) * n + tid;
    a.parent[out] = -1;
    a.tok[out] = -1;
    a.score[out] = -INFINITY;
  }
}

// A chunk of a row in aligned 16-byte vectors; all places count from the first of them (a row has at most 2^24 logits).
struct Chunk {
  const uint16_t* from;
  int lo, hi, vecs;      // the chunk's logits are lo .. hi - 1
  uint32_t first_token;  // of place 0 (wraps below a row's first)
};

// The thread's vectors of the tile at t0; -inf outside the chunk.  (Tiles that lie wholly in it apart: [64, 8, 152064] 48.7 -> 46.8 us, with 512 threads.)
__device__ __forceinline__ void load_tile(const Chunk& c, int t0, uint4 (&x)[kVecs]) {
  if (8 * t0 >= c.lo && 8 * (t0 + kTileVecs) <= c.hi) {
    const uint4* at = reinterpret_cast<const uint4*>(c.from) + t0 + threadIdx.x;
#pragma unroll
    for (int i = 0; i < kVecs; ++i) x[i] = ld_stream_v4(at + i * kThreads);
    return;
  }
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const int v = t0 + i * kThreads + threadIdx.x;
    x[i] = make_uint4(kLowest, kLowest, kLowest, kLowest);
    if (v >= c.vecs) continue;
    if (8 * v >= c.lo && 8 * v + 8 <= c.hi) {
      x[i] = ld_stream_v4(c.from + 8 * v);
    } else {  // the chunk's first or last vector: what is its own
      uint32_t* w = reinterpret_cast<uint32_t*>(&x[i]);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (8 * v + e >= c.lo && 8 * v + e < c.hi)
          w[e >> 1] = e & 1 ? (w[e >> 1] & 0xFFFFu) | static_cast<uint32_t>(c.from[8 * v + e]) << 16
                            : (w[e >> 1] & 0xFFFF0000u) | c.from[8 * v + e];
    }
  }
}
__device__ __forceinline__ uint32_t key_of(const uint4 (&x)[kVecs], int i, int e) {
  const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
  return ordered(e & 1 ? w[e >> 1] >> 16 : w[e >> 1] & 0xFFFFu);
}
// Collects a logit.
__device__ __forceinline__ void collect(BeamShared& sh, uint32_t key, uint32_t token) {
  const int at = atomicAdd(&sh.n_list, 1);
  if (at < kList + kMaxN) sh.list[at] = static_cast<unsigned long long>(key) << 32 | (0xFFFFFFFFu - token);
}

// The n best of the list's first `count` entries, in order, become the list (and top): a key's place is the number of larger
// ones.  All threads; ends with a barrier.
__device__ __noinline__ void cut_down(BeamShared& sh, int count, int n) {
  const int tid = threadIdx.x;
  if (tid < kMaxN) sh.top[tid] = 0;
  __syncthreads();
  for (int i = tid; i < count; i += kThreads) {
    const unsigned long long key = sh.list[i];
    int place = 0;
#pragma unroll 8
    for (int j = 0; j < count; ++j) place += sh.list[j] > key;
    if (place < n && key != 0) sh.top[place] = key;
  }
  __syncthreads();
  if (tid < n) sh.list[tid] = sh.top[tid];
  if (tid == 0) sh.n_list = n;
  __syncthreads();
}

// The tiles from t0 on, kCheck of them, brought far more logits than there are places, as with many equal ones: what of them is among
// the list's first `count` entries is taken out again, and their exact n-th largest (logit, lowest token) found bit by bit.  Returns
// the number of entries.
__device__ __noinline__ int exact_tiles(BeamShared& sh, const Chunk& c, int t0, int count, int n) {
  const int tid = threadIdx.x;
  const uint32_t tile0 = c.first_token + 8 * t0;
  for (int i = tid; i < kList; i += kThreads)
    if (i >= count || 0xFFFFFFFFu - static_cast<uint32_t>(sh.list[i]) - tile0 < 8u * kCheck * kTileVecs) sh.list[i] = 0;
  uint4 x[kVecs];
  auto rank_of = [&](int k, int i, int e) {
    return key_of(x, i, e) << 16 | (0xFFFFu - static_cast<uint32_t>((k * kTileVecs + i * kThreads + tid) * 8 + e));
  };
  static_assert(8 * kCheck * kTileVecs <= 0x10000, "a place in these tiles has 16 bits");
  uint32_t exact = 0;
  for (int bit = 31; bit >= 0; --bit) {
    const uint32_t cand = exact | 1u << bit;
    int above = 0;
#pragma unroll 1
    for (int k = 0; k < kCheck; ++k) {
      load_tile(c, t0 + k * kTileVecs, x);
#pragma unroll
      for (int i = 0; i < kVecs; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) above += rank_of(k, i, e) >= cand;
    }
    above = __reduce_add_sync(0xFFFFFFFFu, above);
    if (tid == 0) sh.count = 0;
    __syncthreads();
    if ((tid & 31) == 0 && above) atomicAdd(&sh.count, above);
    __syncthreads();
    if (sh.count >= n) exact = cand;
    __syncthreads();
  }
  if (tid == 0) sh.n_list = kList;
  __syncthreads();
#pragma unroll 1
  for (int k = 0; k < kCheck; ++k) {
    load_tile(c, t0 + k * kTileVecs, x);
#pragma unroll
    for (int i = 0; i < kVecs; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t key = key_of(x, i, e);
        if (key > kKeyLowest && rank_of(k, i, e) >= exact) collect(sh, key, tile0 + 8 * (k * kTileVecs + i * kThreads + tid) + e);
      }
  }
  __syncthreads();
  return sh.n_list;
}

// What a thread carries from tile to tile.
struct Running {
  float m, s;      // its maximum and sum of exponentials
  uint32_t bound;  // of the n-th largest logit, from below
  bool bad;        // a NaN or +inf among its logits
};

// The n-th largest of 64 groups of threads' maxima: a bound of the n-th largest logit that they have seen.  A warp finds the places of
// eight, with four lanes to each (all of them in every warp: 1.5 us, the warps' issue slots).  All threads; two barriers,
// and the list of vectors, which all have read, is empty.
__device__ __forceinline__ uint32_t bound_of(BeamShared& sh, uint32_t mine, int n) {
  const int tid = threadIdx.x;
  constexpr int kSize = kThreads / kMaxN;
#pragma unroll
  for (int off = kSize / 2; off >= 1; off >>= 1) mine = max(mine, __shfl_xor_sync(0xFFFFFFFFu, mine, off));
  if (tid % kSize == 0) sh.group[tid / kSize] = mine << 6 | (kMaxN - 1 - tid / kSize);  // (no two alike)
  __syncthreads();
  constexpr int kLanes = kThreads / kMaxN, kEach = kMaxN / kLanes;
  static_assert(kMaxN == 64 && kLanes >= 1 && kLanes <= 32, "six bits; a group's lanes in one warp");
  const uint32_t v = sh.group[tid / kLanes];
  int before = 0;
#pragma unroll
  for (int j = 0; j < kEach; ++j) before += sh.group[j * kLanes + tid % kLanes] > v;
#pragma unroll
  for (int off = kLanes / 2; off >= 1; off >>= 1) before += __shfl_xor_sync(0xFFFFFFFFu, before, off);
  if (before == n - 1) sh.bound = v >> 6;
  if (tid == 0) sh.n_vec = 0;
  __syncthreads();
  return sh.bound;
}

__device__ __forceinline__ void take_tile(BeamShared& sh, const Chunk& c, int n, int t0, uint4 (&x)[kVecs], Running& r) {
  const int tid = threadIdx.x;
  uint32_t pair = kLowest, most[kVecs];  // largest values, of even and odd places
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    most[i] = max2(max2(x[i].x, x[i].y), max2(x[i].z, x[i].w));
    pair = max2(pair, most[i]);
  }
  auto top_of = [](uint32_t p) { return max(ordered(p & 0xFFFFu), ordered(p >> 16)); };
  const uint32_t mine = top_of(pair);
  r.bad = r.bad || mine >= kKeyInf;  // +inf or a NaN (max.NaN's is positive)
  // ---- the sum of exponentials, by a tree in the tile: errors of few roundings
  const float top = fmaxf(r.m, fmaxf(bf16_lo(pair), bf16_hi(pair)));
  if (top > -INFINITY) {
    const uint64_t away = pair_of(-top, -top), scale = pair_of(kLog2e, kLog2e);
    uint64_t part[kVecs];
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
      uint64_t p[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) p[e] = pow2_pair(pair_of(bf16_lo(w[e]), bf16_hi(w[e])), away, scale);
      part[i] = add_pair(add_pair(p[0], p[1]), add_pair(p[2], p[3]));
    }
#pragma unroll
    for (int h = kVecs / 2; h >= 1; h >>= 1)
#pragma unroll
      for (int i = 0; i < h; ++i) part[i] = add_pair(part[i], part[i + h]);
    float even, odd;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(even), "=f"(odd) : "l"(part[0]));
    r.s = (r.m > -INFINITY ? r.s * pow2((r.m - top) * kLog2e) : 0.0f) + (even + odd);
    r.m = top;
  }
  if (t0 == 0) r.bound = max(bound_of(sh, mine, n), kKeyLowest + 1);
  // ---- vectors with a logit that reaches the bound, as they are.  (Their logits taken out here, by a lane or by eight of them, kept some warps
  // for 500 cycles each while the others waited at the next barrier: [64, 8, 152064] 60 us, without any collecting 46.)
  if (__any_sync(0xFFFFFFFFu, mine >= r.bound)) {
#pragma unroll
    for (int i = 0; i < kVecs; ++i)
      if (top_of(most[i]) >= r.bound) {
        const int at = atomicAdd(&sh.n_vec, 1);
        if (at < kVecList) {
          sh.vec[at] = x[i];
          sh.token[at] = c.first_token + 8 * (t0 + i * kThreads + tid);
        }
      }
  }
  load_tile(c, t0 + 2 * kTileVecs, x);
}

// After the kCheck tiles from t0 on (or those that were left): the collected vectors' logits go to the list, which keeps its n best
// where it is filling up, and the bound rises to what all tiles so far allow.
__device__ __forceinline__ void take_stock(BeamShared& sh, const Chunk& c, int n, int t0, Running& r) {
  const int tid = threadIdx.x;
  __syncthreads();
  const int vecs = sh.n_vec;
  if (vecs <= kVecList) {
    const uint16_t* x = reinterpret_cast<const uint16_t*>(sh.vec);
    for (int i = tid; i < 8 * vecs; i += kThreads) {
      const uint32_t key = ordered(x[i]);
      if (key >= r.bound) collect(sh, key, sh.token[i >> 3] + (i & 7));
    }
  }
  r.bound = max(r.bound, bound_of(sh, ordered(__float_as_uint(r.m) >> 16), n));  // (barriers inside)
  int count = sh.n_list;
  if (vecs > kVecList || count > kListFull) {
    __syncthreads();
    if (vecs > kVecList || count > kList) count = exact_tiles(sh, c, t0, min(count, kList), n);
    cut_down(sh, count, n);
    r.bound = max(r.bound, static_cast<uint32_t>(sh.top[n - 1] >> 32));
  }
}

__global__ void __launch_bounds__(kThreads, kCtasPerSm) beam_kernel(const BeamArgs a) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  BeamShared& sh = *reinterpret_cast<BeamShared*>(smem_raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int row = blockIdx.x / a.chunks, chunk = blockIdx.x - row * a.chunks, b = row / a.K;
  const long long row0 = static_cast<long long>(row) * a.V;
  const long long e0 = row0 + static_cast<long long>(chunk) * a.chunk_len, e1 = min(e0 + a.chunk_len, row0 + a.V);
  Chunk c{a.logits + (e0 & ~7ll), static_cast<int>(e0 & 7)};
  c.hi = c.lo + static_cast<int>(e1 - e0);
  c.vecs = (c.hi + 7) >> 3;
  c.first_token = static_cast<uint32_t>((e0 & ~7ll) - row0);
  if (tid == 0) sh.n_list = sh.n_vec = 0;
  __syncthreads();
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // a beam that has ended, or that has no score, offers nothing of its logits: they are not read
  if ((a.done && a.done[row] != 0) || a.scores[row] == -INFINITY) c.vecs = 0;

  Running r{-INFINITY, 0.0f, 0, false};
  if (c.vecs > 0) {  // two tiles under way
    uint4 x[kVecs], y[kVecs];
    load_tile(c, 0, x);
    load_tile(c, kTileVecs, y);
    static_assert(kCheck % 2 == 0, "tiles go in pairs");
#pragma unroll 1
    for (int t0 = 0; t0 < c.vecs; t0 += 2 * kTileVecs) {
      take_tile(sh, c, a.n, t0, x, r);
      if (t0 + kTileVecs < c.vecs) take_tile(sh, c, a.n, t0 + kTileVecs, y, r);
      if (t0 / kTileVecs % kCheck == kCheck - 2 || t0 + 2 * kTileVecs >= c.vecs)
        take_stock(sh, c, a.n, t0 / (kCheck * kTileVecs) * (kCheck * kTileVecs), r);
    }
  }
  // ---- the CTA's maximum and sum
  {
    float top = r.m;
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, off));
    float s = r.m > -INFINITY ? r.s * pow2((r.m - top) * kLog2e) : 0.0f;
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, off);
    if (lane == 0) sh.warp_stat[warp] = make_float2(top, s);
  }
  const bool bad = __syncthreads_or(r.bad);
  cut_down(sh, sh.n_list, a.n);
  const long long list = static_cast<long long>(row) * a.chunks + chunk;
  if (tid < a.n) a.offers[list * a.n + tid] = bad ? 0ull : sh.top[tid];
  if (warp == 0) {
    const float2 w = lane < kWarps ? sh.warp_stat[lane] : make_float2(-INFINITY, 0.0f);
    float top = w.x;
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, off));
    float sum = w.x > -INFINITY ? w.y * pow2((w.x - top) * kLog2e) : 0.0f;
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, off);
    if (lane == 0) a.stats[list] = bad ? make_float2(NAN, 0.0f) : make_float2(top, sum);
  }
  __syncthreads();  // (the release below covers what the barrier made this thread see)
  if (tid == 0) {
    unsigned int old;
    asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(old) : "l"(a.tickets + b) : "memory");
    sh.last = old == static_cast<unsigned int>(a.K * a.chunks - 1);
    if (sh.last) a.tickets[b] = 0;
  }
  __syncthreads();
  if (sh.last) merge(a, sh, b);
}

struct BeamPlan {
  int chunks, chunk_len;
  size_t stats, offers;  // where they lie
  size_t total;          // what this shape and every smaller one need
};

// Chunks of a row: two to an SM, of 4096 logits at least; at most a list a thread in the merge.  (More of them cost the merge
// and their own beginnings and ends: [16, 4, 128256] 14.0 us with four to a row, 15.2 with nine, 15.0 with two.  Four blocks fit an
// SM, so rows that just miss a second chunk leave places empty: 152 rows of 128256 logits take 16.8 us, 160 take 21.9, 304 23.6.)
bool beam_plan(int64_t B, int64_t K, int64_t V, int64_t n, BeamPlan& p) {
  if (B < 1 || K < 1 || K > kMaxBeams || V < 2 || V > QSPEC_MAX_V || n < 1 || n > kMaxN || n > K * V || B > 65535 ||
      B * K * V >= (int64_t(1) << 40))
    return false;
  const int64_t places = 2 * num_sms(), most = (V + 4095) / 4096;
  int64_t c = places / (B * K);
  if (c > most) c = most;
  if (c < 1) c = 1;
  if (c > kMaxLists / K) c = kMaxLists / K;
  p.chunk_len = static_cast<int>((V + c - 1) / c);
  p.chunks = static_cast<int>((V + p.chunk_len - 1) / p.chunk_len);
  p.stats = sizeof(unsigned int) * 65536;  // (tickets of the largest batch: they are where they were for calls of any shape)
  auto offers_at = [&](int64_t lists) { return (p.stats + sizeof(float2) * lists + 255) & ~size_t(255); };
  p.offers = offers_at(B * K * p.chunks);
  // Fewer rows have more chunks each, so a smaller batch can have more lists: never more than two to an SM, or one to a row, or one to
  // 4096 logits of these rows.
  int64_t lists = B * K * most < places ? B * K * most : places;
  if (lists < B * K) lists = B * K;
  p.total = offers_at(lists) + sizeof(unsigned long long) * lists * n;
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
  const int64_t rows = static_cast<int64_t>(B) * beams, best = static_cast<int64_t>(B) * n;
  const Words in[] = {{scores, rows}, {done, rows}, {weights, rows}}, out[] = {{parent, best}, {tok, best}, {score, best}};
  if (outputs_overlap(out, 3, in, 3)) return QSPEC_ERR_INVALID_ARG;  // (a sequence's last block writes while others' read)
  char* w = static_cast<char*>(ws);
  BeamArgs a{logits, scores, done, weights, parent, tok, score, linear_error_word(), reinterpret_cast<unsigned int*>(w),
             reinterpret_cast<float2*>(w + p.stats), reinterpret_cast<unsigned long long*>(w + p.offers),
             B, beams, V, n, p.chunks, p.chunk_len, end_tok};
  if (!a.err) return QSPEC_ERR_CUDA;
  static_assert(sizeof(BeamShared) <= 48 * 1024, "no opt-in needed");
  return launch_pdl(beam_kernel, dim3(static_cast<unsigned int>(blocks)), dim3(kThreads), sizeof(BeamShared),
                    reinterpret_cast<cudaStream_t>(stream), a);
}
