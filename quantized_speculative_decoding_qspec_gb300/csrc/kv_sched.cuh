// How the attention kernels share out their work, and what they have in common.
//
// An item is one (sequence, tile of query rows, key head): the rows of a sequence and key head are its new tokens
// times the G query heads that read that key head, packed as row = token * G + g.  An item's keys come
// in tiles of a kernel's kKeys positions; a unit is one such tile of one item.  All units of the call, in the order
// (sequence, row tile, head, key tile), are cut into equal runs, one per CTA, whatever the lengths of the
// sequences: every CTA reads the same number of cache bytes, and one launch serves ragged batches, single
// long sequences and anything a graph replay finds in kv_len.  Items that lie in one run are finished
// there; an item cut by run boundaries leaves its partial sums in the workspace, and the last of its CTAs to
// arrive (atomic ticket) adds them in run order, so results do not depend on timing.
#pragma once

#include "kv_internal.h"
#include "tc_ptx.cuh"

namespace qspec {
namespace att {

constexpr long long kWaitLimit = 4000000000LL;   // clock cycles (about 2 s) before a wait gives up
constexpr float kNoMax = -3.3e38f;               // reference of a row that has seen nothing
// P = 2^(z - m) is fp16 for the product with the values.  A row's reference m is set kLift below its largest score and
// stays until a score exceeds it by kSlack: P <= 2^15 fits, and a key keeps a share of the product down to 2^-33 of the
// largest weight.  (With m at the largest score it ended at 2^-25: behind one dominant key, a million others of 2^-25.5,
// 2% of the sum, were lost.  It costs some more moves of m: 4096 tokens over 8192 positions 375 -> 380 us.)
constexpr float kSlack = 15.0f, kLift = 8.0f;
// The reference for a largest score `top`.  Scores beyond kFar are so coarse that a sum with kLift could round to another
// 8 below: the reference is the score itself there.
constexpr float kFar = 4194304.0f;
__device__ __forceinline__ float reference_of(float top) { return fabsf(top) < kFar ? top - kLift : top; }

constexpr int kSmemPerSm = 228 * 1024, kSmemReserved = 1024;  // of sm_103: an SM's shared memory, and what a CTA takes unseen

struct CutItem {
  int parts, tok0, row0, rows, head;  // parts: runs with a part of it, or 0: none
  int pad[3];
};

struct AttArgs {
  qspec_kv_cache c;
  qspec_kv_batch b;
  const uint16_t* q;
  uint16_t* out;
  float* lse;
  const unsigned long long* tree;
  unsigned int* err;
  unsigned int* tickets;  // [3][grid]
  float* partial;         // [grid][2][rows * (D + 2)]
  int64_t q_token, out_token;
  int heads_q, group, window;
  uint32_t group_mul, group_shift;  // row / group = row * group_mul >> group_shift, rows below 2^31
  int max_tiles;          // row tiles of a sequence (a group) of max_tok tokens
  float scale_log2;       // scale * log2(e)
  // attention over shared prefixes alone (kv_shared.cuh)
  const int32_t* cu_seq;  // [groups + 1]
  const int32_t* prefix;  // [groups]
  int groups, group_tok;  // group_tok: new tokens of a group at most
  CutItem* cuts;          // [grid], prefill kernel: the item that begins in each run and goes on in the next

  __device__ int token_of(int packed) const {
    return static_cast<int>(static_cast<uint64_t>(static_cast<uint32_t>(packed)) * group_mul >> group_shift);
  }
};

// One item as the kernels walk it.
struct Item {
  int b, tile, head;
  int tok0, n, kv;     // the sequence's first new token, their number, its cache length
  int row0, rows;      // packed rows of the tile
  int lo, hi;          // visible positions of any of its rows: [lo, hi)
  int kt0, kt1;        // key tiles of this run's part
  long long ub, ue;    // units of the whole item
};

// The first position that a token at position p (below 2^30, negative before the cache) sees through a window.
__host__ __device__ __forceinline__ int window_start(int p, int window) {
  return window > 0 ? max(max(p + 1, 0) - window, 0) : 0;  // (p + 1 - window can leave 32 bits where p is negative)
}
__host__ __device__ __forceinline__ void key_range(int i0, int i1, int base, int kv, bool tree, int window, int& lo, int& hi) {
  hi = tree ? kv : min(max(base + i1 + 1, 0), kv);
  lo = window_start(base + i0, window);
  if (lo > hi) lo = hi;
}
template <int kKeys>
__host__ __device__ __forceinline__ int key_tiles(int lo, int hi) {
  return max((hi + kKeys - 1) / kKeys - lo / kKeys, 1);
}

// n / d of non-negative numbers; the 64-bit division, some hundreds of cycles, only where the numbers need it.
__host__ __device__ __forceinline__ long long quotient(long long n, long long d) {
  if (((n | d) >> 32) == 0) return static_cast<uint32_t>(n) / static_cast<uint32_t>(d);
  return n / d;
}

// Sequences in shared memory: seq[b] = {first new token, cache length, or -1 for one that is left out}, b <= B.
template <int kRows, int kKeys>
struct Walk {
  const int2* seq;
  int B, heads, group, window;
  uint32_t group_mul, group_shift;
  bool tree;
  long long u, u1;
  Item it;
  long long first;  // units before the current (sequence, tile)
  int nk;

  __host__ __device__ int tiles(int b, int& n) const {
    n = seq[b].y < 0 ? 0 : seq[b + 1].x - seq[b].x;
    return (n * group + kRows - 1) / kRows;
  }
  __host__ __device__ void tile_range(int n, int kv, int t, int& lo, int& hi) const {
    const uint32_t r0 = t * kRows, r1 = min((t + 1) * kRows, n * group) - 1;
    const int i0 = static_cast<int>(static_cast<uint64_t>(r0) * group_mul >> group_shift);
    const int i1 = static_cast<int>(static_cast<uint64_t>(r1) * group_mul >> group_shift);
    key_range(i0, i1, kv - n, kv, tree, window, lo, hi);
  }
  // Units of row tile t of sequence b (0 beyond its last).
  __host__ __device__ long long units(int b, int t) const {
    int n;
    if (t >= tiles(b, n)) return 0;
    int lo, hi;
    tile_range(n, seq[b].y, t, lo, hi);
    return static_cast<long long>(key_tiles<kKeys>(lo, hi)) * heads;
  }
  // Positions the walk at a row tile that begins at unit `before` <= u.
  __host__ __device__ void start(int b, int tile, long long before) {
    it.b = b;
    it.tile = tile - 1;
    first = before;
    nk = 0;
    left_ = tiles(b, it.n);
  }
  // The next part of this run, or false.
  __host__ __device__ bool next() {
    if (u >= u1) return false;
    while (nk == 0 || u >= first + static_cast<long long>(nk) * heads) {
      first += static_cast<long long>(nk) * heads;
      ++it.tile;
      while (it.tile >= left_) {
        if (++it.b >= B) return false;
        it.tile = 0;
        left_ = tiles(it.b, it.n);
      }
      it.tok0 = seq[it.b].x;
      it.kv = seq[it.b].y;
      it.row0 = it.tile * kRows;
      it.rows = min(it.n * group - it.row0, kRows);
      tile_range(it.n, it.kv, it.tile, it.lo, it.hi);
      nk = key_tiles<kKeys>(it.lo, it.hi);
    }
    const long long r = u - first;
    it.head = static_cast<int>(quotient(r, nk));
    it.ub = first + static_cast<long long>(it.head) * nk;
    it.ue = it.ub + nk;
    const int base = it.lo / kKeys;
    it.kt0 = base + static_cast<int>(u - it.ub);
    const long long end = it.ue < u1 ? it.ue : u1;
    it.kt1 = base + static_cast<int>(end - it.ub);
    u = end;
    return true;
  }
  // The next item of the run [run0, run1) that run boundaries cut, or false.
  __host__ __device__ bool next_cut(long long run0, long long run1) {
    while (next())
      if (it.ub < run0 || it.ue > run1) return true;
    return false;
  }
  int left_;  // row tiles of the current sequence
};

// A walk in shared memory, one per warp: a lane advances it, all read its item.
template <class W>
__device__ __forceinline__ bool walk_next(W* w) {
  __syncwarp();
  bool more = false;
  if ((threadIdx.x & 31) == 0) more = w->next();
  more = __any_sync(0xFFFFFFFFu, more);
  __syncwarp();
  return more;
}

struct ScanShared {
  long long warp_sum[32];
  long long total, before;
  int b, tile, runs;
};

// The first unit of run c, and the run that holds unit u.
__host__ __device__ __forceinline__ long long run_start(long long c, const ScanShared* sh) {
  return c < sh->runs ? quotient(c * sh->total, sh->runs) : sh->total;
}
__host__ __device__ __forceinline__ int owner_of(long long u, const ScanShared* sh) {
  return static_cast<int>(quotient((u + 1) * sh->runs - 1, sh->total));
}

// Shares out the units of `owners` sequences (or groups) of a.max_tiles row tiles at most, and positions the walk for this
// CTA.  count.units(owner, row tile).  Ends with a barrier.
template <int kThreads, class W, class Count>
__device__ __forceinline__ void deal(const AttArgs& a, int owners, ScanShared* sh, W& w, const Count& count) {
  // (sequence, row tile) pairs, a run of them per thread; sequences of fewer tiles leave gaps
  const uint32_t pairs = static_cast<uint32_t>(owners) * a.max_tiles;  // (below 2^30)
  const uint32_t per = (pairs + kThreads - 1) / kThreads;
  const uint32_t e0 = threadIdx.x * per, e1 = min(e0 + per, pairs);
  int b = e0 < pairs ? e0 / static_cast<uint32_t>(a.max_tiles) : 0, tile = e0 - b * a.max_tiles;
  const int b_first = b, tile_first = tile;
  long long mine = 0;
  for (uint32_t e = e0; e < e1; ++e) {
    mine += count.units(b, tile);
    if (++tile == a.max_tiles) {
      tile = 0;
      ++b;
    }
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  long long incl = mine;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const long long o = __shfl_up_sync(0xFFFFFFFFu, incl, off);
    if (lane >= off) incl += o;
  }
  if (lane == 31) sh->warp_sum[warp] = incl;
  __syncthreads();
  long long before = incl - mine, total = 0;
  if constexpr (kThreads > 256) {  // (by lanes: the loop's sums cost the prefill kernels registers: 4096 tokens over 8192 positions 379 -> 367 us)
    constexpr int kWarps = kThreads / 32;
    long long sums = lane < kWarps ? sh->warp_sum[lane] : 0;
#pragma unroll
    for (int off = 1; off < kWarps; off <<= 1) {
      const long long o = __shfl_up_sync(0xFFFFFFFFu, sums, off);
      if (lane >= off) sums += o;
    }
    total = __shfl_sync(0xFFFFFFFFu, sums, kWarps - 1);
    const long long o = __shfl_sync(0xFFFFFFFFu, sums, warp == 0 ? 0 : warp - 1);
    if (warp > 0) before += o;
  } else {
    for (int i = 0; i < kThreads / 32; ++i) {
      if (i < warp) before += sh->warp_sum[i];
      total += sh->warp_sum[i];
    }
  }
  // as many runs as CTAs, none of them empty; CTAs beyond the last run have no work.  (Runs of some tiles at least
  // were slower: what an item costs to take up and leave is better paid by many CTAs at once.)
  const long long runs = total < gridDim.x ? total : gridDim.x, c = blockIdx.x;
  w.u = c < runs ? quotient(c * total, runs) : 0;
  w.u1 = c < runs ? quotient((c + 1) * total, runs) : 0;
  if (w.u < w.u1 && w.u >= before && w.u < before + mine) {  // (one thread)
    b = b_first;
    tile = tile_first;
    for (long long n; w.u >= before + (n = count.units(b, tile)); before += n)
      if (++tile == a.max_tiles) {
        tile = 0;
        ++b;
      }
    sh->b = b;
    sh->tile = tile;
    sh->before = before;
  }
  if (threadIdx.x == 0) {
    sh->total = total;
    sh->runs = static_cast<int>(runs);
  }
  __syncthreads();
  if (w.u < w.u1) w.start(sh->b, sh->tile, sh->before);
}

// Fills seq (all threads), shares the units out and positions the walk for this CTA.  Ends with a barrier.
template <int kThreads, int kRows, int kKeys>
__device__ __forceinline__ void share_out(const AttArgs& a, int2* seq, ScanShared* sh, Walk<kRows, kKeys>& w) {
  const int B = a.b.B;
  for (int b = threadIdx.x; b <= B; b += kThreads) {
    if (b == B) {
      seq[b] = make_int2(a.b.cu_tok[B], -1);
    } else {
      const SeqSpan s = seq_span(a.b, a.c.page, b);
      if (!s.ok && blockIdx.x == 0) atomicOr(a.err, kErrInvalid);
      seq[b] = make_int2(s.tok0, s.ok ? s.kv : -1);
    }
  }
  __syncthreads();
  w.seq = seq;
  w.B = B;
  w.heads = a.c.heads;
  w.group = a.group;
  w.group_mul = a.group_mul;
  w.group_shift = a.group_shift;
  w.window = a.window;
  w.tree = a.tree != nullptr;
  deal<kThreads>(a, B, sh, w, w);
}


// Adds to a counter that other CTAs share: what this CTA wrote (or saw through a barrier) before is visible to whoever
// reads the sum, and what earlier adders had written is visible afterwards.
__device__ __forceinline__ unsigned int add_acq_rel(unsigned int* p, unsigned int v) {
  unsigned int old;
  asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], %2;" : "=r"(old) : "l"(p), "r"(v) : "memory");
  return old;
}

__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity, volatile int* abort_flag, unsigned int* err) {
  if (ptx::mbar_try_wait(bar, parity)) return true;
  const long long t0 = clock64();
  while (true) {
    if (*abort_flag) return false;
    if (ptx::mbar_try_wait(bar, parity)) return true;
    if (clock64() - t0 > kWaitLimit) {
      *abort_flag = 1;
      atomicOr(err, kErrTimeout);
      return false;
    }
  }
}
// Ignores the abort flag (lets copies in flight land before the CTA exits); bounded.
__device__ __forceinline__ void wait_bar_final(uint64_t* bar, uint32_t parity, unsigned int* err) {
  const long long t0 = clock64();
  while (!ptx::mbar_try_wait(bar, parity))
    if (clock64() - t0 > kWaitLimit) {
      atomicOr(err, kErrTimeout);
      return;
    }
}

// Untiled bulk copy to shared memory; 16-byte aligned addresses and size.
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(ptx::smem_u32(dst)),
      "l"(src), "r"(bytes), "r"(ptx::smem_u32(bar))
      : "memory");
}

// 16 bytes from global to shared memory, tracked by the thread's copy groups.
__device__ __forceinline__ void copy16_async(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_group() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// A pair of scores x, y -> exponents x m + b, y m + b; a pair of probabilities packed to fp16 and added to a running
// pair of sums.  Volatile, so the order in which a row's pairs go through stays as written: exponentials run on a
// pipe of their own at 4 cycles a warp, and the packing and summing of pairs whose exponentials are back go between.
__device__ __forceinline__ uint64_t twice(float x) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %1};" : "=l"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ void exponents(float& x, float& y, uint64_t m, uint64_t b) {
  asm volatile(
      "{\n\t.reg .b64 v;\n\t"
      "mov.b64 v, {%0, %1};\n\t"
      "fma.rn.f32x2 v, v, %2, %3;\n\tmov.b64 {%0, %1}, v;\n\t}"
      : "+f"(x), "+f"(y)
      : "l"(m), "l"(b));
}
__device__ __forceinline__ void ex2_in_order(float& x) { asm volatile("ex2.approx.ftz.f32 %0, %0;" : "+f"(x)); }
__device__ __forceinline__ uint32_t pack_and_add(float x, float y, uint64_t& sum) {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .b64 v;\n\t"
      "cvt.rn.f16x2.f32 %0, %3, %2;\n\t"
      "mov.b64 v, {%2, %3};\n\t"
      "add.rn.f32x2 %1, %1, v;\n\t}"
      : "=r"(p), "+l"(sum)
      : "f"(x), "f"(y));
  return p;
}
__device__ __forceinline__ float both(uint64_t pair) {
  float x, y;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(pair));
  return x + y;
}

__device__ __forceinline__ float max3(float x, float y, float z) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(x), "f"(y), "f"(z));
  return r;
}

// What a query row needs: its factor 2^-e for fp16 (largest value at 2^14 or just above) and what turns a
// product of such rows with codes into a score in powers of two.  amax: largest |value| as bf16 bits.
__device__ __forceinline__ float row_shrink(uint32_t amax) {
  // 2^(14 + 127 - exponent), limited to fp32's normal range (rows below 2^-112 are scaled less)
  const int e = 14 + 127 - static_cast<int>(amax >> 7);
  return exp2_int(min(max(e, -126), 126));
}
__device__ __forceinline__ float row_mult(uint32_t amax, float scale_log2) {
  const int e = min(max(14 + 127 - static_cast<int>(amax >> 7), -126), 126);
  return scale_log2 * exp2_int(-e);
}
// The factor of one group of keys with scale 2^ek: finite, so a zero product stays a zero score.
__device__ __forceinline__ float score_mult(float mult, int ek) {
  return fminf(fmaxf(mult * exp2_int(ek), -3e38f), 3e38f);
}

// Stage bookkeeping of the producer: the key segments (pages, or halves of 128-slot pages) of an item.
// Lane l of the producer warp holds segment seg0 + l: its page and its exponents, or page -1.
struct SegBatch {
  int seg0 = -1, page = -1, ek = 0, ev = 0;
};
constexpr int kBadGroup = 1000;  // in the place of an exponent: no keys there
__device__ __forceinline__ SegBatch load_segs(const AttArgs& a, const Item& it, int seg0, int seg_keys) {
  SegBatch s;
  s.seg0 = seg0;
  const long long key = static_cast<long long>(seg0 + (threadIdx.x & 31)) * seg_keys;
  if (key < it.hi && key + seg_keys > it.lo) {
    const int page = a.b.pages[static_cast<int64_t>(it.b) * a.b.max_pages + key / a.c.page];
    if (page >= 0 && page < a.c.n_pages) {
      s.page = page;
      const int64_t ph = static_cast<int64_t>(page) * a.c.heads + it.head;
      s.ek = a.c.k_exp[ph];
      s.ev = a.c.v_exp[ph];
      s.ek = min(max(s.ek, kKvMinExp), kKvMaxExp);
      s.ev = min(max(s.ev, kKvMinExp), kKvMaxExp);
    } else {
      atomicOr(a.err, kErrInvalid);
    }
  }
  return s;
}

}  // namespace att
}  // namespace qspec
