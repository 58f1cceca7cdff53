// Page tables of sequences that fork, shorten, grow and end; copies of pages; the accepted path of a tree moved
// behind the committed tokens.  Integers and codes only: latency bounds the tables, memory the copies.
#include <cooperative_groups.h>

#include "kv_internal.h"

namespace qspec {
namespace {

namespace cg = cooperative_groups;

// ------------------------------------------------------------------ page tables

// One thread-block cluster does the whole step, so its phases are separated by the hardware's cluster barrier and
// nothing waits on memory:
//   1  new rows take over their parents' entries (+1 on each page's count), old rows are released (-1);
//   2  every CTA looks at all new rows: which of them would write in a page that others hold as well;
//   3  free pages (count 0) are counted by ranges of ids, the counts exchanged through distributed shared memory;
//   4  the k-th free page goes to the k-th page that the rows lack.
// Every result goes by indices alone, never by the order in which atomics arrive.
// 4 rows of 24 entries, 256 of 66: 8 to 13 us, a chain of some twenty reads of memory, cluster barriers and
// scans; the bytes are a few hundred KB at most.
constexpr int kPageThreads = 1024;
constexpr int kMaxRows = QSPEC_KV_MAX_B;
constexpr int kHash = 2 * kMaxRows;
constexpr int kMaxCluster = 8;
static_assert(kMaxRows <= kPageThreads, "a thread to a row");

struct PagesArgs {
  const int32_t* pages;
  const int32_t* room;
  const int32_t* parent;  // null: row r comes from row r
  const int32_t* keep;
  const int32_t* need;
  const int32_t* refs;
  int32_t* new_pages;
  int32_t* new_refs;
  int32_t* src;
  int32_t* dst;
  int32_t* len;
  int32_t* left;
  unsigned int* err;
  int64_t n_pages;
  int rows, new_rows, width, new_width, shift;
};

struct PagesShared {
  int page[kHash], count[kHash], lowest[kHash];  // the pages that new rows would write in, by open addressing
  int first[kMaxRows];                           // each row's first entry that gets a fresh page, twice, and 1 for a copy
  long long start[kMaxRows + 1];                 // fresh pages of the rows before
  long long warp_sum[32];
  int free_of[kMaxCluster];                      // free pages in each CTA's range
};

// Pages that hold n positions.
__device__ __forceinline__ int pages_of(const PagesArgs& a, int n) {
  return static_cast<int>((static_cast<uint32_t>(n) + (1u << a.shift) - 1u) >> a.shift);
}
// Positions that old row b holds pages for; 0 where its number is out of range.
__device__ __forceinline__ int room_of(const PagesArgs& a, int b, bool& bad) {
  const int n = a.room[b];
  if (n >= 0 && static_cast<int64_t>(n) <= static_cast<int64_t>(a.width) << a.shift) return n;
  bad = true;
  return 0;
}
struct NewRow {
  int parent, keep, need;
};
// A row whose numbers do not fit gets nothing.
__device__ __forceinline__ NewRow new_row(const PagesArgs& a, int r, bool& bad) {
  NewRow w{a.parent ? a.parent[r] : r, a.keep[r], a.need[r]};
  bool ok = w.parent < a.rows && w.keep >= 0 && w.need >= w.keep &&
            static_cast<int64_t>(w.need) <= static_cast<int64_t>(a.new_width) << a.shift;
  if (ok) ok = w.keep <= (w.parent >= 0 ? room_of(a, w.parent, bad) : 0);
  if (!ok) {
    bad = true;
    w = NewRow{-1, 0, 0};
  }
  return w;
}

// Adds `sign` to the counts of what the new rows take over and takes it from those of what the old rows held.  A warp to a
// row.  `write`: the entries are written as well.
__device__ __forceinline__ void count_rows(const PagesArgs& a, int warp, int warps, int sign, bool write, bool& bad) {
  const int lane = threadIdx.x & 31;
  for (int w = warp; w < a.rows + a.new_rows; w += warps) {
    const bool fresh = w >= a.rows;
    int from = w, n;
    if (fresh) {
      const NewRow r = new_row(a, w - a.rows, bad);
      from = r.parent;
      n = pages_of(a, r.keep);
    } else {
      n = pages_of(a, room_of(a, w, bad));
    }
    const int32_t* in = a.pages + static_cast<int64_t>(from) * a.width;
    int32_t* out = a.new_pages + static_cast<int64_t>(w - a.rows) * a.new_width;
#pragma unroll 4
    for (int j = lane; j < n; j += 32) {
      const int p = in[j];
      if (fresh && write) out[j] = p;
      if (p >= 0 && p < a.n_pages)
        atomicAdd(a.new_refs + p, fresh ? sign : -sign);
      else
        bad = true;
    }
  }
}

// Sum of v over the threads before this one, and the total.  Two barriers.
__device__ __forceinline__ long long block_scan(long long v, long long* warp_sum, long long& total) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  long long incl = v;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const long long o = __shfl_up_sync(0xFFFFFFFFu, incl, off);
    if (lane >= off) incl += o;
  }
  __syncthreads();
  if (lane == 31) warp_sum[warp] = incl;
  __syncthreads();
  // (each warp scans the warps' sums; with a loop over them in every thread a scan took 2 us)
  static_assert(kPageThreads == 1024, "a lane to a warp");
  long long sums = warp_sum[lane];
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const long long o = __shfl_up_sync(0xFFFFFFFFu, sums, off);
    if (lane >= off) sums += o;
  }
  total = __shfl_sync(0xFFFFFFFFu, sums, 31);
  const long long before = __shfl_sync(0xFFFFFFFFu, sums, warp == 0 ? 0 : warp - 1);
  return (warp == 0 ? 0 : before) + incl - v;
}

__global__ void __launch_bounds__(kPageThreads) pages_kernel(const PagesArgs a) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  PagesShared& sh = *reinterpret_cast<PagesShared*>(smem_raw);
  cg::cluster_group cluster = cg::this_cluster();
  const int ctas = cluster.num_blocks(), cta = cluster.block_rank(), tid = threadIdx.x;
  const int warp = cta + (tid >> 5) * ctas, warps = ctas * (kPageThreads / 32);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  bool bad = false;
  // the ids of this CTA's range, a multiple of four so that counts are read by sixteen bytes
  const int64_t per = ((a.n_pages + 4 * ctas - 1) / (4 * ctas)) * 4, id0 = min(cta * per, a.n_pages), id1 = min(id0 + per, a.n_pages);
  const bool apart = a.new_refs != a.refs;
  auto take_over_counts = [&]() {
    for (int64_t i = id0 + tid; i < id1; i += kPageThreads) a.new_refs[i] = a.refs[i];
  };
  for (int i = tid; i < kHash; i += kPageThreads) {
    sh.page[i] = -1;
    sh.count[i] = 0;
    sh.lowest[i] = kMaxRows;
  }
  if (apart) {
    take_over_counts();
    cluster.sync();
  }
  count_rows(a, warp, warps, 1, true, bad);
  cluster.sync();

  // ---- the rows that go on writing in a page they hold a part of
  int last = -1, slot = 0, part = 0, n_keep = 0, n_need = 0;
  if (tid < a.new_rows) {
    const NewRow r = new_row(a, tid, bad);
    n_keep = pages_of(a, r.keep);
    n_need = pages_of(a, r.need);
    part = r.keep & ((1 << a.shift) - 1);
    if (part != 0 && r.need > r.keep) {
      last = a.pages[static_cast<int64_t>(r.parent) * a.width + (r.keep >> a.shift)];
      if (last >= a.n_pages) last = -1;
    }
  }
  if (last >= 0) {
    slot = static_cast<uint32_t>(last) * 0x9E3779B1u >> 21;  // (2^11 places for at most 2^10 pages)
    for (int seen; (seen = atomicCAS(&sh.page[slot], -1, last)) != -1 && seen != last;) slot = (slot + 1) & (kHash - 1);
    atomicAdd(&sh.count[slot], 1);
    atomicMin(&sh.lowest[slot], tid);
  }
  static_assert(kHash == 1 << 11, "the hash's shift");
  __syncthreads();
  // a copy, unless all that hold the page would write in it and this row is the lowest of them
  const bool copy = last >= 0 && (__ldcg(a.new_refs + last) != sh.count[slot] || sh.lowest[slot] != tid);
  long long lacking;
  const long long start = block_scan(tid < a.new_rows ? n_need - n_keep + copy : 0, sh.warp_sum, lacking);
  if (tid < a.new_rows) {
    sh.start[tid] = start;
    sh.first[tid] = 2 * (n_keep - copy) + copy;
  }

  // ---- free pages of this CTA's range
  long long mine = 0;
  for (int64_t i = id0 + 4 * tid; i < id1; i += 4 * kPageThreads) {
    int c[4] = {1, 1, 1, 1};
    if (i + 4 <= id1) {
      const int4 v = __ldcg(reinterpret_cast<const int4*>(a.new_refs + i));
      c[0] = v.x, c[1] = v.y, c[2] = v.z, c[3] = v.w;
    } else {
      for (int e = 0; i + e < id1; ++e) c[e] = __ldcg(a.new_refs + i + e);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      mine += c[e] == 0;
      bad = bad || c[e] < 0;
    }
  }
  long long in_range;
  block_scan(mine, sh.warp_sum, in_range);
  if (tid < ctas) *cluster.map_shared_rank(&sh.free_of[cta], tid) = static_cast<int>(in_range);
  cluster.sync();
  long long before = 0, free_pages = 0;
  for (int i = 0; i < ctas; ++i) {
    if (i < cta) before += sh.free_of[i];
    free_pages += sh.free_of[i];
  }
  if (bad) atomicOr(a.err, kErrInvalid);
  if (cta == 0 && tid == 0) {
    const long long l = free_pages - lacking;
    *a.left = static_cast<int>(l < -0x7FFFFFFF ? -0x7FFFFFFF : l);
  }
  const bool enough = lacking <= free_pages;
  if (cta == 0 && tid < a.new_rows) {
    const bool c = copy && enough;
    a.src[tid] = c ? last : -1;
    a.len[tid] = c ? part : 0;
    if (!c) a.dst[tid] = -1;
    if (c) atomicSub(a.new_refs + last, 1);  // (still held by another row: never free)
  }
  if (!enough) {  // nothing happened
    if (apart)
      take_over_counts();
    else
      count_rows(a, warp, warps, -1, false, bad);
    return;
  }

  // ---- the k-th free page is the k-th that the rows lack
  for (int64_t i0 = id0; i0 < id1 && before < lacking; i0 += 4 * kPageThreads) {
    const int64_t i = i0 + 4 * tid;
    uint32_t zero = 0;
    if (i + 4 <= id1) {
      const int4 v = __ldcg(reinterpret_cast<const int4*>(a.new_refs + i));
      zero = (v.x == 0) | (v.y == 0) << 1 | (v.z == 0) << 2 | (v.w == 0) << 3;
    } else {
      for (int e = 0; i + e < id1; ++e) zero |= (__ldcg(a.new_refs + i + e) == 0) << e;
    }
    long long here;
    long long k = before + block_scan(__popc(zero), sh.warp_sum, here);
    for (; zero && k < lacking; zero &= zero - 1, ++k) {
      const int id = static_cast<int>(i) + __ffs(zero) - 1;
      int lo = 0, hi = a.new_rows;  // the last row that begins at or before k
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (sh.start[mid] <= k)
          lo = mid;
        else
          hi = mid;
      }
      const int e = (sh.first[lo] >> 1) + static_cast<int>(k - sh.start[lo]);
      a.new_pages[static_cast<int64_t>(lo) * a.new_width + e] = id;
      a.new_refs[id] = 1;
      if (k == sh.start[lo] && (sh.first[lo] & 1)) a.dst[lo] = id;
    }
    before += here;
  }
}

// ------------------------------------------------------------------ copies

// Layers are pointers in the kernel's parameters: one launch for all.
struct Layers {
  uint8_t* codes[2][QSPEC_KV_MAX_LAYERS];
  int8_t* exps[2][QSPEC_KV_MAX_LAYERS];
};

constexpr int kCopyThreads = 256;

struct CopyArgs {
  Layers l;
  const int32_t* src;
  const int32_t* dst;
  const int32_t* len;  // null: whole pages
  unsigned int* err;
  int64_t n_pages;
  int heads, page, dim, heads_per;  // heads of a block: 16 KB of codes at most
};

// A block copies one side (z) of some heads of one pair of pages (x) in one layer (y): four 16-byte loads a thread, then
// the stores.  One round of memory bounds it: 2 to 4 us for up to 13 MB.
__global__ void __launch_bounds__(kCopyThreads) copy_pages_kernel(const __grid_constant__ CopyArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int s = a.src[blockIdx.x], d = a.dst[blockIdx.x], side = blockIdx.z & 1, h0 = (blockIdx.z >> 1) * a.heads_per;
  if (s < 0) return;
  const int n = a.len ? a.len[blockIdx.x] : a.page;
  if (s >= a.n_pages || d < 0 || d >= a.n_pages || n < 0 || n > a.page) {
    if (threadIdx.x == 0) atomicOr(a.err, kErrInvalid);
    return;
  }
  if (s == d) return;
  const int heads = min(a.heads_per, a.heads - h0), head_bytes = a.page * a.dim, per_head = n * a.dim / 16;
  const int8_t* es = a.l.exps[side][blockIdx.y] + static_cast<int64_t>(s) * a.heads + h0;
  int8_t* ed = a.l.exps[side][blockIdx.y] + static_cast<int64_t>(d) * a.heads + h0;
  for (int h = threadIdx.x; h < heads; h += kCopyThreads) ed[h] = es[h];
  const uint8_t* cs = a.l.codes[side][blockIdx.y] + (static_cast<int64_t>(s) * a.heads + h0) * head_bytes;
  uint8_t* cd = a.l.codes[side][blockIdx.y] + (static_cast<int64_t>(d) * a.heads + h0) * head_bytes;
  const int items = heads * per_head;
  constexpr int kAtOnce = 4;
  for (int i0 = threadIdx.x; i0 < items; i0 += kAtOnce * kCopyThreads) {
    uint4 v[kAtOnce];
    int at[kAtOnce];
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      const int i = i0 + k * kCopyThreads;
      if (i < items) {
        const int h = i / per_head;
        at[k] = h * head_bytes + (i - h * per_head) * 16;
        v[k] = *reinterpret_cast<const uint4*>(cs + at[k]);
      }
    }
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k)
      if (i0 + k * kCopyThreads < items) *reinterpret_cast<uint4*>(cd + at[k]) = v[k];
  }
}

// ------------------------------------------------------------------ the accepted path of a tree

constexpr int kCompactWarps = 8;

struct CompactArgs {
  Layers l;
  qspec_kv_batch b;
  const int32_t* nodes;
  const int32_t* count;
  unsigned int* err;
  int64_t n_pages;
  int heads, page, shift, T, first, layers, layers_per;
};

// The smallest e with amax <= 448 * 2^e = 1.75 * 2^(e + 8), limited to the stored range; amax >= 0 as fp32 bits.
__device__ __forceinline__ int exp_of_f32(uint32_t bits) {
  const int e = static_cast<int>(bits >> 23) - 127 - ((bits & 0x7FFFFFu) <= 0x600000u ? 8 : 7);
  return min(max(e, kKvMinExp), kKvMaxExp);
}

// Largest |value| of 16 codes, as the bits of a non-negative fp32 number (bytes below 0x7F order as their values do).
__device__ __forceinline__ uint32_t amax_codes(const uint4& c) {
  uint32_t m = __vmaxu4(__vmaxu4(c.x & 0x7F7F7F7Fu, c.y & 0x7F7F7F7Fu), __vmaxu4(c.z & 0x7F7F7F7Fu, c.w & 0x7F7F7F7Fu));
  m = __vmaxu4(m, m >> 16);
  m = max(m & 0xFFu, m >> 8 & 0xFFu);
  return __float_as_uint(e4m3x2_to_f32(m).x);
}

// 16 codes under 2^from as codes under 2^to.
__device__ __forceinline__ uint4 rescaled(uint4 c, int from, int to) {
  if (from == to) return c;
  // (2^(from - to) can leave fp32's range of exponents by no more than 80, and the codes' values have 17 of their own)
  const float f = exp2_int(from - to);
  uint32_t* w = reinterpret_cast<uint32_t*>(&c);
#pragma unroll
  for (int m = 0; m < 4; ++m) {
    const float2 lo = e4m3x2_to_f32(w[m] & 0xFFFFu), hi = e4m3x2_to_f32(w[m] >> 16);
    w[m] = f32_to_e4m3x2(lo.x * f, lo.y * f) | f32_to_e4m3x2(hi.x * f, hi.y * f) << 16;
  }
  return c;
}

// A block owns one side of up to eight heads of one sequence, a warp one head, in some layers one after the other (the chain of
// indices is paid once for them).  A lane takes 16 codes of a token, the warp 16 tokens (with heads of 64: 32) at a time: paths of
// up to that length are read once, longer ones once for the scales and once to be moved.  A path's nodes rise, so a token's new
// place is never behind the places that are still to be read, in the order of the tokens.  What is written follows the append: a
// page begun here takes the scale of what it receives, another one grows where it must.
// One path in one layer takes 4 us.  64 paths in 32 layers take 22 us, 1.5 TB/s in reads and writes of 64 or 128 bytes; with the
// places worked out for each layer anew, by divisions, it took 43, so instructions bounded it.  (The next layer's codes loaded
// ahead: 23 us.)
template <int D>
__global__ void __launch_bounds__(32 * kCompactWarps, 4) compact_kernel(const __grid_constant__ CompactArgs a) {
  constexpr int kPerTok = D / 16, kItems = 4, kAtOnce = 32 * kItems / kPerTok, kPages = QSPEC_MAX_TREE / 16 + 1;
  __shared__ int64_t from_of[QSPEC_MAX_TREE], to_of[QSPEC_MAX_TREE];  // a token's codes of head 0
  __shared__ int64_t exp_of[QSPEC_MAX_TREE];                          // and the scale that they have
  __shared__ int page_of[kPages + 1];  // pages of the tree's positions, from the path's first on
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int b = blockIdx.x, side = blockIdx.z & 1, lane = threadIdx.x & 31;
  const int head = blockIdx.y * kCompactWarps + (threadIdx.x >> 5);
  const SeqSpan sp = seq_span(a.b, a.page, b);
  const int n = a.count[b];
  const int tree = sp.n - a.first;  // nodes that were appended
  const int base = sp.kv - tree;    // the position of node 0, and of the path's first token
  const int P = a.page, pg0 = base >> a.shift;
  bool ok = sp.ok && n >= 0 && n <= a.T && n <= max(tree, 0) && sp.n <= sp.kv;
  int j = 0;
  if (ok && n > 0) {
    if (threadIdx.x < n) {
      const int32_t* at = a.nodes + static_cast<int64_t>(b) * a.T + threadIdx.x;
      j = at[0];
      ok = j >= 0 && j < tree && (threadIdx.x == 0 || j > at[-1]);
    }
    const int t = threadIdx.x - QSPEC_MAX_TREE;
    if (tree > QSPEC_MAX_TREE) {
      ok = false;
    } else if (t >= 0 && t < kPages + 1) {
      int p = 0;
      if (pg0 + t <= (sp.kv - 1) >> a.shift) {
        p = a.b.pages[static_cast<int64_t>(b) * a.b.max_pages + pg0 + t];
        ok = p >= 0 && p < a.n_pages;
      }
      page_of[t] = p;
    }
  }
  ok = __syncthreads_and(ok);
  if (!ok) {
    if (threadIdx.x == 0) atomicOr(a.err, kErrInvalid);
    return;
  }
  if (n == 0) return;
  const int64_t page_codes = static_cast<int64_t>(a.heads) * P * D;
  if (threadIdx.x < n) {
    const int from = base + j, to = base + threadIdx.x, page = page_of[(from >> a.shift) - pg0];
    exp_of[threadIdx.x] = static_cast<int64_t>(page) * a.heads;
    from_of[threadIdx.x] = page * page_codes + (from & (P - 1)) * D;
    to_of[threadIdx.x] = page_of[(to >> a.shift) - pg0] * page_codes + (to & (P - 1)) * D;
  }
  __syncthreads();
  if (head >= a.heads) return;
  const int pages = ((base + n - 1) >> a.shift) - pg0 + 1;
  const int layer0 = (blockIdx.z >> 1) * a.layers_per, layer1 = min(layer0 + a.layers_per, a.layers);
#pragma unroll 1
  for (int layer = layer0; layer < layer1; ++layer) {
    uint8_t* const codes = a.l.codes[side][layer] + static_cast<int64_t>(head) * P * D;
    int8_t* const exps = a.l.exps[side][layer] + head;
    auto exp_at = [&](int64_t i) { return min(max(static_cast<int>(exps[i]), kKvMinExp), kKvMaxExp); };
    uint4 c[kItems];
    int e_of[kItems];
    auto load = [&](int t0) {  // tokens t0 ...: the codes of the lane's items and their scales
#pragma unroll
      for (int k = 0; k < kItems; ++k) {
        const int i = k * 32 + lane, t = t0 + i / kPerTok;
        if (t0 + k * (32 / kPerTok) >= n) break;
        c[k] = make_uint4(0, 0, 0, 0);
        e_of[k] = 0;
        if (t < n) {
          c[k] = *reinterpret_cast<const uint4*>(codes + from_of[t] + (i % kPerTok) * 16);
          e_of[k] = exp_at(exp_of[t]);
        }
      }
    };
    const int old = exp_at(static_cast<int64_t>(page_of[0]) * a.heads);  // (the first page alone can be one that goes on)
    uint32_t amax[kPages] = {};
#pragma unroll 1
    for (int t0 = 0; t0 < n; t0 += kAtOnce) {
      load(t0);
#pragma unroll
      for (int k = 0; k < kItems; ++k) {
        if (t0 + k * (32 / kPerTok) >= n) break;
        const int t = t0 + (k * 32 + lane) / kPerTok, q = ((base + t) >> a.shift) - pg0;
        const uint32_t v = __float_as_uint(__uint_as_float(amax_codes(c[k])) * exp2_int(e_of[k]));
#pragma unroll
        for (int p = 0; p < kPages; ++p)
          if (t < n && q == p) amax[p] = max(amax[p], v);
      }
    }
    int e_new[kPages];
#pragma unroll
    for (int p = 0; p < kPages; ++p) {
      e_new[p] = 0;
      if (p >= pages) break;
      e_new[p] = exp_of_f32(__reduce_max_sync(0xFFFFFFFFu, amax[p]));
      if ((pg0 + p) * P < base) e_new[p] = max(old, e_new[p]);
    }
#pragma unroll 1
    for (int t0 = 0; t0 < n; t0 += kAtOnce) {
      if (n > kAtOnce) load(t0);
      __syncwarp();  // (what these tokens' places hold has been read by all lanes)
#pragma unroll
      for (int k = 0; k < kItems; ++k) {
        if (t0 + k * (32 / kPerTok) >= n) break;
        const int i = k * 32 + lane, t = t0 + i / kPerTok, q = ((base + t) >> a.shift) - pg0;
        if (t < n) {
          int e = e_new[0];
#pragma unroll
          for (int p = 1; p < kPages; ++p) e = q == p ? e_new[p] : e;
          *reinterpret_cast<uint4*>(codes + to_of[t] + (i % kPerTok) * 16) = rescaled(c[k], e_of[k], e);
        }
      }
      __syncwarp();
    }
    if (pg0 * P < base && e_new[0] > old) {  // the page grows: its other slots again
      uint4* at = reinterpret_cast<uint4*>(codes + page_of[0] * page_codes);
      for (int i = lane; i < P * kPerTok; i += 32) {
        const int t = pg0 * P + i / kPerTok - base;
        if (t < 0 || t >= n) at[i] = rescaled(at[i], old, e_new[0]);
      }
    }
    if (lane == 0) {
#pragma unroll
      for (int p = 0; p < kPages; ++p)
        if (p < pages) exps[static_cast<int64_t>(page_of[p]) * a.heads] = static_cast<int8_t>(e_new[p]);
    }
  }
}

// Layers of one shape; their pointers.
qspec_status check_layers(const qspec_kv_cache* c, int32_t n, Layers& l) {
  if (!c || n <= 0) return QSPEC_ERR_INVALID_ARG;
  if (n > QSPEC_KV_MAX_LAYERS) return QSPEC_ERR_UNSUPPORTED_SHAPE;
  for (int i = 0; i < n; ++i) {
    if (!c[i].k || !c[i].v || !c[i].k_exp || !c[i].v_exp || c[i].reserved != 0 || c[i].n_pages <= 0 || c[i].heads <= 0)
      return QSPEC_ERR_INVALID_ARG;
    if (c[i].n_pages != c[0].n_pages || c[i].heads != c[0].heads || c[i].page != c[0].page || c[i].dim != c[0].dim)
      return QSPEC_ERR_UNSUPPORTED_SHAPE;
    if (!aligned16(c[i].k) || !aligned16(c[i].v)) return QSPEC_ERR_MISALIGNED;
    l.codes[0][i] = c[i].k;
    l.codes[1][i] = c[i].v;
    l.exps[0][i] = c[i].k_exp;
    l.exps[1][i] = c[i].v_exp;
  }
  if ((c->page != 16 && c->page != 32 && c->page != 64 && c->page != 128) || (c->dim != 64 && c->dim != 128) ||
      c->heads > 4096 || c->n_pages > 0x7FFFFFFF)
    return QSPEC_ERR_UNSUPPORTED_SHAPE;
  return QSPEC_OK;
}

}  // namespace
}  // namespace qspec

using namespace qspec;

extern "C" qspec_status qspec_kv_pages(const int32_t* pages, const int32_t* room, int32_t rows, int32_t max_pages,
                                       const int32_t* parent, const int32_t* keep, const int32_t* need, int32_t new_rows,
                                       int32_t new_max_pages, const int32_t* refs, int64_t n_pages, int32_t page,
                                       int32_t* new_pages, int32_t* new_refs, int32_t* copy_src, int32_t* copy_dst,
                                       int32_t* copy_len, int32_t* left, qspec_stream_t stream) {
  if (rows < 0 || new_rows < 0 || rows + static_cast<int64_t>(new_rows) == 0 || !refs || !new_refs || !left || n_pages <= 0)
    return QSPEC_ERR_INVALID_ARG;
  if (rows > 0 && (!pages || !room || max_pages <= 0)) return QSPEC_ERR_INVALID_ARG;
  if (new_rows > 0 && (!keep || !need || !new_pages || !copy_src || !copy_dst || !copy_len || new_max_pages <= 0))
    return QSPEC_ERR_INVALID_ARG;
  if (page != 16 && page != 32 && page != 64 && page != 128) return QSPEC_ERR_UNSUPPORTED_SHAPE;
  if (rows > kMaxRows || new_rows > kMaxRows || n_pages > 0x7FFFFFFF ||
      (rows > 0 && static_cast<int64_t>(max_pages) * page > (int64_t(1) << 30)) ||
      (new_rows > 0 && static_cast<int64_t>(new_max_pages) * page > (int64_t(1) << 30)))
    return QSPEC_ERR_UNSUPPORTED_SHAPE;
  if (rows > 0 && new_rows > 0) {  // a table is read while the other is written
    const char *p = reinterpret_cast<const char*>(pages), *q = reinterpret_cast<const char*>(new_pages);
    if (p < q + 4 * static_cast<int64_t>(new_rows) * new_max_pages && q < p + 4 * static_cast<int64_t>(rows) * max_pages)
      return QSPEC_ERR_INVALID_ARG;
  }
  if (refs != new_refs) {
    const char *p = reinterpret_cast<const char*>(refs), *q = reinterpret_cast<const char*>(new_refs);
    if (p < q + 4 * n_pages && q < p + 4 * n_pages) return QSPEC_ERR_INVALID_ARG;
  }
  if (!aligned16(refs) || !aligned16(new_refs) || !aligned4(pages) || !aligned4(room) || !aligned4(parent) || !aligned4(keep) ||
      !aligned4(need) || !aligned4(new_pages) || !aligned4(copy_src) || !aligned4(copy_dst) || !aligned4(copy_len) || !aligned4(left))
    return QSPEC_ERR_MISALIGNED;
  // no other input is written either, as rows are read again behind the first writes; the counts alone may be in place
  const Words in[] = {{rows > 0 ? pages : nullptr, static_cast<int64_t>(rows) * max_pages}, {rows > 0 ? room : nullptr, rows},
                      {new_rows > 0 ? parent : nullptr, new_rows}, {new_rows > 0 ? keep : nullptr, new_rows},
                      {new_rows > 0 ? need : nullptr, new_rows}, {refs != new_refs ? refs : nullptr, n_pages}};
  const Words out[] = {{new_refs, n_pages}, {left, 1}, {new_pages, static_cast<int64_t>(new_rows) * new_max_pages}, {copy_src, new_rows},
                       {copy_dst, new_rows}, {copy_len, new_rows}};
  if (outputs_overlap(out, new_rows > 0 ? 6 : 2, in, 6)) return QSPEC_ERR_INVALID_ARG;
  PagesArgs a{pages, room, parent, keep, need, refs, new_pages, new_refs, copy_src, copy_dst, copy_len, left, linear_error_word(),
              n_pages, rows, new_rows, rows > 0 ? max_pages : 0, new_rows > 0 ? new_max_pages : 0};
  if (!a.err) return QSPEC_ERR_CUDA;
  while ((1 << a.shift) < page) ++a.shift;
  const int smem = sizeof(PagesShared);
  if (cudaFuncSetAttribute(pages_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) return QSPEC_ERR_CUDA;
  const int ctas = kMaxCluster;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kPageThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = reinterpret_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim = {static_cast<unsigned int>(ctas), 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, pages_kernel, static_cast<const PagesArgs>(a)) == cudaSuccess ? QSPEC_OK : QSPEC_ERR_CUDA;
}

extern "C" qspec_status qspec_kv_copy_pages(const qspec_kv_cache* caches, int32_t n_caches, const int32_t* src, const int32_t* dst,
                                            const int32_t* len, int32_t n, qspec_stream_t stream) {
  const bool none = n == 0 && !src && !dst && !len;
  if (!none && (!src || !dst || n <= 0)) return QSPEC_ERR_INVALID_ARG;
  CopyArgs a;
  const qspec_status st = check_layers(caches, n_caches, a.l);
  if (st != QSPEC_OK || none) return st;
  if (!aligned4(src) || !aligned4(dst) || !aligned4(len)) return QSPEC_ERR_MISALIGNED;
  a.src = src;
  a.dst = dst;
  a.len = len;
  a.err = linear_error_word();
  if (!a.err) return QSPEC_ERR_CUDA;
  a.n_pages = caches->n_pages;
  a.heads = caches->heads;
  a.page = caches->page;
  a.dim = caches->dim;
  const int fit = 16384 / (a.page * a.dim);
  a.heads_per = fit < a.heads ? fit : a.heads;
  const dim3 grid(n, n_caches, 2 * ((a.heads + a.heads_per - 1) / a.heads_per));
  return launch_pdl(copy_pages_kernel, grid, dim3(kCopyThreads), 0, reinterpret_cast<cudaStream_t>(stream), a);
}

extern "C" qspec_status qspec_kv_compact(const qspec_kv_cache* caches, int32_t n_caches, const qspec_kv_batch* batch,
                                         const int32_t* nodes, const int32_t* count, int32_t T, int32_t first, qspec_stream_t stream) {
  if (!nodes || !count || T <= 0 || first < 0) return QSPEC_ERR_INVALID_ARG;
  CompactArgs a;
  qspec_status st = check_layers(caches, n_caches, a.l);
  if (st != QSPEC_OK) return st;
  if ((st = check_kv(caches, batch)) != QSPEC_OK) return st;
  for (int i = 1; i < n_caches; ++i)  // (a path that moved twice at once)
    for (int j = 0; j < i; ++j)
      if (a.l.codes[0][i] == a.l.codes[0][j] || a.l.codes[1][i] == a.l.codes[1][j]) return QSPEC_ERR_INVALID_ARG;
  if (T > QSPEC_MAX_TREE) return QSPEC_ERR_UNSUPPORTED_SHAPE;
  if (!aligned4(nodes) || !aligned4(count)) return QSPEC_ERR_MISALIGNED;
  a.b = *batch;
  a.nodes = nodes;
  a.count = count;
  a.err = linear_error_word();
  if (!a.err) return QSPEC_ERR_CUDA;
  a.n_pages = caches->n_pages;
  a.heads = caches->heads;
  a.page = caches->page;
  for (a.shift = 0; (1 << a.shift) < a.page;) ++a.shift;
  a.T = T;
  a.first = first;
  // layers of a block: one, unless the blocks are more than three times what is resident (64 paths in 32 layers: two 22 us, three 24,
  // six 33)
  const int64_t all = static_cast<int64_t>(batch->B) * ((a.heads + kCompactWarps - 1) / kCompactWarps) * 2 * n_caches;
  const int64_t per = all / (12 * num_sms());
  a.layers = n_caches;
  a.layers_per = per < 1 ? 1 : per > n_caches ? n_caches : static_cast<int>(per);
  const dim3 grid(batch->B, (a.heads + kCompactWarps - 1) / kCompactWarps, 2 * ((n_caches + a.layers_per - 1) / a.layers_per));
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return caches->dim == 128 ? launch_pdl(compact_kernel<128>, grid, dim3(32 * kCompactWarps), 0, s, a)
                            : launch_pdl(compact_kernel<64>, grid, dim3(32 * kCompactWarps), 0, s, a);
}
