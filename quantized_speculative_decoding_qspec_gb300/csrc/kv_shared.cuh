// Attention for groups of sequences that share a prefix: what the kernels walk.
//
// The rows of a group and key head are the new tokens of all its sequences times the G query heads, packed as ever; an item
// is one (group, row tile, key head).  Its keys come as one stream of tiles: first the prefix, which all its rows see and
// which is read once for them, then what each sequence of the tile has alone, which is masked for the others' rows.  A
// sequence's own keys are read once as well (by the row tiles that its tokens lie in); the products with the other rows cost
// nothing where memory bounds a tile, and tiles of the tensor cores have 16 rows or 128 in any case.  So one launch does both
// parts, the softmax of a row runs over both, and the equal runs, tickets and sums of kv_sched.cuh serve unchanged.
#pragma once

#include "kv_sched.cuh"

namespace qspec {
namespace att {

// Key tiles of [lo, hi).
template <int kKeys>
__host__ __device__ __forceinline__ int tiles_between(int lo, int hi) {
  return lo < hi ? (hi + kKeys - 1) / kKeys - lo / kKeys : 0;
}

// As Walk, over groups.  grp[g] = {first sequence, prefix length or -1 for a group that is left out}, g <= groups; cu and kv are
// the batch's arrays (sequences of a group that is not left out are in order).  Of an item, b is the group, tok0 its first token,
// n its tokens, [lo, hi) what the tile's rows see of the prefix, kv the sequence through whose pages the prefix is read; kt0 and
// kt1 count the tiles of the item's own stream.
template <int kRows, int kKeys>
struct SharedWalk {
  static constexpr int kRowsOf = kRows;
  const int2* grp;
  const int32_t* cu;
  const int32_t* kv;
  int groups, heads, group, window;
  uint32_t group_mul, group_shift;
  bool tree;
  long long u, u1;
  Item it;
  long long first;  // units before the current (group, tile)
  int nk;

  __host__ __device__ int token_of(int packed) const {
    return static_cast<int>(static_cast<uint64_t>(static_cast<uint32_t>(packed)) * group_mul >> group_shift);
  }
  // The sequence among [s0, s1) that has the token; the group has it.
  __host__ __device__ int seq_of(int token, int s0, int s1) const {
    while (s1 - s0 > 1) {
      const int mid = (s0 + s1) >> 1;
      if (cu[mid] <= token)
        s0 = mid;
      else
        s1 = mid;
    }
    return s0;
  }
  // What the tokens t0 .. t1 of the step see of sequence s behind the first p positions.
  __host__ __device__ void own_range(int s, int t0, int t1, int p, int& lo, int& hi) const {
    const int c0 = cu[s], n = cu[s + 1] - c0;
    key_range(max(t0 - c0, 0), min(t1 - c0, n - 1), kv[s] - n, kv[s], tree, window, lo, hi);
    lo = min(max(lo, p), hi);
  }
  __host__ __device__ int tiles(int g, int& n) const {
    n = grp[g].y < 0 ? 0 : cu[grp[g + 1].x] - cu[grp[g].x];
    return (n * group + kRows - 1) / kRows;
  }
  // Key tiles of row tile t of group g with n tokens: what one of `lanes` lanes that share the sequences has to add (the first of
  // them the prefix, given the first position of it that a row sees).
  __host__ __device__ int own_tiles(int g, int t, int n, int lane, int lanes, int& lo) const {
    const int s0 = grp[g].x, s1 = grp[g + 1].x, p = grp[g].y, tok0 = cu[s0];
    const int t0 = tok0 + token_of(t * kRows), t1 = tok0 + token_of(min((t + 1) * kRows, n * group) - 1);
    int total = 0;
    lo = window > 0 ? p : 0;
    for (int s = seq_of(t0, s0, s1) + lane; s < s1 && cu[s] <= t1; s += lanes) {
      if (cu[s + 1] == cu[s]) continue;
      int a, b;
      own_range(s, t0, t1, p, a, b);
      total += tiles_between<kKeys>(a, b);
      if (window > 0) lo = min(lo, window_start(kv[s] - cu[s + 1] + max(t0, cu[s]), window));
    }
    return total;
  }
  __host__ __device__ int all_tiles(int g, int own, int lo) const {
    return max(own + tiles_between<kKeys>(lo, grp[g].y), 1);  // (rows that see nothing are written as well)
  }
  __host__ __device__ long long units(int g, int t) const {
    int n, lo;
    if (t >= tiles(g, n)) return 0;
    const int own = own_tiles(g, t, n, 0, 1, lo);
    return static_cast<long long>(all_tiles(g, own, lo)) * heads;
  }
  __host__ __device__ void enter(int g) {
    left_ = tiles(g, it.n);
    if (left_ > 0) {
      it.kv = grp[g].x;
      while (cu[it.kv + 1] == cu[it.kv]) ++it.kv;
    }
  }
  __host__ __device__ void start(int g, int tile, long long before) {
    it.b = g;
    it.tile = tile - 1;
    first = before;
    nk = 0;
    enter(g);
  }
  // One step of a walk: -1 at the end of the run, 0 for a row tile whose key tiles are to be counted into nk and it.lo, 1 for
  // the next part of the run in `it`.
  __host__ __device__ int step() {
    if (u >= u1) return -1;
    if (nk == 0 || u >= first + static_cast<long long>(nk) * heads) {
      first += static_cast<long long>(nk) * heads;
      nk = 0;
      ++it.tile;
      while (it.tile >= left_) {
        if (++it.b >= groups) return -1;
        it.tile = 0;
        enter(it.b);
      }
      it.tok0 = cu[grp[it.b].x];
      it.row0 = it.tile * kRows;
      it.rows = min(it.n * group - it.row0, kRows);
      it.hi = grp[it.b].y;
      return 0;
    }
    const long long r = u - first;
    it.head = static_cast<int>(quotient(r, nk));
    it.ub = first + static_cast<long long>(it.head) * nk;
    it.ue = it.ub + nk;
    const long long end = it.ue < u1 ? it.ue : u1;
    it.kt0 = static_cast<int>(u - it.ub);
    it.kt1 = static_cast<int>(end - it.ub);
    u = end;
    return 1;
  }
  __host__ __device__ bool next() {
    for (int s; (s = step()) <= 0;) {
      if (s < 0) return false;
      const int own = own_tiles(it.b, it.tile, it.n, 0, 1, it.lo);
      nk = all_tiles(it.b, own, it.lo);
    }
    return true;
  }
  __host__ __device__ bool next_cut(long long run0, long long run1) {
    while (next())
      if (it.ub < run0 || it.ue > run1) return true;
    return false;
  }
  int left_;  // row tiles of the current group
};

// The whole warp advances a walk in shared memory: a lane steps, all count.
template <int kRows, int kKeys>
__device__ __forceinline__ bool walk_next(SharedWalk<kRows, kKeys>* w) {
  const int lane = threadIdx.x & 31;
  while (true) {
    __syncwarp();
    int s = 0;
    if (lane == 0) s = w->step();
    s = __shfl_sync(0xFFFFFFFFu, s, 0);
    __syncwarp();
    if (s != 0) return s > 0;
    int lo;
    const int own = __reduce_add_sync(0xFFFFFFFFu, w->own_tiles(w->it.b, w->it.tile, w->it.n, lane, 32, lo));
    lo = __reduce_min_sync(0xFFFFFFFFu, lo);
    __syncwarp();
    if (lane == 0) {
      w->it.lo = lo;
      w->nk = w->all_tiles(w->it.b, own, lo);
    }
  }
}

template <bool kShared, int kRows, int kKeys>
struct WalkOf {
  using type = Walk<kRows, kKeys>;
};
template <int kRows, int kKeys>
struct WalkOf<true, kRows, kKeys> {
  using type = SharedWalk<kRows, kKeys>;
};

// Units of (group, row tile) pairs, counted ahead in shared memory where the pairs are few: by a thread to a sequence, which adds its own
// tiles to the row tiles that it has tokens in.  (By a thread to a pair, one that goes through 64 sequences takes 5 us, and the
// walk begins with three such counts.)
constexpr int kCounted = 512;
struct Count {
  int own, lo;  // tiles of the sequences' own keys; the first position of the prefix that a row sees
};
template <class W>
struct Counted {
  const W& w;
  const Count* count;  // null: not counted ahead
  int max_tiles;
  __device__ long long units(int g, int t) const {
    if (!count) return w.units(g, t);
    int n;
    if (t >= w.tiles(g, n)) return 0;
    const Count c = count[g * max_tiles + t];
    return static_cast<long long>(w.all_tiles(g, c.own, c.lo)) * w.heads;
  }
};

// The group of sequence b: the last one that begins at or before it.
__device__ __forceinline__ int group_of(const int2* grp, int groups, int b) {
  int lo = 0, hi = groups;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (grp[mid].x <= b)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

// Fills grp (all threads), shares the units out and positions the walk for this CTA.  Ends with a barrier.
// A prefix ends where the new tokens of one of its sequences begin, at the latest.  A group with a sequence whose numbers are
// out of range is left out; so are all if the groups' bounds are not in order.  scratch: kCounted numbers of shared memory that is
// not in use yet.
template <int kThreads, int kRows, int kKeys>
__device__ __forceinline__ void share_out(const AttArgs& a, int2* grp, ScanShared* sh, SharedWalk<kRows, kKeys>& w,
                                          Count* scratch) {
  const int G = a.groups, B = a.b.B;
  bool bad = false;
  for (int g = threadIdx.x; g <= G; g += kThreads) {
    const int s = a.cu_seq[g];
    if (s < 0 || s > B || (g > 0 && a.cu_seq[g - 1] > s)) bad = true;
    int p = -1;
    if (g < G) {
      p = a.prefix[g];
      if (p < 0 || p > static_cast<int64_t>(a.b.max_pages) * a.c.page) p = -1;
      if (p < 0 && blockIdx.x == 0) atomicOr(a.err, kErrInvalid);
    }
    grp[g] = make_int2(s, p);
  }
  const bool disorder = __syncthreads_or(bad);
  if (disorder) {
    for (int g = threadIdx.x; g <= G; g += kThreads) grp[g] = make_int2(0, -1);
    if (blockIdx.x == 0 && threadIdx.x == 0) atomicOr(a.err, kErrInvalid);
  } else {
    for (int b = grp[0].x + threadIdx.x; b < grp[G].x; b += kThreads) {
      const int lo = group_of(grp, G, b);
      const SeqSpan s = seq_span(a.b, a.c.page, b);
      if (!s.ok && blockIdx.x == 0) atomicOr(a.err, kErrInvalid);
      if (!s.ok)
        atomicMin(&grp[lo].y, -1);
      else if (s.n > 0)
        atomicMin(&grp[lo].y, max(s.kv - s.n, 0));
    }
  }
  __syncthreads();
  for (int g = threadIdx.x; g < G; g += kThreads) {  // (their sequences' numbers are in order, or they are out already)
    if (grp[g].y >= 0 && a.b.cu_tok[grp[g + 1].x] - a.b.cu_tok[grp[g].x] > a.group_tok) {
      grp[g].y = -1;
      if (blockIdx.x == 0) atomicOr(a.err, kErrInvalid);
    }
  }
  __syncthreads();
  w.grp = grp;
  w.cu = a.b.cu_tok;
  w.kv = a.b.kv_len;
  w.groups = G;
  w.heads = a.c.heads;
  w.group = a.group;
  w.group_mul = a.group_mul;
  w.group_shift = a.group_shift;
  w.window = a.window;
  w.tree = a.tree != nullptr;
  const uint32_t pairs = static_cast<uint32_t>(G) * a.max_tiles;
  const bool counted = pairs <= kCounted;
  if (counted) {
    for (uint32_t e = threadIdx.x; e < pairs; e += kThreads) scratch[e] = Count{0, a.window > 0 ? 0x7FFFFFFF : 0};
    __syncthreads();
    for (int b = grp[0].x + threadIdx.x; b < grp[G].x; b += kThreads) {
      const int g = group_of(grp, G, b), p = grp[g].y;
      if (p < 0) continue;
      const int c0 = w.cu[b], c1 = w.cu[b + 1], tok0 = w.cu[grp[g].x];
      if (c1 == c0) continue;
      const int row0 = (c0 - tok0) * a.group, row1 = (c1 - tok0) * a.group, all = (w.cu[grp[g + 1].x] - tok0) * a.group;
      for (int t = row0 / kRows; t * kRows < row1; ++t) {
        const int t0 = tok0 + w.token_of(t * kRows), t1 = tok0 + w.token_of(min((t + 1) * kRows, all) - 1);
        Count* const at = scratch + g * a.max_tiles + t;
        int lo, hi;
        w.own_range(b, t0, t1, p, lo, hi);
        atomicAdd(&at->own, tiles_between<kKeys>(lo, hi));
        if (a.window > 0) atomicMin(&at->lo, min(window_start(w.kv[b] - c1 + max(t0, c0), a.window), p));
      }
    }
    __syncthreads();
  }
  const Counted<SharedWalk<kRows, kKeys>> c{w, counted ? scratch : nullptr, a.max_tiles};
  deal<kThreads>(a, G, sh, w, c);
}

// An item's stream: its segments in order, [0] the prefix.  seg = {tiles up to its end, first key tile, sequence or -1, end of
// what is seen}.
// Own tiles of the prefill kernel's full items are taken in turn from the sequences of the first and of the second query tile, so
// that one's softmax runs under the other's products (128 sequences of up to 4000 positions of their own: 310 -> 278 us): behind the prefix
// come those of a sequence that has rows in both, then the others in proportion to what each query tile has.
struct Plan {
  int count;
  int prefix, half0, both, half1;  // tiles, in the order of the segments
  int seq0, seq1;        // the group's sequences
  int pre_lo;            // from here on every row sees the prefix
  int one_lo, one_hi;    // where all rows are of one sequence: what they all see of its own
};

// One warp makes the plan of the walk's item.  Returns its tiles.
template <int kKeys, class W>
__device__ __forceinline__ int make_plan(const W* w, Plan* plan, int4* seg) {
  // the rows of the second query tile begin here, counted in the group's rows
  const long long half = static_cast<long long>(w->it.row0) + (W::kRowsOf > 128 && w->it.rows > W::kRowsOf / 2 ? W::kRowsOf / 2 : W::kRowsOf);
  const Item& it = w->it;
  const int lane = threadIdx.x & 31, s0 = w->grp[it.b].x, s1 = w->grp[it.b + 1].x, p = it.hi;
  const int t0 = it.tok0 + w->token_of(it.row0), t1 = it.tok0 + w->token_of(it.row0 + it.rows - 1);
  const int first = w->seq_of(t0, s0, s1);
  int end = tiles_between<kKeys>(it.lo, p), count = 1, pre_lo = 0, one_lo = 0, one_hi = 0;
  int first_half = 0, in_both = 0;
  const int prefix = end;
  if (lane == 0) seg[0] = make_int4(end, it.lo / kKeys, -1, p);
  for (int s_at = first;; s_at += 32) {
    const int s = s_at + lane;
    const bool in = s < s1 && w->cu[s] <= t1, real = in && w->cu[s + 1] > w->cu[s];
    int lo = 0, hi = 0;
    if (real) {
      w->own_range(s, t0, t1, p, lo, hi);
      const int c0 = w->cu[s], c1 = w->cu[s + 1], kv = w->kv[s], base = kv - (c1 - c0);
      pre_lo = max(pre_lo, window_start(base + min(t1, c1 - 1) - c0, w->window));
      if (c0 <= t0 && c1 > t1) {
        one_lo = max(window_start(base + t1 - c0, w->window), p);
        one_hi = w->tree ? max(base, 0) : min(max(base + t0 - c0 + 1, 0), kv);
      }
    }
    const int mine = tiles_between<kKeys>(lo, hi);
    if (mine > 0) {
      if (static_cast<long long>(w->cu[s + 1] - it.tok0) * w->group <= half)
        first_half += mine;
      else if (static_cast<long long>(w->cu[s] - it.tok0) * w->group < half)
        in_both += mine;
    }
    int incl = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int o = __shfl_up_sync(0xFFFFFFFFu, incl, off);
      if (lane >= off) incl += o;
    }
    const uint32_t has = __ballot_sync(0xFFFFFFFFu, mine > 0);
    if (mine > 0) seg[count + __popc(has & ((1u << lane) - 1u))] = make_int4(end + incl, lo / kKeys, s, hi);
    count += __popc(has);
    end += __shfl_sync(0xFFFFFFFFu, incl, 31);
    if (!__all_sync(0xFFFFFFFFu, in)) break;
  }
  pre_lo = __reduce_max_sync(0xFFFFFFFFu, pre_lo);
  one_lo = __reduce_max_sync(0xFFFFFFFFu, one_lo);
  one_hi = __reduce_max_sync(0xFFFFFFFFu, one_hi);
  first_half = __reduce_add_sync(0xFFFFFFFFu, first_half);
  in_both = __reduce_add_sync(0xFFFFFFFFu, in_both);
  if (lane == 0)
    *plan = Plan{count, prefix, first_half, in_both, end - prefix - first_half - in_both, s0, s1, pre_lo, one_lo, one_hi};
  __syncwarp();
  return max(end, 1);
}

// As walk_next, by the warp that makes the plans: the count comes with the plan, which serves all heads of a row tile.
template <int kRows, int kKeys>
__device__ __forceinline__ bool walk_next_planned(SharedWalk<kRows, kKeys>* w, Plan* plan, int4* seg) {
  const int lane = threadIdx.x & 31;
  while (true) {
    __syncwarp();
    int s = 0;
    if (lane == 0) s = w->step();
    s = __shfl_sync(0xFFFFFFFFu, s, 0);
    __syncwarp();
    if (s != 0) return s > 0;
    int lo = 0;
    if (w->window > 0) {
      w->own_tiles(w->it.b, w->it.tile, w->it.n, lane, 32, lo);
      lo = __reduce_min_sync(0xFFFFFFFFu, lo);
    }
    if (lane == 0) w->it.lo = lo;
    __syncwarp();
    const int tiles = make_plan<kKeys>(w, plan, seg);
    if (lane == 0) w->nk = tiles;
  }
}

// The v-th tile that is taken, counted in the order of the segments.
__host__ __device__ __forceinline__ int in_turn(const Plan* plan, int v) {
  int u = v - plan->prefix;
  const int n0 = plan->half0, n1 = plan->half1, both = plan->both;
  if (u < 0 || n0 + n1 == 0) return v;  // (an item that sees nothing has a tile all the same, which is in no segment)
  if (u < both) return plan->prefix + n0 + u;
  u -= both;
  const int n = n0 + n1;
  const auto first_of = [&](int k) { return static_cast<int>((static_cast<long long>(k) * n0 + n - 1) / n); };  // among the first k
  const int before = first_of(u);
  return plan->prefix + (first_of(u + 1) > before ? before : n0 + both + u - before);
}

// Key tile v of the stream: its segment (or -1), the position of its first key.
template <int kKeys>
__host__ __device__ __forceinline__ int seg_of(const int4* seg, int count, int v, int& key0) {
  int lo = 0, hi = count;  // the first segment that ends behind v
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (seg[mid].x <= v)
      lo = mid + 1;
    else
      hi = mid;
  }
  if (lo == count) return -1;
  const int4 s = seg[lo];
  key0 = (s.y + v - (lo > 0 ? seg[lo - 1].x : 0)) * kKeys;
  return lo;
}

// Stage bookkeeping of the prefill kernel's copy warp over such a stream, as load_segs: lane l holds page (page0 + l) of the
// stream, per_tile to a tile.  Of the lane's tile: its first key, the end of what is seen, the sequence or -1, and what all rows see.
// Which query tiles it concerns (bits 0 and 1): see the kernel.
struct SharedSegs {
  int key0 = 0, end = 0, seq = -1, all_lo = 0, all_hi = 0, parts = 1;
};
template <int kKeys, class W>
__device__ __forceinline__ SegBatch load_shared_segs(const AttArgs& a, const W& w, const Plan* plan, const int4* seg, int page0,
                                                     int per_tile, SharedSegs& x) {
  const Item& it = w.it;
  SegBatch s;
  s.seg0 = page0;
  const int at_page = page0 + (threadIdx.x & 31), v = at_page / per_tile;
  x = SharedSegs{};
  const bool narrow = it.rows <= W::kRowsOf / 2;
  if (narrow) x.parts = 1 << (v & 1);
  const int at = v < it.kt1 ? seg_of<kKeys>(seg, plan->count, in_turn(plan, v), x.key0) : -1;
  if (at < 0) return s;
  const int4 sg = seg[at];
  x.end = sg.w;
  x.seq = sg.z;
  x.all_lo = at == 0 ? plan->pre_lo : plan->one_lo;
  x.all_hi = at == 0 ? it.hi : plan->one_hi;
  if (!narrow) {
    x.parts = 3;
    if (at > 0) {  // the rows of the sequence's tokens
      const int64_t half = it.row0 + W::kRowsOf / 2;
      x.parts = (static_cast<int64_t>(w.cu[sg.z] - it.tok0) * a.group < half ? 1 : 0) |
                (static_cast<int64_t>(w.cu[sg.z + 1] - it.tok0) * a.group > half ? 2 : 0);
    }
  }
  // positions before a window may have no page any more, those of the prefix none in this sequence's table
  int own_lo = at == 0 ? it.lo : it.hi;
  if (a.window > 0 && at > 0) {
    int own_hi;
    w.own_range(sg.z, it.tok0 + a.token_of(it.row0), it.tok0 + a.token_of(it.row0 + it.rows - 1), it.hi, own_lo, own_hi);
  }
  const int key = x.key0 + (at_page - v * per_tile) * a.c.page;
  if (key < sg.w && key + a.c.page > own_lo) {
    const int page = a.b.pages[static_cast<int64_t>(at == 0 ? it.kv : sg.z) * a.b.max_pages + key / a.c.page];
    if (page >= 0 && page < a.c.n_pages) {
      s.page = page;
      const int64_t ph = static_cast<int64_t>(page) * a.c.heads + it.head;
      s.ek = min(max(static_cast<int>(a.c.k_exp[ph]), kKvMinExp), kKvMaxExp);
      s.ev = min(max(static_cast<int>(a.c.v_exp[ph]), kKvMinExp), kKvMaxExp);
    } else {
      atomicOr(a.err, kErrInvalid);
    }
  }
  return s;
}

// What a query row sees: its own sequence, positions [low, lim), and from base on what its tree word says.
struct RowSight {
  int seq, low, lim, base;
};
template <class W>
__device__ __forceinline__ RowSight row_sight(const W* w, int token, int s0, int s1) {
  const int s = w->seq_of(token, s0, s1), n = w->cu[s + 1] - w->cu[s], i = token - w->cu[s], kv = w->kv[s], base = kv - n;
  return RowSight{s, window_start(base + i, w->window), w->tree ? kv : min(max(base + i + 1, 0), kv), base};
}

}  // namespace att
}  // namespace qspec
