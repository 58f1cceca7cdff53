// Attention for many query rows per key head (prompt chunks, wide trees) on the tcgen05 tensor cores.
//
// A CTA owns an item of 256 rows as two tiles X = 0, 1 of 128, and streams 128 keys at a time:
//   S_X = Q_X K^T (both from shared memory), P_X = 2^(S_X c + ev - m) by one thread per row, O_X += P_X V
// with S, P and O in TMEM (S 2 x 128 columns, P over the S it came from, O 2 x D).  The two tiles alternate
// on the tensor core, PV_0 S_0' PV_1 S_1', so that the softmax of one tile runs under the products of the other.
//  * The cache's codes arrive by bulk copies in a ring of raw tiles; six warps turn them into fp16 (exact) in
//    the 128-byte swizzled layout.  Keys are read along channels (K-major); the same layout of the values is
//    read along tokens (N-major B operand), so nothing is transposed.  Their lane mapping (two keys, opposite
//    halves of the channels per quarter warp) keeps loads and stores free of bank conflicts.
//  * Scales as in the decode kernel: 2^ek on the scores, 2^ev in the exponent, l = sum P 2^-ev.
//  * m, set 2^8 below the largest score, moves only when a score exceeds it by 2^15; then the row's O is rescaled in TMEM (S of a tile is
//    complete only after the tile's last PV, so O is at rest).
//  * What bounds a tile is the time from its scores to its P, about 1900 cycles, and back to the next scores
//    (PV and S of the tile, about 1500): the other tile's products cover about 1000 of them.  A thread holds its
//    row's 128 scores in registers, taken from the other roles' share, and issues the exponentials, which run on a
//    pipe of their own, between the packing and summing of earlier ones.  (Two threads to a row, 64 scores
//    each, had no registers for that: 372 to 441 us against 372 for 4096 new tokens over 8192 positions, 32 heads;
//    reading the scores from TMEM twice, 387.)
//  * One lane issues all MMAs.  An MMA runs 64 cycles; with descriptors built in a diverged lane it took 110 to
//    150 to issue one and the whole kernel 556 us, so the issuing warp stays converged and only its MMAs are elected.
// Warps: 0-7 softmax, 8 copies, 9 MMA issue, 10-15 converters.  Stages change hands by mbarriers; every wait is
// bounded and ends the CTA in order (kErrTimeout) when it runs out.
#pragma once

#include "kv_shared.cuh"

namespace qspec {
namespace att {

// Per 16 keys of a tile: the keys' scale, the values' exponent, its inverse scale, whether there are keys at all.
struct TileMeta {
  float4 group[8];
  // [0]: all eight groups have keys; kShared: and, 2, all rows see all keys, 4 and 8, the query tiles that take part; first key,
  // end, sequence or -1
  int whole[4];
};

template <int D>
struct PrefillCfg {
  static constexpr int kRows = 256, kKeys = 128;
  static constexpr int kSoftmax = 8, kCopy = 8, kMma = 9, kConv0 = 10, kConvs = 6;  // warps
  static constexpr int kThreads = 16 * 32;
  // Registers of 512 threads x 128: the softmax holds 128 scores a thread and takes part of the others' share.
  static constexpr int kRegsSoftmax = 184, kRegsOther = 72;
  static constexpr int kRaw = kKeys * D;          // one side of a tile, codes
  static constexpr int kConv = kKeys * D * 2;     // the same in fp16
  static constexpr int kHalves = D / 64;          // 128-byte wide sub-tiles
  static constexpr int kQ = 128 * D * 2;          // one tile of queries
  static constexpr int kNR = 3 * (128 / D), kNC = 3, kMeta = 8;
  static constexpr int kTiles = 1024 + 2 * kQ + kNC * kConv + kNR * kRaw, kState = 6144;
  static constexpr int kSmem = kTiles + kState;
  // kShared: a plan of the item's stream, its segments, and what each row sees.  The state as it is, as 512 groups just fit.
  using SW = SharedWalk<kRows, kKeys>;
  static constexpr int kBars = 2 * kNR + 2 * kNC + 2 * kMeta + 9;
  static constexpr int kSharedState = static_cast<int>(sizeof(TileMeta) * kMeta + 8 * kBars + sizeof(ScanShared) + 16 + 16 * sizeof(SW));
  static constexpr int kPlan = static_cast<int>(sizeof(Plan) + 8 + sizeof(int4) * (kRows + 1) + sizeof(RowSight) * kRows);
  static constexpr int kSmemShared = kTiles + kSharedState + kPlan;
  static_assert(kSharedState <= kState && kSmemShared + sizeof(int2) * (QSPEC_KV_MAX_GROUPS + 1) <= 227 * 1024, "shared memory");
};

// kShared: adds the parts of the items that runs have cut.  A CTA to an item (that begins in run blockIdx.x) and kMergeSplit of its
// channels, a thread to a row: few items are cut into many parts here, and one SM reads at 125 GB/s (added by the last CTA to
// arrive, ten parts of 256 rows took 27 us; by groups, the code alone slowed the softmax down by a tenth).
constexpr int kMergeSplit = 8;
template <int D>
__global__ void __launch_bounds__(PrefillCfg<D>::kRows) merge_kernel(const AttArgs a) {
  constexpr int kRows = PrefillCfg<D>::kRows, kSlot = kRows * (D + 2), kQuads = D / 4 / kMergeSplit;  // of four channels
  ptx::grid_launch_dependents();
  ptx::grid_dependency_wait();
  const CutItem it = a.cuts[blockIdx.x];
  const int r = threadIdx.x, c0 = blockIdx.x, q0 = blockIdx.y * kQuads;
  if (r >= it.rows || it.parts == 0) return;
  auto part = [&](int k) { return a.partial + (static_cast<int64_t>(c0 + k) * 2 + (k == 0 ? 1 : 0)) * kSlot; };
  float mm = kNoMax, ll = 0.0f;
#pragma unroll 8
  for (int k = 0; k < it.parts; ++k) mm = fmaxf(mm, __ldcg(part(k) + kRows * D + 2 * r));
  float4 acc[kQuads];
#pragma unroll
  for (int e = 0; e < kQuads; ++e) acc[e] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
  for (int k = 0; k < it.parts; ++k) {
    const float* p = part(k);
    const float2 x = __ldcg(reinterpret_cast<const float2*>(p + kRows * D + 2 * r));
    const float f = ex2(x.x - mm);
    ll = fmaf(x.y, f, ll);
#pragma unroll
    for (int e = 0; e < kQuads; ++e) {
      const float4 v = __ldcg(reinterpret_cast<const float4*>(p + ((q0 + e) * kRows + r) * 4));
      acc[e].x = fmaf(v.x, f, acc[e].x);
      acc[e].y = fmaf(v.y, f, acc[e].y);
      acc[e].z = fmaf(v.z, f, acc[e].z);
      acc[e].w = fmaf(v.w, f, acc[e].w);
    }
  }
  const float inv = ll == 0.0f ? 0.0f : 1.0f / ll;
  const int tk = a.token_of(it.row0 + r), hq = it.head * a.group + it.row0 + r - tk * a.group;
  uint16_t* op = a.out + static_cast<int64_t>(it.tok0 + tk) * a.out_token + static_cast<int64_t>(hq) * D + 4 * q0;
#pragma unroll
  for (int e = 0; e < kQuads; ++e)
    *reinterpret_cast<uint2*>(op + 4 * e) = make_uint2(pack_bf16(acc[e].x * inv, acc[e].y * inv), pack_bf16(acc[e].z * inv, acc[e].w * inv));
  if (a.lse && blockIdx.y == 0)
    a.lse[static_cast<int64_t>(it.tok0 + tk) * a.heads_q + hq] = ll == 0.0f ? -INFINITY : (mm + log2f(ll)) * 0.693147180559945f;
}

// Side i of an item of T tiles in that order: its tile, and whether it is the values.
struct SideAt {
  int tile, v;
};
__device__ __forceinline__ SideAt side_at(int i, int T) {
  const bool last = i == 2 * T - 1, keys = i == 0 || ((i & 1) && !last);
  return SideAt{last ? T - 1 : keys ? (i + 1) / 2 : i / 2 - 1, keys ? 0 : 1};
}
__device__ __forceinline__ int side_of_values(int tile, int T) { return tile == T - 1 ? 2 * T - 1 : 2 * tile + 2; }

// kBigPages: pages of 64 slots or more, so 64 keys lie in one page and share its scales.
// kShared: items of groups that share a prefix (kv_shared.cuh).  The copy warp alone knows the stream; what the others need of
// a tile stands in its TileMeta.  A key tile need not concern both query tiles: one of a sequence's own keys goes to the query tile that
// has its rows, and items of up to 128 rows have their rows in both and take key tiles in turn, so that here as well the
// softmax of one runs under the products of the other (the two sums meet in shared memory at the end).  The converted sides come in
// the order K0 K1 V0 K2 V1 ...: with the values of a tile right behind its keys they held one of the three places for as long as its
// softmax took, and the next keys' conversion stood open (16 groups of 32 single tokens over 6001 + 300 positions: 337 us).
// 64 samples over 32768 + 512 positions, 64 heads on 8: 113 us; 128 sequences of four tokens under three prompts of 16384 with up to 2000
// of their own, 32 heads on 8: 198 (as single sequences 575 and 397).  A prefix tile of 256 rows takes 4100 cycles, 64% of the
// measured bf16 rate (two softmax steps of 64 keys, 2000 cycles a query tile, with the waits around them); a tile of a
// sequence's own keys, or of an item of up to 128 rows, takes as long as the converters need for its two sides, 2400.
template <int D, bool kBigPages, bool kShared = false>
__global__ void __launch_bounds__(PrefillCfg<D>::kThreads, 1) prefill_kernel(const AttArgs a) {
  using C = PrefillCfg<D>;
  using W = typename WalkOf<kShared, C::kRows, C::kKeys>::type;
  using namespace ptx;
  constexpr int kRows = C::kRows, kKeys = C::kKeys, kNR = C::kNR, kNC = C::kNC, kMeta = C::kMeta;
  constexpr int kSub = kKeys * 128;  // bytes of a sub-tile: 128 rows of 128 bytes
  constexpr uint32_t kOCol = 256, kCols = 512;
  // kShared: a warp for the products of each query tile
  constexpr int kMmas = kShared ? 2 : 1, kConv0 = C::kConv0 + kMmas - 1, kConvs = C::kConvs - kMmas + 1;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* qs = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* conv = qs + 2 * C::kQ;
  uint8_t* raw = conv + kNC * C::kConv;
  TileMeta* meta = reinterpret_cast<TileMeta*>(raw + kNR * C::kRaw);
  uint64_t* rawfull = reinterpret_cast<uint64_t*>(meta + kMeta);
  uint64_t* rawempty = rawfull + kNR;
  uint64_t* convfull = rawempty + kNR;
  uint64_t* convempty = convfull + kNC;
  uint64_t* metafull = convempty + kNC;
  uint64_t* sfull = metafull + kMeta;  // [2]
  uint64_t* pfull = sfull + 2;         // [2]
  uint64_t* qfull = pfull + 2;
  uint64_t* odone = qfull + 1;
  uint64_t* ofree = odone + 1;
  uint64_t* metaempty = ofree + 1;     // [kMeta], kShared alone
  uint64_t* drain = metaempty + kMeta;  // [2]
  ScanShared* scan = reinterpret_cast<ScanShared*>(metaempty + (kShared ? kMeta + 2 : 0));
  volatile int* flags = reinterpret_cast<volatile int*>(scan + 1);  // abort, last to arrive, abort as the item ended
  uint32_t* tmem_base = reinterpret_cast<uint32_t*>(scan + 1) + 3;
  W* walks = reinterpret_cast<W*>(reinterpret_cast<int2*>(scan + 1) + 2);  // [16]
  Plan* plan = reinterpret_cast<Plan*>(walks + 16);  // (the copy warp's)
  int4* seg = reinterpret_cast<int4*>((reinterpret_cast<uintptr_t>(plan + 1) + 15) & ~uintptr_t(15));
  RowSight* row_sees = reinterpret_cast<RowSight*>(seg + kRows + 1);
  int2* seq = kShared ? reinterpret_cast<int2*>(row_sees + kRows) : reinterpret_cast<int2*>(walks + 16);
  volatile int* abort_flag = flags;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kNR; ++i) {
      mbar_init(rawfull + i, 1);
      mbar_init(rawempty + i, kConvs);
    }
    for (int i = 0; i < kNC; ++i) {
      mbar_init(convfull + i, kConvs);
      mbar_init(convempty + i, kMmas);
    }
    for (int i = 0; i < kMeta; ++i) mbar_init(metafull + i, 1);
    if (kShared) {
      for (int i = 0; i < kMeta; ++i) mbar_init(metaempty + i, C::kSoftmax);
      mbar_init(drain, 1);
      mbar_init(drain + 1, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(sfull + i, 1);
      mbar_init(pfull + i, 4);
    }
    mbar_init(qfull, 8);
    mbar_init(odone, kMmas);
    mbar_init(ofree, 8);
    flags[0] = 0;
    fence_mbar_init();
  }
  if (warp == C::kMma) {
    tmem_alloc(tmem_base, kCols);
    tmem_relinquish();
  }
  grid_launch_dependents();
  grid_dependency_wait();
  if (kShared && threadIdx.x == 0) a.cuts[blockIdx.x].parts = 0;
  tc_fence_before();
  W* walk = walks + warp;  // (in shared memory: its state would cost every role 40 registers)
  long long run0, run1;
  {
    W w;
    if constexpr (kShared)
      share_out<C::kThreads>(a, seq, scan, w, reinterpret_cast<Count*>(qs));
    else
      share_out<C::kThreads>(a, seq, scan, w);  // (barriers inside)
    run0 = w.u;
    run1 = w.u1;
    if (lane == 0) *walk = w;
    __syncwarp();
  }
  tc_fence_after();
  const uint32_t tmem = *tmem_base;

  static_assert(2 * C::kRegsSoftmax + 2 * C::kRegsOther <= 4 * 128, "registers of the launch");
  if (warp < C::kSoftmax) {
    reg_take<C::kRegsSoftmax>();
    // ------------------------------------------------------------------ softmax: thread = row
    const int X = warp >> 2;
    int row = threadIdx.x;  // of the item
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + lane_base + X * 128, to = tmem + lane_base + kOCol + X * D;
    // The warp's 32 rows of the queries' shared memory, reached row by row (lane = row) or with D / 8 lanes to a
    // row (kPer rows at a time); a row's 16-byte chunks are swizzled as its MMA operand wants them.
    constexpr int kChunks = D / 8, kPer = 32 / kChunks, kSteps = 32 / kPer;
    uint8_t* const q_rows = qs + X * C::kQ + (warp & 3) * 32 * 128;
    auto chunk_at = [&](int r, int k) { return q_rows + (k >> 3) * kSub + r * 128 + (((k & 7) ^ (r & 7)) << 4); };
    const int my_chunk = lane % kChunks, my_row = lane / kChunks;
    int t = 0;
    uint32_t item = 0, ns = 0;
    bool ok = true;
    while (walk_next(walk)) {
      const Item& it = walk->it;
      const int kt0 = it.kt0, tiles = it.kt1 - it.kt0;
      const bool narrow = kShared && it.rows <= 128;  // the rows are in both query tiles
      const int warp_row = narrow ? (warp & 3) * 32 : warp * 32;
      if (kShared) row = warp_row + lane;
      const bool active = narrow || X * 128 < it.rows, there = row < it.rows;
      // ---- queries: coalesced, largest value of each row to 2^14; fp16 then holds all bits of bf16
      uint32_t amax = 0;  // of the thread's row
      if (active) {
        const uint16_t* qp = a.q + static_cast<int64_t>(it.tok0) * a.q_token + static_cast<int64_t>(it.head) * a.group * D + 8 * my_chunk;
        int tk = a.token_of(it.row0 + warp_row + my_row), in_group = it.row0 + warp_row + my_row - tk * a.group;
#pragma unroll 1
        for (int i0 = 0; i0 < kSteps; i0 += 8) {  // (8 loads in flight; rolled, as cold code costs its fetch)
          uint4 w[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const bool real = warp_row + (i0 + i) * kPer + my_row < it.rows;
            w[i] = real ? *reinterpret_cast<const uint4*>(qp + tk * a.q_token + in_group * D) : make_uint4(0, 0, 0, 0);
            in_group += kPer;
            while (in_group >= a.group) {
              in_group -= a.group;
              ++tk;
            }
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint32_t v[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
            const uint32_t pair = __vmaxu2(__vmaxu2(v[0] & 0x7FFF7FFFu, v[1] & 0x7FFF7FFFu), __vmaxu2(v[2] & 0x7FFF7FFFu, v[3] & 0x7FFF7FFFu));
            uint32_t top = max(pair & 0xFFFFu, pair >> 16);
#pragma unroll
            for (int off = kChunks / 2; off >= 1; off >>= 1) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, off));
            const uint32_t got = __shfl_sync(0xFFFFFFFFu, top, (lane % kPer) * kChunks);
            if (lane / kPer == i0 + i) amax = got;
            const bool bad = top >= 0x7F80u;
            const float shrink = copysignf(row_shrink(top), a.scale_log2);
            uint32_t f[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) f[e] = bad ? 0u : pack_f16(bf16_lo(v[e]) * shrink, bf16_hi(v[e]) * shrink);
            *reinterpret_cast<uint4*>(chunk_at((i0 + i) * kPer + my_row, my_chunk)) = make_uint4(f[0], f[1], f[2], f[3]);
          }
        }
      }
      const bool odd = amax >= 0x7F80u;  // the row has a NaN or an infinity
      const float mult = row_mult(amax, fabsf(a.scale_log2));
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(qfull);
      int all_lo = 0, all_hi = 0;  // positions that every row of the item sees
      if constexpr (kShared) {
        const int token = a.token_of(it.row0 + (there ? row : 0));
        row_sees[threadIdx.x] = row_sight(walk, it.tok0 + token, walk->grp[it.b].x, walk->grp[it.b + 1].x);  // (its own thread reads it)
      } else {
        const int i0 = a.token_of(it.row0), i1 = a.token_of(it.row0 + it.rows - 1), base = it.kv - it.n;
        all_hi = a.tree ? max(base, 0) : min(max(base + i0 + 1, 0), it.kv);
        all_lo = window_start(base + i1, a.window);
      }
      // What a row sees, taken up anew for each tile with masks (few have any, and registers are short), and which of 16
      // keys from key j0 on that is (bit e: key j0 + e).
      struct Sight {
        int base, lim, low;
        unsigned long long bits;
      };
      auto sight = [&]() {
        Sight v;
        const int token = a.token_of(it.row0 + (row < it.rows ? row : 0));
        v.base = it.kv - it.n;
        v.lim = a.tree ? it.kv : min(max(v.base + token + 1, 0), it.kv);
        v.low = window_start(v.base + token, a.window);
        v.bits = a.tree && row < it.rows ? a.tree[it.tok0 + token] : 0ull;
        return v;
      };
      auto sees = [&](const Sight& v, int j0, float keys) {
        uint32_t see = 0xFFFFu;
        if (v.lim - j0 < 16) see = v.lim > j0 ? (1u << (v.lim - j0)) - 1u : 0u;
        if (v.low > j0) see = v.low - j0 < 16 ? see & ~((1u << (v.low - j0)) - 1u) : 0u;
        if (a.tree && j0 + 16 > v.base) {  // from base on as the tree's word says
          const int d = j0 - v.base;
          see &= d >= 64 ? 0u : d >= 0 ? static_cast<uint32_t>(v.bits >> d) : static_cast<uint32_t>(v.bits << -d) | ((1u << -d) - 1u);
        }
        return keys != 0.0f ? see : 0u;
      };
      constexpr int kBlockGroups = kBigPages ? 1 : 4;  // kShared: of 64 keys, groups with scales of their own
      float m = kNoMax, l = 0.0f;
      bool far = false;  // a reference of the warp's rows is so large that its rounding matters in an exponent
      bool begun = false;  // kShared: a key tile concerned this query tile
      if (active) {
        for (int n = 0; n < tiles; ++n) {
          const int tt = t + n;
          ok = ok && wait_bar(metafull + tt % kMeta, (tt / kMeta) & 1, abort_flag, a.err);
          const TileMeta& md = meta[tt % kMeta];
          // (Lanes can leave a wait differently when another warp gives up, and the branch below has a warp barrier: they agree
          // first.  64 samples over 32768 + 512 positions 111.4 -> 113.0 us.)
          if (kShared) {
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (!ok) break;
          }
          if (kShared && (md.whole[0] >> 2 >> X & 1) == 0) {
            __syncwarp();
            if (lane == 0) mbar_arrive(metaempty + tt % kMeta);
            continue;
          }
          // what the groups of keys bring, read ahead of the scores: factor, exponent, inverse scale
          constexpr int kGroups = kBigPages ? 2 : 8, kPairs = 64 / kGroups;  // groups with scales of their own, pairs of keys in each
          float gm[kGroups], ge[kGroups], gu[kGroups];
#pragma unroll
          for (int g = 0; g < kGroups; ++g) {
            const float4 v = md.group[g * 8 / kGroups];
            gm[g] = fminf(mult * v.x, 3e38f);
            ge[g] = v.y;
            gu[g] = v.z;
          }
          const bool whole_tile = (md.whole[0] & 1) != 0;
          ok = ok && wait_bar(sfull + X, ns & 1, abort_flag, a.err);
          ok = __all_sync(0xFFFFFFFFu, ok);
          if (!ok) break;
          ++ns;
          tc_fence_after();
          const int key0 = kShared ? md.whole[1] : (kt0 + n) * kKeys;
          const bool plain = kShared ? (md.whole[0] & 3) == 3 : key0 + kKeys <= all_hi && key0 >= all_lo && whole_tile;
          float top = -INFINITY;
          float s[4][32];
          // kShared: the warp's rows see none of the tile; the positions that the row sees, and from where on its tree word tells
          bool nothing = false;
          int low = 0, lim = 0x7FFFFFFF, tree_from = 0x7FFFFFFF;
          if (kShared && !plain) {
            const int own = md.whole[3];
            const RowSight r = row_sees[threadIdx.x];
            nothing = !__any_sync(0xFFFFFFFFu, own < 0 || own == r.seq);
            if (a.tree) tree_from = r.base;
            lim = own < 0 ? md.whole[2] : own == r.seq ? r.lim : 0;
            low = own < 0 ? r.low : max(r.low, it.hi);
          }
          if constexpr (kShared) {
            // Two rolled steps of 64 keys, once for the maximum and once for the exponentials: a score is read from TMEM twice, but
            // the code is a fifth as long.  Here the warps do not run in step (a tile concerns one query tile, or a warp of it), and
            // the code of 128 scores in registers came from memory for each: 2000 cycles a tile where all warps run it
            // together, 3700 to 4800 where four or one do.  Rows see all of 64 keys or none of them but where their range begins or
            // ends; scores that are hidden there go back to TMEM as -inf.  (By integer operations on words of 32 keys; by a general
            // mask for each score a tile took 6000 cycles.)
            if (!nothing) {
#pragma unroll 1
              for (int b = 0; b < 2; ++b) {
                float sb[2][32];
                tmem_ld32(ts + 64 * b, sb[0]);
                tmem_ld32(ts + 64 * b + 32, sb[1]);
                tmem_wait_ld();
                const int first = low - (key0 + 64 * b), end = lim - (key0 + 64 * b);
                const bool seen = end > 0 && first < 64;
                if (!__all_sync(0xFFFFFFFFu, !seen || (first <= 0 && end >= 64 && tree_from >= key0 + 64 * b + 64))) {
#pragma unroll
                  for (int w = 0; w < 2; ++w) {
                    const int f = first - 32 * w, n = end - 32 * w;
                    uint32_t see = n >= 32 ? 0xFFFFFFFFu : n <= 0 ? 0u : (1u << n) - 1u;
                    if (f > 0) see &= f >= 32 ? 0u : ~((1u << f) - 1u);
                    const int d = key0 + 64 * b + 32 * w - tree_from;
                    if (d > -32) {
                      const unsigned long long bits = there ? a.tree[it.tok0 + a.token_of(it.row0 + row)] : 0ull;
                      see &= d >= 64 ? 0u : d >= 0 ? static_cast<uint32_t>(bits >> d) : static_cast<uint32_t>(bits << -d) | ((1u << -d) - 1u);
                    }
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                      const int keep = static_cast<int>(see << (31 - e)) >> 31;
                      sb[w][e] = __int_as_float((__float_as_int(sb[w][e]) & keep) | (static_cast<int>(0xFF800000u) & ~keep));
                    }
                    tmem_st32(ts + 64 * b + 32 * w, sb[w]);
                  }
                  tmem_wait_st();
                }
#pragma unroll
                for (int g = 0; g < kBlockGroups; ++g) {
                  const float4 gv = md.group[4 * b + g];
                  constexpr int kEach = 64 / kBlockGroups;
                  auto at = [&](int e) { return sb[(kEach * g + e) / 32][(kEach * g + e) % 32]; };
                  float x = at(0), y = at(1);
#pragma unroll
                  for (int e = 2; e < kEach - 2; e += 4) {
                    x = max3(x, at(e), at(e + 1));
                    y = max3(y, at(e + 2), at(e + 3));
                  }
                  x = max3(x, at(kEach - 2), at(kEach - 1));
                  if (seen) top = fmaxf(top, fmaf(fmaxf(x, y), fminf(mult * gv.x, 3e38f), gv.y));  // (-inf times 0 is no maximum)
                }
              }
            }
          }
          if (kShared) {
          } else if (plain) {
            tmem_ld32(ts, s[0]);
            tmem_ld32(ts + 32, s[1]);
            tmem_wait_ld();
            tmem_ld32(ts + 64, s[2]);
            tmem_ld32(ts + 96, s[3]);
            float x = -INFINITY;
#pragma unroll
            for (int g = 0; g < 8; ++g) {
              if (g == 4) tmem_wait_ld();
              const float* sg = s[g >> 1] + 16 * (g & 1);
              float y = max3(sg[0], sg[1], sg[2]);
              x = max3(x, sg[3], sg[4]);
#pragma unroll
              for (int e = 5; e < 13; e += 4) {
                y = max3(y, sg[e], sg[e + 1]);
                x = max3(x, sg[e + 2], sg[e + 3]);
              }
              y = max3(y, sg[13], sg[14]);
              x = max3(x, y, sg[15]);
              if (!kBigPages || g % 4 == 3) {
                top = fmaxf(top, fmaf(x, gm[g * kGroups / 8], ge[g * kGroups / 8]));
                x = -INFINITY;
              }
            }
          } else {
            const Sight v = sight();
#pragma unroll 1
            for (int g = 0; g < 8; ++g) {
              float sg[16];
              tmem_ld16(ts + g * 16, reinterpret_cast<uint32_t*>(sg));
              tmem_wait_ld();
              const float4 gv = md.group[g];
              const uint32_t see = sees(v, key0 + 16 * g, gv.w);
              float x = -INFINITY;
#pragma unroll
              for (int e = 0; e < 16; ++e)
                if (see >> e & 1u) x = fmaxf(x, sg[e]);
              // (-inf times a factor 0 would be NaN: a group that the row does not see stays out)
              if (see) top = fmaxf(top, fmaf(x, fminf(mult * gv.x, 3e38f), gv.y));
            }
          }
          if (__any_sync(0xFFFFFFFFu, top - m > kSlack)) {  // (a sum m + kSlack would round)
            const float m1 = fmaxf(m, reference_of(top));
            const float keep = ex2(m - m1);
            m = m1;
            l *= keep;
            // (kShared: rows that have seen nothing yet are no such rows)
            far = __any_sync(0xFFFFFFFFu, fabsf(m) > kFar && !(kShared && m == kNoMax));
            if (kShared ? begun : n > 0) {
#pragma unroll 1
              for (int c = 0; c < D; c += 16) {
                uint32_t o[16];
                tmem_ld16(to + c, o);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * keep);
                tmem_st16(to + c, o);
              }
            }
          }
          if (nothing) {
            const uint32_t zero[16] = {};
#pragma unroll
            for (int f = 0; f < 4; ++f) tmem_st16(ts + f * 16, zero);
          } else if (kShared) {
            if (far) {  // scores in powers of two, rounded as their maximum was, take the products' place
#pragma unroll 1
              for (int g = 0; g < 8; ++g) {
                const float4 gv = md.group[g];
                uint32_t z[16];
                tmem_ld16(ts + 16 * g, z);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 16; ++e) z[e] = __float_as_uint(fmaf(__uint_as_float(z[e]), fmaxf(fminf(mult * gv.x, 3e38f), 1e-37f), gv.y));
                tmem_st16(ts + 16 * g, z);
              }
              tmem_wait_st();
            }
#pragma unroll 1
            for (int b = 0; b < 2; ++b) {
              float sb[2][32];
              tmem_ld32(ts + 64 * b, sb[0]);
              tmem_ld32(ts + 64 * b + 32, sb[1]);
              tmem_wait_ld();
              const bool seen = lim > key0 + 64 * b && low < key0 + 64 * b + 64;
              constexpr int kLag0 = 2, kLag1 = 8, kBlockPairs = 32 / kBlockGroups;
              uint64_t mm = 0, bb = 0, sum = 0;
              uint32_t p[16];
#pragma unroll
              for (int e = 0; e < 32 + kLag1; ++e) {  // as below
                const int x = e - kLag0, f = e - kLag1;
                if (e < 32 && e % kBlockPairs == 0) {
                  const float4 gv = md.group[4 * b + e / kBlockPairs];
                  mm = twice(far ? 1.0f : fmaxf(fminf(mult * gv.x, 3e38f), 1e-37f));  // (-inf times 0 would be NaN)
                  bb = twice(!seen ? -INFINITY : far ? -m : gv.y - m);
                }
                if (e < 32) exponents(sb[e / 16][2 * e % 32], sb[e / 16][2 * e % 32 + 1], mm, bb);
                if (x >= 0 && x < 32) ex2_in_order(sb[x / 16][2 * x % 32]);
                if (f >= 0) {
                  p[f % 16] = pack_and_add(sb[f / 16][2 * f % 32], sb[f / 16][2 * f % 32 + 1], sum);
                  if (f % kBlockPairs == kBlockPairs - 1) {
                    l = fmaf(both(sum), md.group[4 * b + f / kBlockPairs].z, l);
                    sum = 0;
                  }
                }
                if (x >= 0 && x < 32) ex2_in_order(sb[x / 16][2 * x % 32 + 1]);
                if (f >= 0 && f % 16 == 15) tmem_st16(ts + 32 * b + f / 16 * 16, p);
              }
            }
          } else if (plain && !far) {
            // pair e of the row: exponents at step e, exponentials kLag0 pairs later, packed and summed kLag1 pairs later
            constexpr int kLag0 = 2, kLag1 = 8;
            uint64_t mm = 0, bb = 0, sum = 0;
            uint32_t p[16];
#pragma unroll
            for (int e = 0; e < 64 + kLag1; ++e) {
              const int x = e - kLag0, f = e - kLag1;
              if (e < 64 && e % kPairs == 0) {
                mm = twice(gm[e / kPairs]);
                bb = twice(ge[e / kPairs] - m);
              }
              if (e < 64) exponents(s[e / 16][2 * e % 32], s[e / 16][2 * e % 32 + 1], mm, bb);
              if (x >= 0 && x < 64) ex2_in_order(s[x / 16][2 * x % 32]);
              if (f >= 0) {
                p[f % 16] = pack_and_add(s[f / 16][2 * f % 32], s[f / 16][2 * f % 32 + 1], sum);
                if (f % kPairs == kPairs - 1) {
                  l = fmaf(both(sum), gu[f / kPairs], l);
                  sum = 0;
                }
              }
              if (x >= 0 && x < 64) ex2_in_order(s[x / 16][2 * x % 32 + 1]);
              if (f >= 0 && f % 16 == 15) tmem_st16(ts + f / 16 * 16, p);
            }
          } else {
            const Sight v = sight();
#pragma unroll 1
            for (int g = 0; g < 8; ++g) {
              float sg[16];
              tmem_ld16(ts + g * 16, reinterpret_cast<uint32_t*>(sg));
              tmem_wait_ld();
              const float4 gv = md.group[g];
              const uint32_t see = sees(v, key0 + 16 * g, gv.w);
              const float mg = fminf(mult * gv.x, 3e38f);
              float sum = 0.0f;
#pragma unroll
              for (int e = 0; e < 16; ++e) {  // (scores rounded as the maximum was)
                sg[e] = see >> e & 1u ? ex2(fmaf(sg[e], mg, gv.y) - m) : 0.0f;
                sum += sg[e];
              }
              l = fmaf(sum, gv.z, l);
              uint32_t p[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) p[e] = pack_f16(sg[2 * e], sg[2 * e + 1]);
              tmem_st8(ts + g * 8, p);
            }
          }
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(pfull + X);
            if (kShared) mbar_arrive(metaempty + tt % kMeta);
          }
          begun = true;
        }
      }
      t += tiles;
      if (odd && l > 0.0f) l = NAN;
      ok = ok && wait_bar(odone, item & 1, abort_flag, a.err);
      ok = __all_sync(0xFFFFFFFFu, ok);
      if (!ok) *abort_flag = 1;
      ++item;
      tc_fence_after();
      const bool whole = it.ub >= run0 && it.ue <= run1;
      constexpr int kSlot = kRows * (D + 2);
      float* slot = a.partial + (static_cast<int64_t>(blockIdx.x) * 2 + (it.ub >= run0 ? 1 : 0)) * kSlot;
      // Rows in shared memory (the queries are used up) -> out, a row's chunks by neighbouring lanes.
      auto store_rows = [&]() {
        __syncwarp();
        uint16_t* op = a.out + static_cast<int64_t>(it.tok0) * a.out_token + static_cast<int64_t>(it.head) * a.group * D + 8 * my_chunk;
#pragma unroll 4
        for (int i = 0; i < kSteps; ++i) {
          const int r = warp * 32 + i * kPer + my_row, packed = it.row0 + r, tk = a.token_of(packed);
          const uint4 w = *reinterpret_cast<const uint4*>(chunk_at(my_row + i * kPer, my_chunk));
          if (r < it.rows) *reinterpret_cast<uint4*>(op + tk * a.out_token + (packed - tk * a.group) * D) = w;
        }
        __syncwarp();
      };
      // kShared: what the second query tile has of a narrow item's rows, by way of the queries' shared memory
      float* const o_second = reinterpret_cast<float*>(qs);  // [channel / 4][row] of four
      float f_first = 1.0f, f_second = 0.0f;
      if (kShared && narrow) {
        float2* const ml_second = reinterpret_cast<float2*>(row_sees + 128);
        if (X == 1) {
#pragma unroll 1
          for (int c = 0; c < D; c += 32) {
            float o[32];
            __syncwarp();
            tmem_ld32(to + c, o);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 8; ++e)
              *reinterpret_cast<float4*>(o_second + ((c / 4 + e) * 128 + row) * 4) =
                  begun ? make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          }
          ml_second[2 * row] = make_float2(m, l);  // (in the thread's own place)
        }
        named_bar_sync(1, 256);
        if (X == 0) {
          const float2 v = ml_second[2 * row];
          const float mm = fmaxf(m, v.x);
          f_first = begun ? ex2(m - mm) : 0.0f;
          f_second = ex2(v.x - mm);
          l = fmaf(l, f_first, v.y * f_second);
          m = mm;
        }
      }
      if (ok && active && !(kShared && narrow && X == 1)) {
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          float o[32];
          __syncwarp();
          tmem_ld32(to + c, o);
          tmem_wait_ld();
          if (kShared && !begun) {  // (no product was written there)
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = 0.0f;
          }
          if (kShared && narrow) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float4 v = *reinterpret_cast<const float4*>(o_second + ((c / 4 + e) * 128 + row) * 4);
              o[4 * e] = fmaf(o[4 * e], f_first, v.x * f_second);
              o[4 * e + 1] = fmaf(o[4 * e + 1], f_first, v.y * f_second);
              o[4 * e + 2] = fmaf(o[4 * e + 2], f_first, v.z * f_second);
              o[4 * e + 3] = fmaf(o[4 * e + 3], f_first, v.w * f_second);
            }
          }
          if (kShared && narrow && whole) {  // (straight out: the staging place holds the second tile's rows)
            if (there) {
              const int tk = a.token_of(it.row0 + row);
              uint16_t* op = a.out + static_cast<int64_t>(it.tok0 + tk) * a.out_token +
                             static_cast<int64_t>(it.head * a.group + it.row0 + row - tk * a.group) * D + c;
#pragma unroll
              for (int k = 0; k < 4; ++k)
                *reinterpret_cast<uint4*>(op + 8 * k) =
                    make_uint4(pack_bf16(o[8 * k] * inv, o[8 * k + 1] * inv), pack_bf16(o[8 * k + 2] * inv, o[8 * k + 3] * inv),
                               pack_bf16(o[8 * k + 4] * inv, o[8 * k + 5] * inv), pack_bf16(o[8 * k + 6] * inv, o[8 * k + 7] * inv));
            }
          } else if (whole) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              uint32_t w[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) w[e] = pack_bf16(o[8 * k + 2 * e] * inv, o[8 * k + 2 * e + 1] * inv);
              *reinterpret_cast<uint4*>(chunk_at(lane, c / 8 + k)) = make_uint4(w[0], w[1], w[2], w[3]);
            }
          } else if (there) {
#pragma unroll
            for (int e = 0; e < 8; ++e)  // [channel / 4][row]: consecutive rows are consecutive addresses
              *reinterpret_cast<float4*>(slot + ((c / 4 + e) * kRows + row) * 4) = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
          }
        }
        if (whole) {
          if (!(kShared && narrow)) store_rows();
          if (a.lse && there) {
            const int token = a.token_of(it.row0 + row), hq = it.head * a.group + it.row0 + row - token * a.group;
            a.lse[static_cast<int64_t>(it.tok0 + token) * a.heads_q + hq] = l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.693147180559945f;
          }
        } else if (there) {
          *reinterpret_cast<float2*>(slot + kRows * D + 2 * row) = make_float2(m, l);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(ofree);
      if (kShared && !whole && it.ub >= run0 && threadIdx.x == 0)
        a.cuts[blockIdx.x] = CutItem{owner_of(it.ue - 1, scan) - static_cast<int>(blockIdx.x) + 1, it.tok0, it.row0, it.rows, it.head};
      if (!kShared && !whole) {
        const int c0 = owner_of(it.ub, scan), c1 = owner_of(it.ue - 1, scan);
        named_bar_sync(1, 256);
        if (threadIdx.x == 0) {
          const bool last = add_acq_rel(a.tickets + c0, 1u) == static_cast<unsigned int>(c1 - c0);
          if (last) a.tickets[c0] = 0;
          flags[1] = last;
          flags[2] = *abort_flag;  // (one reading for all warps: they leave together)
        }
        named_bar_sync(1, 256);
        if (flags[2]) break;
        if (flags[1]) {
          // all 256 threads add the parts up: `span` threads take the rows (a power of two, so that a warp reads neighbours), as
          // many as fit share the channels of a row
          int span = 32;
          while (span < it.rows) span *= 2;
          const int r = threadIdx.x & (span - 1), c_first = threadIdx.x / span, c_step = 256 / span;
          if (r < it.rows) {
            auto part = [&](int k) { return a.partial + (static_cast<int64_t>(k) * 2 + (k == c0 ? 1 : 0)) * kSlot; };
            float mm = kNoMax, ll = 0.0f;
#pragma unroll 4
            for (int k = c0; k <= c1; ++k) mm = fmaxf(mm, __ldcg(part(k) + kRows * D + 2 * r));
#pragma unroll 4
            for (int k = c0; k <= c1; ++k) {
              const float2 x = __ldcg(reinterpret_cast<const float2*>(part(k) + kRows * D + 2 * r));
              ll = fmaf(x.y, ex2(x.x - mm), ll);
            }
            const float inv = ll == 0.0f ? 0.0f : 1.0f / ll;
            const int tk = a.token_of(it.row0 + r), hq = it.head * a.group + it.row0 + r - tk * a.group;
            uint16_t* op = a.out + static_cast<int64_t>(it.tok0 + tk) * a.out_token + static_cast<int64_t>(hq) * D;
            constexpr int kBatch = 4;  // of four channels
#pragma unroll 1
            for (int c = c_first; c < D / 4; c += kBatch * c_step) {
              float4 acc[kBatch];
#pragma unroll
              for (int e = 0; e < kBatch; ++e) acc[e] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
              for (int k = c0; k <= c1; ++k) {
                const float* p = part(k);
                const float f = ex2(__ldcg(p + kRows * D + 2 * r) - mm);
#pragma unroll
                for (int e = 0; e < kBatch; ++e)
                  if (c + e * c_step < D / 4) {
                    const float4 v = __ldcg(reinterpret_cast<const float4*>(p + ((c + e * c_step) * kRows + r) * 4));
                    acc[e].x = fmaf(v.x, f, acc[e].x);
                    acc[e].y = fmaf(v.y, f, acc[e].y);
                    acc[e].z = fmaf(v.z, f, acc[e].z);
                    acc[e].w = fmaf(v.w, f, acc[e].w);
                  }
              }
#pragma unroll
              for (int e = 0; e < kBatch; ++e)
                if (c + e * c_step < D / 4)
                  *reinterpret_cast<uint2*>(op + 4 * (c + e * c_step)) =
                      make_uint2(pack_bf16(acc[e].x * inv, acc[e].y * inv), pack_bf16(acc[e].z * inv, acc[e].w * inv));
            }
            if (a.lse && c_first == 0)
              a.lse[static_cast<int64_t>(it.tok0 + tk) * a.heads_q + hq] = ll == 0.0f ? -INFINITY : (mm + log2f(ll)) * 0.693147180559945f;
          }
        }
      } else {
        // the flags are taken up again by the next item, in step
        named_bar_sync(1, 256);
        if (threadIdx.x == 0) flags[2] = *abort_flag;
        named_bar_sync(1, 256);
        if (flags[2]) break;
      }
    }
  } else {
    reg_give<C::kRegsOther>();
    if (warp >= kConv0) {
      // ------------------------------------------------------------------ converters
      const int cw = warp - kConv0;
      int i = 0, tile0 = 0;  // sides, and tiles of the items before
      bool ok = true;
      while (ok && walk_next(walk)) {
        const Item& it = walk->it;
        if (kShared && i > 0) tile0 = i / 2;
        for (int kt = it.kt0; ok && kt < it.kt1; ++kt) {
          int kv_in = it.kv - kt * kKeys;  // slots from here on hold anything
          for (int side = 0; side < 2; ++side, ++i) {
            const int st = i % kNR, sc = i % kNC;
            ok = ok && wait_bar(rawfull + st, (i / kNR) & 1, abort_flag, a.err);
            // (kShared: the place is waited for once the codes are in registers)
            if (!kShared && i >= kNC) ok = ok && wait_bar(convempty + sc, ((i / kNC) - 1) & 1, abort_flag, a.err);
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (!ok) break;
            const uint8_t* src = raw + st * C::kRaw;
            uint8_t* dst = conv + sc * C::kConv;
            const TileMeta& md =
                meta[(kShared ? tile0 + side_at(2 * (kt - it.kt0) + side, it.kt1 - it.kt0).tile : i >> 1) % kMeta];
            if (kShared) kv_in = md.whole[2] - md.whole[1];
            // a quarter warp takes two keys; D = 128: the first key's chunks of one half, the second's of the other
            const int quad = lane & 3, sub = (lane >> 2) & 1;
            const bool all = (md.whole[0] & 1) != 0 && kv_in >= kKeys;
            // 16 steps of 8 keys, two or three to a warp; all loads first
            constexpr int kMine = (kKeys / 8 + kConvs - 1) / kConvs;
            uint4 w[kMine][C::kHalves];
#pragma unroll
            for (int n = 0; n < kMine; ++n) {
              const int step = cw + n * kConvs, key = step * 8 + 2 * (lane >> 3) + sub;
              if (n < kMine - 1 || step < kKeys / 8) {
                const bool live = all || (md.group[key >> 4].w != 0.0f && key < kv_in);
#pragma unroll
                for (int h = 0; h < C::kHalves; ++h) {
                  const int half = C::kHalves == 2 ? (h ^ sub) : 0;
                  w[n][h] = live ? *reinterpret_cast<const uint4*>(src + key * D + half * 64 + quad * 16) : make_uint4(0, 0, 0, 0);
                }
              }
            }
            if (kShared) {
              __syncwarp();
              if (lane == 0) mbar_arrive(rawempty + st);
              if (i >= kNC) ok = wait_bar(convempty + sc, ((i / kNC) - 1) & 1, abort_flag, a.err);
              ok = __all_sync(0xFFFFFFFFu, ok);
              if (!ok) break;
            }
#pragma unroll
            for (int n = 0; n < kMine; ++n) {
              const int step = cw + n * kConvs, key = step * 8 + 2 * (lane >> 3) + sub;
              if (n < kMine - 1 || step < kKeys / 8) {
#pragma unroll
                for (int h = 0; h < C::kHalves; ++h) {
                  const int half = C::kHalves == 2 ? (h ^ sub) : 0;
                  const uint4 v = w[n][h];
                  uint8_t* row = dst + half * kSub + key * 128;
                  uint4 x, y;
                  if (kShared) {
                    e4m3x4_to_f16x4(v.x, x.x, x.y);
                    e4m3x4_to_f16x4(v.y, x.z, x.w);
                    e4m3x4_to_f16x4(v.z, y.x, y.y);
                    e4m3x4_to_f16x4(v.w, y.z, y.w);
                  } else {
                    x = make_uint4(e4m3x2_to_f16x2(v.x), e4m3x2_to_f16x2(v.x >> 16), e4m3x2_to_f16x2(v.y), e4m3x2_to_f16x2(v.y >> 16));
                    y = make_uint4(e4m3x2_to_f16x2(v.z), e4m3x2_to_f16x2(v.z >> 16), e4m3x2_to_f16x2(v.w), e4m3x2_to_f16x2(v.w >> 16));
                  }
                  *reinterpret_cast<uint4*>(row + (((2 * quad) ^ (key & 7)) << 4)) = x;
                  *reinterpret_cast<uint4*>(row + (((2 * quad + 1) ^ (key & 7)) << 4)) = y;
                }
              }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              if (!kShared) mbar_arrive(rawempty + st);
              mbar_arrive(convfull + sc);
            }
          }
        }
      }
    } else if (warp == C::kCopy) {
      // ------------------------------------------------------------------ copies
      const int P = a.c.page, per_tile = kKeys / P;
      const uint32_t seg_bytes = P * D;
      int t = 0, issued = 0;
      while (walk_next(walk)) {
        const Item& it = walk->it;
        SegBatch sb;
        if constexpr (kShared) {
          SharedSegs ss;
          make_plan<kKeys>(walk, plan, seg);
          const int T = it.kt1 - it.kt0;
          // of the tile whose keys were last copied and of the one before: the lane's page or none, the pages there are
          int64_t at = 0, at_before = 0;
          uint32_t who = 0, who_before = 0;
          int l0 = 0, l0_before = 0;
          bool ok = true;
          for (int i = 0; i < 2 * T; ++i, ++issued) {
            const SideAt side = side_at(i, T);
            const int st = issued % kNR, tt = t + side.tile;
            if (issued >= kNR) ok = wait_bar(rawempty + st, ((issued / kNR) - 1) & 1, abort_flag, a.err);
            if (side.v == 0 && tt >= kMeta) ok = ok && wait_bar(metaempty + tt % kMeta, ((tt / kMeta) - 1) & 1, abort_flag, a.err);
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (!ok) break;
            if (side.v == 0) {
              const int seg0 = (it.kt0 + side.tile) * per_tile;
              if (sb.seg0 < 0 || seg0 >= sb.seg0 + 32) sb = load_shared_segs<kKeys>(a, *walk, plan, seg, seg0, per_tile, ss);
              at_before = at;
              who_before = who;
              l0_before = l0;
              l0 = seg0 - sb.seg0;
              const bool mine = lane >= l0 && lane < l0 + per_tile && sb.page >= 0;
              who = __ballot_sync(0xFFFFFFFFu, mine);
              at = mine ? (static_cast<int64_t>(sb.page) * a.c.heads + it.head) * seg_bytes : -1;
              TileMeta& md = meta[tt % kMeta];
              if (lane < 8) md.group[lane] = make_float4(0.0f, -INFINITY, 1.0f, 0.0f);  // (no keys: no weight)
              if (lane == l0) {
                md.whole[0] = (__popc(who) != per_tile ? 0 : ss.key0 >= ss.all_lo && ss.key0 + kKeys <= ss.all_hi ? 3 : 1) | ss.parts << 2;
                md.whole[1] = ss.key0;
                md.whole[2] = ss.end;
                md.whole[3] = ss.seq;
              }
              __syncwarp();
              if (mine) {
                const int g0 = (lane - l0) * (P / 16);
                const float4 v = make_float4(exp2_int(sb.ek), static_cast<float>(sb.ev), exp2_int(-sb.ev), 1.0f);
                for (int g = g0; g < g0 + P / 16; ++g) md.group[g] = v;
              }
              __syncwarp();
              if (lane == 0) mbar_arrive(metafull + tt % kMeta);
            }
            // (values of the tile before the one whose keys came last, but for the item's last)
            const bool old = side.v != 0 && i < 2 * T - 1;
            const int64_t from = old ? at_before : at;
            const uint32_t pages = old ? who_before : who;
            if (lane == 0) mbar_arrive_expect_tx(rawfull + st, __popc(pages) * seg_bytes);
            __syncwarp();
            if (pages >> lane & 1u)
              bulk_load(raw + st * C::kRaw + (lane - (old ? l0_before : l0)) * seg_bytes, (side.v ? a.c.v : a.c.k) + from, seg_bytes, rawfull + st);
          }
          t += T;
        } else for (int kt = it.kt0; kt < it.kt1; ++kt, ++t) {
          const int seg0 = kt * per_tile;
          if (sb.seg0 < 0 || seg0 >= sb.seg0 + 32) sb = load_segs(a, it, seg0, P);
          const int l0 = seg0 - sb.seg0;
          const bool mine = lane >= l0 && lane < l0 + per_tile && sb.page >= 0;
          const uint32_t who = __ballot_sync(0xFFFFFFFFu, mine);
          const int64_t at = mine ? (static_cast<int64_t>(sb.page) * a.c.heads + it.head) * seg_bytes : 0;
          bool ok = true;
#pragma unroll
          for (int side = 0; side < 2; ++side) {
            const int i = 2 * t + side, st = i % kNR;
            if (i >= kNR) ok = wait_bar(rawempty + st, ((i / kNR) - 1) & 1, abort_flag, a.err);
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (!ok) break;
            if (side == 0) {
              // tiles up to t - 4 are through the softmax here: the raw slot's last tile was converted, so the
              // converted slot before that was used up by an MMA that followed their PVs
              TileMeta& md = meta[t % kMeta];
              if (lane < 8) md.group[lane] = make_float4(0.0f, 0.0f, 1.0f, 0.0f);
              if (lane == 0) md.whole[0] = __popc(who) == per_tile;
              __syncwarp();
              if (mine) {
                const int g0 = (lane - l0) * (P / 16);
                const float4 v = make_float4(exp2_int(sb.ek), static_cast<float>(sb.ev), exp2_int(-sb.ev), 1.0f);
                for (int g = g0; g < g0 + P / 16; ++g) md.group[g] = v;
              }
              __syncwarp();
              if (lane == 0) mbar_arrive(metafull + t % kMeta);
            }
            if (lane == 0) mbar_arrive_expect_tx(rawfull + st, __popc(who) * seg_bytes);
            ++issued;
            __syncwarp();
            if (mine) bulk_load(raw + st * C::kRaw + (lane - l0) * seg_bytes, (side ? a.c.v : a.c.k) + at, seg_bytes, rawfull + st);
          }
          if (!ok) break;
        }
        if (__any_sync(0xFFFFFFFFu, *abort_flag)) break;
      }
      // nothing may still be copying into shared memory when the CTA exits
      for (int i = issued > kNR ? issued - kNR : 0; i < issued; ++i) wait_bar_final(rawfull + i % kNR, (i / kNR) & 1, a.err);
      __syncwarp();
    } else {
      // ------------------------------------------------------------------ MMA issue
      // One lane feeds the tensor core, so an MMA may cost it at most the 64 cycles that it runs: the warp stays
      // together up to the elected lane's MMAs, which keeps descriptors (bases plus constants) in uniform registers.
      const uint32_t idesc_s = idesc_f16_f32(128, kKeys);
      const uint32_t idesc_o = idesc_f16_f32(128, D) | kIdescBMajorMN;
      const uint64_t q_desc = smem_desc_sw128(smem_u32(qs));
      const uint64_t k_desc = smem_desc_sw128(smem_u32(conv)), v_desc = smem_desc_sw128_mn(smem_u32(conv), kSub);
      const uint32_t tm = __shfl_sync(0xFFFFFFFFu, tmem, 0);
      uint32_t item = 0, np0 = 0, np1 = 0;
      int slot = 0;           // of the next converted side
      uint32_t phase = 0;
      bool ok = true;
      auto wait_all = [&](uint64_t* bar, uint32_t parity) {
        ok = ok && __all_sync(0xFFFFFFFFu, wait_bar(bar, parity, abort_flag, a.err));
        tc_fence_after();
      };
      auto take = [&]() {     // waits for the next converted side; its slot
        const int s = slot;
        wait_all(convfull + s, phase);
        if (++slot == kNC) {
          slot = 0;
          phase ^= 1u;
        }
        return s;
      };
      auto commit = [&](uint64_t* bar) {
        if (elect_one()) mma_commit(bar);
        __syncwarp();
      };
      auto scores = [&](uint32_t X, int s) {
        const uint64_t qd = q_desc + X * (C::kQ >> 4), kd = k_desc + static_cast<uint32_t>(s) * (C::kConv >> 4);
        if (elect_one()) {
#pragma unroll
          for (uint32_t ks = 0; ks < D / 16; ++ks) {
            const uint32_t off = ((ks >> 2) * kSub + (ks & 3) * 32) >> 4;
            mma_f16_ss(tm + X * 128, qd + off, kd + off, idesc_s, ks > 0);
          }
          mma_commit(sfull + X);
        }
        __syncwarp();
      };
      auto values = [&](uint32_t X, int s, bool first) {
        const uint64_t vd = v_desc + static_cast<uint32_t>(s) * (C::kConv >> 4);
        if (elect_one()) {
          mma_bf16_ts(tm + kOCol + X * D, tm + X * 128, vd, idesc_o, first ? 0u : 1u);
#pragma unroll
          for (uint32_t ks = 1; ks < kKeys / 16; ++ks)
            mma_bf16_ts(tm + kOCol + X * D, tm + X * 128 + ks * 8, vd + ((ks * 2048) >> 4), idesc_o, 1u);
        }
        __syncwarp();
      };
      // kShared: a warp to each query tile, so that the steps between a softmax and the next one of the same query tile are the warp's
      // own: some 20 of them at about 200 cycles a tile, as each instruction comes from far while sixteen warps in five roles share the
      // instruction caches.  (One warp for both: 3500 to 5500 cycles a key tile, never waiting for anything.)  The
      // warps go through the converted sides in their order; one that does not concern a query tile is only let go.
      uint32_t side0 = 0, tile0 = 0, turn = 0;
      const uint32_t X = kShared ? __shfl_sync(0xFFFFFFFFu, warp - C::kMma, 0) : 0;
      while (kShared && ok && walk_next(walk)) {
        const int tiles = __shfl_sync(0xFFFFFFFFu, walk->it.kt1 - walk->it.kt0, 0);
        bool begun = false;
        int pend = -1, early = -1;  // the key tile whose scores wait for their values; the one whose values were taken ahead of the next keys
        wait_all(qfull, item & 1);
#pragma unroll 1
        for (int i = 0; ok && i < 2 * tiles; ++i) {
          const SideAt side = side_at(i, tiles);
          if (side.v != 0 && early == side.tile) continue;
          const uint32_t at = side0 + i, slot = at % kNC;
          wait_all(convfull + slot, (at / kNC) & 1);
          if (!ok) break;
          const bool mine = side.v != 0 ? pend == side.tile : (meta[(tile0 + side.tile) % kMeta].whole[0] >> (2 + X) & 1) != 0;
          if (!__any_sync(0xFFFFFFFFu, mine)) {
            if (lane == 0) mbar_arrive(convempty + slot);
            __syncwarp();
            continue;
          }
          if (pend >= 0) {  // the scores' place is taken by weights: they are multiplied first
            const uint32_t v_at = side0 + side_of_values(pend, tiles), v = v_at % kNC;
            wait_all(convfull + v, (v_at / kNC) & 1);
            wait_all(pfull + X, turn & 1);
            if (!begun && item > 0) wait_all(ofree, (item - 1) & 1);
            if (!ok) break;
            values(X, v, !begun);
            commit(convempty + v);
            ++turn;
            begun = true;
            early = side.v != 0 ? -1 : pend;
            pend = -1;
          }
          if (side.v == 0) {
            scores(X, slot);
            commit(convempty + slot);
            pend = side.tile;
          }
        }
        side0 += 2 * tiles;
        tile0 += tiles;
        if (ok) {
          commit(odone);
          ++item;
        }
      }
      while (!kShared && ok && walk_next(walk)) {
        const bool both = __shfl_sync(0xFFFFFFFFu, walk->it.rows, 0) > 128;
        const int tiles = __shfl_sync(0xFFFFFFFFu, walk->it.kt1 - walk->it.kt0, 0);
        wait_all(qfull, item & 1);
        int ks = take(), vs;
        if (!ok) break;
        scores(0, ks);
        if (both) scores(1, ks);
        commit(convempty + ks);
        for (int n = 0; n < tiles; ++n) {
          const bool more = n + 1 < tiles;
          vs = take();
          if (n == 0 && item > 0) wait_all(ofree, (item - 1) & 1);
          wait_all(pfull, np0++ & 1);
          if (!ok) break;
          values(0, vs, n == 0);
          if (!both) commit(convempty + vs);
          if (more) {
            ks = take();
            if (!ok) break;
            scores(0, ks);
          }
          if (both) {
            wait_all(pfull + 1, np1++ & 1);
            if (!ok) break;
            values(1, vs, n == 0);
            commit(convempty + vs);  // (before the scores: a commit waits for all MMAs issued so far)
            if (more) scores(1, ks);
          }
          if (more) commit(convempty + ks);
        }
        if (ok) {
          commit(odone);
          ++item;
        }
      }
      // every MMA issued has finished before the CTA gives its TMEM and shared memory back: odone or, after
      // a wait ran out, one more commit
      if (!ok) {
        if (lane == 0) *abort_flag = 1;
        commit(kShared ? drain + X : odone);
        if (lane == 0) wait_bar_final(kShared ? drain + X : odone, kShared ? 0 : item & 1, a.err);
        __syncwarp();
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == C::kMma) {
    tc_fence_after();
    tmem_dealloc(tmem, kCols);
  }
  // A run given up (the softmax left its walk half way) still arrives wherever it would have: the outputs are void, but
  // the workspace's tickets are back at zero when the call ends.  (Here and not where the softmax leaves: there the
  // walk's registers cost 376 -> 394 us, 4096 tokens over 8192 positions.)
  if (!kShared && *abort_flag && threadIdx.x == 0) {
    const long long c = blockIdx.x, u0 = run_start(c, scan), u1 = run_start(c + 1, scan);
    while (walks->next_cut(u0, u1)) {
      const int c0 = owner_of(walks->it.ub, scan), c1 = owner_of(walks->it.ue - 1, scan);
      if (add_acq_rel(a.tickets + c0, 1u) == static_cast<unsigned int>(c1 - c0)) a.tickets[c0] = 0;
    }
  }
}

}  // namespace att
}  // namespace qspec
