// Attention for few query rows per key head (decode, verify and tree steps): bound by the cache's bytes.
//
// Per 16 keys and 16 rows a warp runs the whole of S = Q K^T, the online softmax and O += P V in
// registers, with mma.sync m16n8k16 (fp16 inputs, fp32 sums): at 16 rows the tensor work of a
// key is 8 KFLOP against 256 bytes of cache, so the legacy tensor path keeps up with HBM, and its register
// fragments let the codes go from shared memory to the MMA with one conversion and no second trip.
//  * The contraction order of an MMA is free, so a thread takes 16 consecutive codes of a key as the k
//    indices of four MMAs (one 16-byte load) with the query fragments laid out to match; and 16 consecutive
//    channels of its four keys as the n index of 16 MMAs, pairs of keys gathered by byte permutes.
//  * Keys' scales multiply the fp32 scores.  Values' scales 2^ev go into the exponent: with
//    z = score + ev and m near max z, P = 2^(z - m) weights the bare codes and l = sum P 2^-ev is the softmax sum,
//    so pages of different scales share one accumulator and fp16 rounds relative to the largest weight.
//  * m is set 8 powers of two below the largest score and moves when a score exceeds it by more than 15 (fp16 has the
//    room on both sides), which one vote per 16 keys decides; the common step has no shuffles.
//  * Every warp streams its own keys: 16 of each tile of 64, three stages of 16-byte asynchronous copies that only
//    the warp itself waits for.  A step is a chain of some 2000 cycles of latency, so the warps on an SM set the
//    rate: 16 of them without a producer or a barrier in the loop, where a ring shared by a CTA (8 consumer
//    warps, bulk copies) reached 59% of the measured bandwidth against 72 to 78% (64 single tokens at 6001 positions, 64
//    heads on 8: 122 against 94 us; one sequence of 131072, 4 tokens: 67 against 55).  The copies place the 16-byte chunks so that
//    the fragment loads are free of bank conflicts (see copy_step).
// With more than 16 rows a second set of four warps takes the next 16 and the two warps of a key group share
// their stages.  Each warp sums its own keys; the sums meet in shared memory once per item.
// kShared: items of groups that share a prefix (kv_shared.cuh).  A key tile's segment decides whose page table it lies in
// and which rows see it.
#pragma once

#include "kv_shared.cuh"

namespace qspec {
namespace att {

template <int D, int RG, bool kShared = false>
struct DecodeCfg {
  static constexpr int kRows = 16 * RG;
  static constexpr int kKeys = 64;
  static constexpr int kThreads = 128 * RG;
  static constexpr int kCtas = 4 / RG;           // resident per SM, at most
  static constexpr int kStages = 3;
  static constexpr int kSide = 16 * D;           // bytes of 16 keys or values
  static constexpr int kRing = 4 * kStages * 2 * kSide;
  static constexpr int kRowPad = D + (D / 32) * 4 * (D == 128 ? 1 : 2);  // floats of a merge row: conflict-free
  static constexpr int kMerge = 4 * RG * 16 * kRowPad * 4;               // takes the ring's place between items
  // the warps' maxima and sums, the walk, the scan, flags
  using W = typename WalkOf<kShared, kRows, kKeys>::type;
  static constexpr int kPlan = kShared ? static_cast<int>(sizeof(Plan) + 8 + sizeof(int4) * (kRows + 1)) : 0;
  static constexpr int kState = 4 * RG * 16 * 8 + sizeof(W) + sizeof(ScanShared) + 16 + kPlan;
  static constexpr int kSmem = 128 + (kRing > kMerge ? kRing : kMerge) + RG * D * 32 + kState;
  // B: sequences, or groups of them
  static constexpr int smem(int B) { return kSmem + static_cast<int>(sizeof(int2)) * (B + 1); }
  // CTAs that an SM's shared memory holds beside each other: with the table of many sequences one less.  (Heads of 128,
  // up to 16 rows: three from 377 sequences on.  A grid of more leaves the rest of its equal runs to a second, mostly
  // empty wave: single tokens over 460000 positions in all, 64 heads on 8, 512 sequences 242 us against 181; 256, where
  // exact sizes let four fit, 220 against 157.)
  static constexpr int ctas(int B) {
    const int fit = kSmemPerSm / ((smem(B) + 127) / 128 * 128 + kSmemReserved);
    return fit < kCtas ? fit : kCtas;
  }
};

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint4& a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}

template <int D, int RG, bool kShared = false>
__global__ void __launch_bounds__(DecodeCfg<D, RG>::kThreads, DecodeCfg<D, RG>::kCtas) decode_kernel(const AttArgs a) {
  using C = DecodeCfg<D, RG, kShared>;
  using W = typename C::W;
  using namespace ptx;
  constexpr int kRows = C::kRows, kKeys = C::kKeys, kS = C::kStages, kSide = C::kSide, kPad = C::kRowPad;
  constexpr int kTiles = D / 8;    // n8 tiles of the output
  constexpr int kHalves = D / 64;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = smem_raw + ((128u - (smem_u32(smem_raw) & 127u)) & 127u);
  float* merge = reinterpret_cast<float*>(ring);  // [4 RG warps][16][kPad], between items
  uint4* qfrag = reinterpret_cast<uint4*>(ring + (C::kRing > C::kMerge ? C::kRing : C::kMerge));  // [RG][D / 16][32]
  float2* ml = reinterpret_cast<float2*>(qfrag + RG * D * 2);  // [4 RG][16] running maximum and sum of each warp's rows
  W* walk = reinterpret_cast<W*>(ml + 4 * RG * 16);
  ScanShared* scan = reinterpret_cast<ScanShared*>(walk + 1);
  int* flags = reinterpret_cast<int*>(scan + 1);  // more items; last to arrive
  Plan* plan = reinterpret_cast<Plan*>(flags + 4);                    // of the item's stream (kShared), and its segments
  int4* seg = reinterpret_cast<int4*>((reinterpret_cast<uintptr_t>(plan + 1) + 15) & ~uintptr_t(15));
  int2* seq = kShared ? reinterpret_cast<int2*>(seg + kRows + 1) : reinterpret_cast<int2*>(flags + 4);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  grid_launch_dependents();
  grid_dependency_wait();
  long long run0, run1;
  {
    W w;
    if constexpr (kShared)
      share_out<C::kThreads>(a, seq, scan, w, reinterpret_cast<Count*>(ring));
    else
      share_out<C::kThreads>(a, seq, scan, w);
    run0 = w.u;
    run1 = w.u1;
    if (threadIdx.x == 0) *walk = w;
  }
  const int g = lane >> 2, c = lane & 3;
  const int rg = warp >> 2, kw = warp & 3;  // row group, key group
  uint8_t* const my_ring = ring + kw * kS * 2 * kSide;

  while (true) {
    if constexpr (kShared) {
      if (warp == 0) {
        const bool more = walk_next_planned(walk, plan, seg);
        if (lane == 0) flags[0] = more;
      }
    } else {
      if (threadIdx.x == 0) flags[0] = walk->next();
    }
    __syncthreads();
    if (!flags[0]) break;
    const Item& it = walk->it;
    const int kt0 = it.kt0, kt1 = it.kt1, lo = it.lo, hi = it.hi;

    // ---- the warp's stream of key groups
    // Lane l holds page and exponents of tile batch0 + l (this warp's 16 keys of it).
    int batch0 = kt0, b_page = -1, b_exps = 0, b_before = 0;  // b_before: the exponents of the batch before
    // kShared: the tile's segment | place of the keys in their page / 16 << 8 | all rows see all keys << 16 | slots behind the
    // end << 17
    int b_where = 0, b_where_before = 0;
    auto load_batch = [&]() {
      b_page = -1;
      b_before = b_exps;
      if constexpr (kShared) {
        b_where_before = b_where;
        int key0 = 0;
        const int at = batch0 + lane < kt1 ? seg_of<kKeys>(seg, plan->count, batch0 + lane, key0) : -1;
        if (at < 0) return;
        const int4 sg = seg[at];
        const int key = key0 + 16 * kw, table = at == 0 ? it.kv : sg.z;
        const int all_lo = at == 0 ? plan->pre_lo : plan->one_lo, all_hi = at == 0 ? it.hi : plan->one_hi;
        // positions before a window may have no page any more, those of the prefix none in this sequence's table
        int own_lo = at == 0 ? it.lo : it.hi;
        if (a.window > 0 && at > 0) {
          int own_hi;
          walk->own_range(sg.z, it.tok0 + a.token_of(it.row0), it.tok0 + a.token_of(it.row0 + it.rows - 1), it.hi, own_lo, own_hi);
        }
        if (key < sg.w && key + 16 > own_lo) {
          const int page = a.b.pages[static_cast<int64_t>(table) * a.b.max_pages + key / a.c.page];
          if (page >= 0 && page < a.c.n_pages) {
            b_page = page;
            b_where = at | (key & (a.c.page - 1)) << 4 | (key >= all_lo && key + 16 <= all_hi) << 16 | (key + 16 > sg.w) << 17;
            const int64_t ph = static_cast<int64_t>(page) * a.c.heads + it.head;
            const int ek = min(max(static_cast<int>(a.c.k_exp[ph]), kKvMinExp), kKvMaxExp);
            const int ev = min(max(static_cast<int>(a.c.v_exp[ph]), kKvMinExp), kKvMaxExp);
            b_exps = (ek + 64) | (ev + 64) << 8;
          } else {
            atomicOr(a.err, kErrInvalid);
          }
        }
        return;
      }
      const long long key = (static_cast<long long>(batch0) + lane) * kKeys + 16 * kw;
      if (batch0 + lane < kt1 && key < hi && key + 16 > lo) {
        const int page = a.b.pages[static_cast<int64_t>(it.b) * a.b.max_pages + key / a.c.page];
        if (page >= 0 && page < a.c.n_pages) {
          b_page = page;
          const int64_t ph = static_cast<int64_t>(page) * a.c.heads + it.head;
          const int ek = min(max(static_cast<int>(a.c.k_exp[ph]), kKvMinExp), kKvMaxExp);
          const int ev = min(max(static_cast<int>(a.c.v_exp[ph]), kKvMinExp), kKvMaxExp);
          b_exps = (ek + 64) | (ev + 64) << 8;
        } else {
          atomicOr(a.err, kErrInvalid);
        }
      }
    };
    // Copies the keys and values of tile kt into a stage; returns whether there are any.  (Their exponents are looked at
    // when the stage is read: the copies need not wait for them.)  A row's
    // 16-byte chunk k lands at k ^ (row & 1) * 4 for keys (a quarter warp reads 4 chunks of two rows) and at
    // k ^ (row / 2 & 3) * 2 for values (2 chunks of four row pairs); rows of 64 bytes: as they are, k ^ (row / 2 & 3).
    auto copy_step = [&](int kt, int stage) {
      bool any = false;
      if (kt < kt1) {
        if (kt - batch0 == 32) {
          batch0 = kt;
          load_batch();
        }
        const int page = __shfl_sync(0xFFFFFFFFu, b_page, kt - batch0);
        if (page >= 0) {
          any = true;
          constexpr int kPerRow = D / 16, kRowsAt = 32 / kPerRow;  // lanes to a row, rows at a time
          const int row0 = lane / kPerRow, chunk = lane % kPerRow;
          const int slot = kShared ? __shfl_sync(0xFFFFFFFFu, b_where, kt - batch0) >> 4 & 0x70 : (kt * kKeys + 16 * kw) & (a.c.page - 1);
          const int64_t at = ((static_cast<int64_t>(page) * a.c.heads + it.head) * a.c.page + slot + row0) * D + chunk * 16;
          const uint32_t dst = smem_u32(my_ring + stage * 2 * kSide);
#pragma unroll
          for (int n = 0; n < 16 / kRowsAt; ++n) {
            const int row = row0 + n * kRowsAt;
            const int ck = D == 128 ? chunk ^ (row & 1) * 4 : chunk;
            const int cv = D == 128 ? chunk ^ (row / 2 & 3) * 2 : chunk ^ (row / 2 & 3);
            if (RG == 1 || rg == 0) copy16_async(dst + row * D + ck * 16, a.c.k + at + n * kRowsAt * D);
            if (RG == 1 || rg == 1) copy16_async(dst + kSide + row * D + cv * 16, a.c.v + at + n * kRowsAt * D);
          }
        }
      }
      copy_group();
      return any;
    };
    // the queries' loads go out first, then the stream's: one latency for both
    uint4 qw[2][kHalves][2];
    int q_tok[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int row = rg * 16 + g + 8 * r, packed = it.row0 + (row < it.rows ? row : 0);
      q_tok[r] = a.token_of(packed);
      const uint16_t* qp = a.q + static_cast<int64_t>(it.tok0 + q_tok[r]) * a.q_token +
                           static_cast<int64_t>(it.head * a.group + packed - q_tok[r] * a.group) * D + 16 * c;
#pragma unroll
      for (int h = 0; h < kHalves; ++h) {
        qw[r][h][0] = *reinterpret_cast<const uint4*>(qp + 64 * h);
        qw[r][h][1] = *reinterpret_cast<const uint4*>(qp + 64 * h + 8);
      }
    }
    load_batch();
    bool pending[kS - 1];
#pragma unroll
    for (int s = 0; s < kS - 1; ++s) pending[s] = copy_step(kt0 + s, s);

    // ---- query fragments (each warp of a row group writes a quarter) and what each of the thread's two rows sees
    float mult[2];
    int lim[2], low[2];
    unsigned long long bits[2];
    bool odd[2];  // rows with a NaN or an infinity
    int of[2], row_base[2];  // kShared: each row's sequence, and where its new tokens begin
    const int base = kShared ? 0 : it.kv - it.n;
    {
      uint32_t* qf = reinterpret_cast<uint32_t*>(qfrag + rg * D * 2);
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int row = rg * 16 + g + 8 * r;
        const bool there = row < it.rows;
        const int i = q_tok[r];
        uint32_t w[kHalves][8];
        uint32_t amax = 0;
#pragma unroll
        for (int h = 0; h < kHalves; ++h) {
          const uint4 x = there ? qw[r][h][0] : make_uint4(0, 0, 0, 0);
          const uint4 y = there ? qw[r][h][1] : make_uint4(0, 0, 0, 0);
          const uint32_t v[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            w[h][e] = v[e];
            amax = max(amax, max(v[e] & 0x7FFFu, (v[e] >> 16) & 0x7FFFu));
          }
        }
        amax = max(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
        amax = max(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 2));
        odd[r] = amax >= 0x7F80u;
        const float shrink = row_shrink(amax);
        mult[r] = row_mult(amax, a.scale_log2);
        // word e of half h is k-step 4 h + e / 2, register r + 2 (e & 1) of the A fragment
#pragma unroll
        for (int h = 0; h < kHalves; ++h)
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if ((4 * h + e / 2) % 4 == kw)
              qf[((4 * h + e / 2) * 32 + lane) * 4 + r + 2 * (e & 1)] =
                  odd[r] ? 0u : pack_f16(bf16_lo(w[h][e]) * shrink, bf16_hi(w[h][e]) * shrink);
        if constexpr (kShared) {
          const RowSight v = row_sight(walk, it.tok0 + i, plan->seq0, plan->seq1);
          of[r] = v.seq;
          low[r] = v.low;
          lim[r] = v.lim;
          row_base[r] = v.base;
          bits[r] = a.tree && there ? a.tree[it.tok0 + i] : 0ull;
        } else
        if (a.tree) {
          lim[r] = it.kv;
          low[r] = 0;
          bits[r] = there ? a.tree[it.tok0 + i] : 0ull;
        } else {
          lim[r] = min(max(base + i + 1, 0), it.kv);
          low[r] = window_start(base + i, a.window);
          bits[r] = 0;
        }
      }
    }
    // positions that every row of the item sees: no masks there
    int all_lo = 0, all_hi = 0;
    if (!kShared) {
      const int i0 = a.token_of(it.row0), i1 = a.token_of(it.row0 + it.rows - 1);
      all_hi = a.tree ? max(base, 0) : min(max(base + i0 + 1, 0), it.kv);
      all_lo = window_start(base + i1, a.window);
    }
    __syncthreads();
    const uint4* q4 = qfrag + rg * D * 2 + lane;

    float o[kTiles][4];
#pragma unroll
    for (int j = 0; j < kTiles; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.0f;
    float m[2] = {kNoMax, kNoMax}, l[2] = {0.0f, 0.0f};

    int stage = 0;
    for (int kt = kt0; kt < kt1; ++kt) {
      copy_wait<kS - 2>();
      if (RG == 1)
        __syncwarp();
      else
        named_bar_sync(1 + kw, 64);  // the two warps of the key group
      const bool any = pending[0];
#pragma unroll
      for (int s = 0; s + 1 < kS - 1; ++s) pending[s] = pending[s + 1];
      const int free_stage = stage == 0 ? kS - 1 : stage - 1;  // the stage read last
      const uint8_t* at_k = my_ring + stage * 2 * kSide;
      stage = stage == kS - 1 ? 0 : stage + 1;
      if (!any) {
        pending[kS - 2] = copy_step(kt + kS - 1, free_stage);
        continue;
      }
      const int exps = __shfl_sync(0xFFFFFFFFu, kt >= batch0 ? b_exps : b_before, (kt - batch0) & 31);
      const int ek = (exps & 255) - 64, ev = (exps >> 8) - 64;
      const int where = kShared ? __shfl_sync(0xFFFFFFFFu, kt >= batch0 ? b_where : b_where_before, (kt - batch0) & 31) : 0;
      int key0 = kt * kKeys + 16 * kw;

      float sc[2][2][4];  // [n tile][chain]
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[t][0][e] = sc[t][1][e] = 0.0f;
#pragma unroll
      for (int h = 0; h < kHalves; ++h) {
        const int chunk = D == 128 ? (4 * h + c) ^ (g & 1) * 4 : c;
        const uint4 x = *reinterpret_cast<const uint4*>(at_k + g * D + chunk * 16);
        const uint4 y = *reinterpret_cast<const uint4*>(at_k + (8 + g) * D + chunk * 16);
        const uint32_t wx[4] = {x.x, x.y, x.z, x.w}, wy[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint4 q = q4[(4 * h + e) * 32];
          uint32_t b0, b1;
          e4m3x4_to_f16x4(wx[e], b0, b1);
          mma_f16(sc[0][e & 1], q, b0, b1);
          e4m3x4_to_f16x4(wy[e], b0, b1);
          mma_f16(sc[1][e & 1], q, b0, b1);
        }
      }
      pending[kS - 2] = copy_step(kt + kS - 1, free_stage);  // (under the MMAs' latency)
      // ---- scores: element e of tile t is row g + 8 (e / 2), key key0 + 8 t + 2 c + (e & 1)
      float z[2][4];
      const float mk[2] = {score_mult(mult[0], ek), score_mult(mult[1], ek)};
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) z[t][e] = fmaf(sc[t][0][e] + sc[t][1][e], mk[e >> 1], static_cast<float>(ev));
      if (kShared ? (where >> 16 & 1) == 0 : key0 + 16 > all_hi || key0 < all_lo) {
        const int at = where & 255;
        if (kShared) key0 = (seg[at].y + kt - (at > 0 ? seg[at - 1].x : 0)) * kKeys + 16 * kw;
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int j = key0 + 8 * t + 2 * c + (e & 1), r = e >> 1;
            bool see = j < lim[r] && j >= low[r];
            if (kShared) {
              see = see && (at == 0 ? j < it.hi : j >= it.hi && of[r] == seg[at].z);
              if (a.tree && j >= row_base[r]) see = see && j - row_base[r] < 64 && (bits[r] >> (j - row_base[r]) & 1ull);
            } else if (a.tree && j >= base) {
              see = see && j - base < 64 && (bits[r] >> (j - base) & 1ull);
            }
            if (!see) z[t][e] = -INFINITY;
          }
      }
      const float top0 = fmaxf(fmaxf(z[0][0], z[0][1]), fmaxf(z[1][0], z[1][1]));
      const float top1 = fmaxf(fmaxf(z[0][2], z[0][3]), fmaxf(z[1][2], z[1][3]));
      if (__any_sync(0xFFFFFFFFu, top0 - m[0] > kSlack || top1 - m[1] > kSlack)) {  // (a sum m + kSlack would round)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          float top = r == 0 ? top0 : top1;
          top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
          top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
          const float m1 = fmaxf(m[r], reference_of(top));
          const float keep = ex2(m[r] - m1);
          m[r] = m1;
          l[r] *= keep;
#pragma unroll
          for (int j = 0; j < kTiles; ++j) {
            o[j][2 * r] *= keep;
            o[j][2 * r + 1] *= keep;
          }
        }
      }
      uint4 pf;
      {
        float p[2][4];
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) p[t][e] = ex2(z[t][e] - m[e >> 1]);
        const float unit = exp2_int(-ev);
        l[0] = fmaf(p[0][0] + p[0][1] + p[1][0] + p[1][1], unit, l[0]);
        l[1] = fmaf(p[0][2] + p[0][3] + p[1][2] + p[1][3], unit, l[1]);
        pf = make_uint4(pack_f16(p[0][0], p[0][1]), pack_f16(p[0][2], p[0][3]), pack_f16(p[1][0], p[1][1]), pack_f16(p[1][2], p[1][3]));
      }
      // ---- values: channels [g * kTiles, + kTiles) of keys 2c, 2c + 1, 2c + 8, 2c + 9 (row / 2 & 3 = c for all four)
      const uint8_t* at_v = at_k + kSide + 2 * c * D + (D == 128 ? (g ^ 2 * c) * 16 : (g / 2 ^ c) * 16 + (g & 1) * 8);
      uint32_t v[4][kTiles / 4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint8_t* at = at_v + ((k & 1) + 8 * (k >> 1)) * D;
        if (D == 128) {
          const uint4 x = *reinterpret_cast<const uint4*>(at);
          v[k][0] = x.x;
          v[k][1] = x.y;
          v[k][kTiles / 4 - 2] = x.z;
          v[k][kTiles / 4 - 1] = x.w;
        } else {
          const uint2 x = *reinterpret_cast<const uint2*>(at);
          v[k][0] = x.x;
          v[k][1] = x.y;
        }
      }
      if (kShared ? where >> 17 & 1 : key0 + 16 > it.kv) {  // slots behind the end hold anything, NaN codes included
        int end = it.kv;
        if (kShared) {
          const int at = where & 255;
          end = seg[at].w;
          key0 = (seg[at].y + kt - (at > 0 ? seg[at - 1].x : 0)) * kKeys + 16 * kw;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (key0 + 2 * c + (k & 1) + 8 * (k >> 1) >= end)
#pragma unroll
            for (int w = 0; w < kTiles / 4; ++w) v[k][w] = 0;
      }
#pragma unroll
      for (int w = 0; w < kTiles / 4; ++w) {
        // bytes (key 0, key 1) of two channels per word
        const uint32_t a0 = __byte_perm(v[0][w], v[1][w], 0x5140), a1 = __byte_perm(v[0][w], v[1][w], 0x7362);
        const uint32_t b0 = __byte_perm(v[2][w], v[3][w], 0x5140), b1 = __byte_perm(v[2][w], v[3][w], 0x7362);
        uint32_t x0, x1, y0, y1;
        e4m3x4_to_f16x4(a0, x0, x1);
        e4m3x4_to_f16x4(b0, y0, y1);
        mma_f16(o[4 * w + 0], pf, x0, y0);
        mma_f16(o[4 * w + 1], pf, x1, y1);
        e4m3x4_to_f16x4(a1, x0, x1);
        e4m3x4_to_f16x4(b1, y0, y1);
        mma_f16(o[4 * w + 2], pf, x0, y0);
        mma_f16(o[4 * w + 3], pf, x1, y1);
      }
    }
    copy_wait<0>();

    // ---- the four key groups of each row meet in shared memory, where the ring was
    __syncthreads();
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      l[r] += __shfl_xor_sync(0xFFFFFFFFu, l[r], 1);
      l[r] += __shfl_xor_sync(0xFFFFFFFFu, l[r], 2);
      if (odd[r] && l[r] > 0.0f) l[r] = NAN;
      float* at = merge + (warp * 16 + g + 8 * r) * kPad;
      if (c == 0) ml[warp * 16 + g + 8 * r] = make_float2(m[r], l[r]);
#pragma unroll
      for (int e = 0; e < 2; ++e)   // channels [(2c + e) kTiles, + kTiles)
#pragma unroll
        for (int j = 0; j < kTiles; j += 4) {
          const int d = (2 * c + e) * kTiles + j;
          *reinterpret_cast<float4*>(at + d + d / (2 * kTiles) * 4) =
              make_float4(o[j][2 * r + e], o[j + 1][2 * r + e], o[j + 2][2 * r + e], o[j + 3][2 * r + e]);
        }
    }
    __syncthreads();
    const int row = threadIdx.x >> 3, part = threadIdx.x & 7;  // row of the item, 4-channel chunks part + 8 k
    const int w0 = (row >> 4) * 4;
    constexpr int kChunks = D / 32;
    float4 acc[kChunks];
    float mm = kNoMax, ll = 0.0f;
    {
      float2 x[4];
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        x[w] = ml[(w0 + w) * 16 + (row & 15)];
        mm = fmaxf(mm, x[w].x);
      }
#pragma unroll
      for (int k = 0; k < kChunks; ++k) acc[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const float f = ex2(x[w].x - mm);
        ll = fmaf(x[w].y, f, ll);
        const float* at = merge + ((w0 + w) * 16 + (row & 15)) * kPad;
#pragma unroll
        for (int k = 0; k < kChunks; ++k) {
          const int d = 4 * (part + 8 * k);
          const float4 v = *reinterpret_cast<const float4*>(at + d + d / (2 * kTiles) * 4);
          acc[k].x = fmaf(v.x, f, acc[k].x);
          acc[k].y = fmaf(v.y, f, acc[k].y);
          acc[k].z = fmaf(v.z, f, acc[k].z);
          acc[k].w = fmaf(v.w, f, acc[k].w);
        }
      }
    }
    bool done = true;
    if (it.ub < run0 || it.ue > run1) {
      // ---- part of an item: leave it in the workspace; the last part to arrive adds all of them in run order.  A
      // long sequence is cut into many parts, so parts meet in groups of kFan first: the last of a group leaves the
      // group's sum in the slot of its first part.  (One sequence of 131072 positions has 76 parts a head; read by one
      // CTA they took 10 of 66 us.)
      constexpr int kSlot = kRows * (D + 2), kFan = 9, kAtOnce = 5;  // (a full group's loads in two goes)
      const int c0 = owner_of(it.ub, scan), c1 = owner_of(it.ue - 1, scan), me = blockIdx.x;
      auto slot_of = [&](int k) { return a.partial + (static_cast<int64_t>(k) * 2 + (k == c0 ? 1 : 0)) * kSlot; };
      auto leave = [&](int k) {
        float* slot = slot_of(k);
        if (row < it.rows) {
#pragma unroll
          for (int e = 0; e < kChunks; ++e) *reinterpret_cast<float4*>(slot + row * D + 4 * (part + 8 * e)) = acc[e];
          if (part == 0) *reinterpret_cast<float2*>(slot + kRows * D + 2 * row) = make_float2(mm, ll);
        }
      };
      // Arrives; true for the last of n, which then sees what the others left.
      auto last_of = [&](unsigned int* ticket, int n) {
        __syncthreads();  // (the release below covers what the barrier made this thread see)
        if (threadIdx.x == 0) {
          const bool last = add_acq_rel(ticket, 1u) == static_cast<unsigned int>(n - 1);
          if (last) *ticket = 0;
          flags[1] = last;
        }
        __syncthreads();
        return flags[1] != 0;
      };
      auto add_up = [&](int first, int step, int end) {  // the slots of first, first + step, ... before end
        if (row >= it.rows) return;
        mm = kNoMax;
        ll = 0.0f;
#pragma unroll
        for (int e = 0; e < kChunks; ++e) acc[e] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        for (int k0 = first; k0 < end; k0 += kAtOnce * step) {
          float2 x[kAtOnce];
          float4 v[kAtOnce][kChunks];
#pragma unroll
          for (int j = 0; j < kAtOnce; ++j) {
            const float* p = slot_of(min(k0 + j * step, end - 1 - (end - 1 - first) % step));
            x[j] = __ldcg(reinterpret_cast<const float2*>(p + kRows * D + 2 * row));
#pragma unroll
            for (int e = 0; e < kChunks; ++e) v[j][e] = __ldcg(reinterpret_cast<const float4*>(p + row * D + 4 * (part + 8 * e)));
          }
          float m1 = mm;
#pragma unroll
          for (int j = 0; j < kAtOnce; ++j)
            if (k0 + j * step < end) m1 = fmaxf(m1, x[j].x);
          const float keep = ex2(mm - m1);
          mm = m1;
          ll *= keep;
#pragma unroll
          for (int e = 0; e < kChunks; ++e) acc[e] = make_float4(acc[e].x * keep, acc[e].y * keep, acc[e].z * keep, acc[e].w * keep);
#pragma unroll
          for (int j = 0; j < kAtOnce; ++j) {
            if (k0 + j * step >= end) continue;
            const float f = ex2(x[j].x - mm);
            ll = fmaf(x[j].y, f, ll);
#pragma unroll
            for (int e = 0; e < kChunks; ++e) {
              acc[e].x = fmaf(v[j][e].x, f, acc[e].x);
              acc[e].y = fmaf(v[j][e].y, f, acc[e].y);
              acc[e].z = fmaf(v[j][e].z, f, acc[e].z);
              acc[e].w = fmaf(v[j][e].w, f, acc[e].w);
            }
          }
        }
      };
      leave(me);
      const int n = c1 - c0 + 1;
      if (n <= kFan) {
        done = last_of(a.tickets + c0, n);
        if (done) add_up(c0, 1, c1 + 1);
      } else {
        const int first = c0 + (me - c0) / kFan * kFan, end = min(first + kFan, c1 + 1);
        // (a run can be the first of one item and a later one of the item before: two sets of tickets)
        done = last_of(a.tickets + (first == c0 ? 1 : 2) * gridDim.x + first, end - first);
        if (done) {
          add_up(first, 1, end);
          leave(first);
          done = last_of(a.tickets + c0, (n + kFan - 1) / kFan);
          if (done) add_up(c0, kFan, c1 + 1);
        }
      }
    }
    if (done && row < it.rows) {
      const int packed = it.row0 + row, i = a.token_of(packed);
      const int64_t t = it.tok0 + i;
      const int hq = it.head * a.group + packed - i * a.group;
      const float inv = ll == 0.0f ? 0.0f : 1.0f / ll;
      uint16_t* op = a.out + t * a.out_token + static_cast<int64_t>(hq) * D;
#pragma unroll
      for (int k = 0; k < kChunks; ++k)
        *reinterpret_cast<uint2*>(op + 4 * (part + 8 * k)) =
            make_uint2(pack_bf16(acc[k].x * inv, acc[k].y * inv), pack_bf16(acc[k].z * inv, acc[k].w * inv));
      if (a.lse && part == 0)
        a.lse[t * a.heads_q + hq] = ll == 0.0f ? -INFINITY : (mm + log2f(ll)) * 0.693147180559945f;
    }
    __syncthreads();  // the item and the merge buffer are read: the next item may take their places
  }
}

}  // namespace att
}  // namespace qspec
