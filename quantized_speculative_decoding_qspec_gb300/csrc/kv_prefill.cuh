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

#include "kv_sched.cuh"

namespace qspec {
namespace att {

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
  static constexpr int kSmem = 1024 + 2 * kQ + kNC * kConv + kNR * kRaw + 6144;
};

// Per 16 keys of a tile: the keys' scale, the values' exponent, its inverse scale, whether there are keys at all.
struct TileMeta {
  float4 group[8];
  int whole[4];  // [0]: all eight groups have keys
};

// kBigPages: pages of 64 slots or more, so 64 keys lie in one page and share its scales.
template <int D, bool kBigPages>
__global__ void __launch_bounds__(PrefillCfg<D>::kThreads, 1) prefill_kernel(const AttArgs a) {
  using C = PrefillCfg<D>;
  using namespace ptx;
  constexpr int kRows = C::kRows, kKeys = C::kKeys, kNR = C::kNR, kNC = C::kNC, kMeta = C::kMeta;
  constexpr int kSub = kKeys * 128;  // bytes of a sub-tile: 128 rows of 128 bytes
  constexpr uint32_t kOCol = 256, kCols = 512;
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
  ScanShared* scan = reinterpret_cast<ScanShared*>(ofree + 1);
  volatile int* flags = reinterpret_cast<volatile int*>(scan + 1);  // abort, last to arrive, abort as the item ended
  uint32_t* tmem_base = reinterpret_cast<uint32_t*>(scan + 1) + 3;
  Walk<kRows, kKeys>* walks = reinterpret_cast<Walk<kRows, kKeys>*>(reinterpret_cast<int2*>(scan + 1) + 2);  // [16]
  int2* seq = reinterpret_cast<int2*>(walks + 16);
  volatile int* abort_flag = flags;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kNR; ++i) {
      mbar_init(rawfull + i, 1);
      mbar_init(rawempty + i, C::kConvs);
    }
    for (int i = 0; i < kNC; ++i) {
      mbar_init(convfull + i, C::kConvs);
      mbar_init(convempty + i, 1);
    }
    for (int i = 0; i < kMeta; ++i) mbar_init(metafull + i, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(sfull + i, 1);
      mbar_init(pfull + i, 4);
    }
    mbar_init(qfull, 8);
    mbar_init(odone, 1);
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
  tc_fence_before();
  Walk<kRows, kKeys>* walk = walks + warp;  // (in shared memory: its state would cost every role 40 registers)
  long long run0, run1;
  {
    Walk<kRows, kKeys> w;
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
    const int X = warp >> 2, row = threadIdx.x;  // of the item
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
      const bool active = X * 128 < it.rows, there = row < it.rows;
      // ---- queries: coalesced, largest value of each row to 2^14; fp16 then holds all bits of bf16
      uint32_t amax = 0;  // of the thread's row
      if (active) {
        const uint16_t* qp = a.q + static_cast<int64_t>(it.tok0) * a.q_token + static_cast<int64_t>(it.head) * a.group * D + 8 * my_chunk;
        int tk = a.token_of(it.row0 + warp * 32 + my_row), in_group = it.row0 + warp * 32 + my_row - tk * a.group;
#pragma unroll 1
        for (int i0 = 0; i0 < kSteps; i0 += 8) {  // (8 loads in flight; rolled, as cold code costs its fetch)
          uint4 w[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const bool real = warp * 32 + (i0 + i) * kPer + my_row < it.rows;
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
      int all_lo, all_hi;  // positions that every row of the item sees
      {
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
      float m = kNoMax, l = 0.0f;
      bool far = false;  // a reference of the warp's rows is so large that its rounding matters in an exponent
      if (active) {
        for (int n = 0; n < tiles; ++n) {
          const int tt = t + n;
          ok = ok && wait_bar(metafull + tt % kMeta, (tt / kMeta) & 1, abort_flag, a.err);
          const TileMeta& md = meta[tt % kMeta];
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
          const bool whole_tile = md.whole[0] != 0;
          ok = ok && wait_bar(sfull + X, ns & 1, abort_flag, a.err);
          ok = __all_sync(0xFFFFFFFFu, ok);
          if (!ok) break;
          ++ns;
          tc_fence_after();
          const int key0 = (kt0 + n) * kKeys;
          const bool plain = key0 + kKeys <= all_hi && key0 >= all_lo && whole_tile;
          float top = -INFINITY;
          float s[4][32];
          if (plain) {
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
            far = __any_sync(0xFFFFFFFFu, fabsf(m) > kFar);
            if (n > 0) {
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
          if (plain && !far) {
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
          if (lane == 0) mbar_arrive(pfull + X);
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
      if (ok && active) {
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          float o[32];
          __syncwarp();
          tmem_ld32(to + c, o);
          tmem_wait_ld();
          if (whole) {
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
          store_rows();
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
      if (!whole) {
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
    if (warp >= C::kConv0) {
      // ------------------------------------------------------------------ converters
      const int cw = warp - C::kConv0;
      int i = 0;
      bool ok = true;
      while (ok && walk_next(walk)) {
        const Item& it = walk->it;
        for (int kt = it.kt0; ok && kt < it.kt1; ++kt) {
          const int kv_in = it.kv - kt * kKeys;  // slots from here on hold anything
          for (int side = 0; side < 2; ++side, ++i) {
            const int st = i % kNR, sc = i % kNC;
            ok = ok && wait_bar(rawfull + st, (i / kNR) & 1, abort_flag, a.err);
            if (i >= kNC) ok = ok && wait_bar(convempty + sc, ((i / kNC) - 1) & 1, abort_flag, a.err);
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (!ok) break;
            const uint8_t* src = raw + st * C::kRaw;
            uint8_t* dst = conv + sc * C::kConv;
            const TileMeta& md = meta[(i >> 1) % kMeta];
            // a quarter warp takes two keys; D = 128: the first key's chunks of one half, the second's of the other
            const int quad = lane & 3, sub = (lane >> 2) & 1;
            const bool all = md.whole[0] != 0 && kv_in >= kKeys;
            // 16 steps of 8 keys, two or three to a warp; all loads first
            constexpr int kMine = (kKeys / 8 + C::kConvs - 1) / C::kConvs;
            uint4 w[kMine][C::kHalves];
#pragma unroll
            for (int n = 0; n < kMine; ++n) {
              const int step = cw + n * C::kConvs, key = step * 8 + 2 * (lane >> 3) + sub;
              if (n < kMine - 1 || step < kKeys / 8) {
                const bool live = all || (md.group[key >> 4].w != 0.0f && key < kv_in);
#pragma unroll
                for (int h = 0; h < C::kHalves; ++h) {
                  const int half = C::kHalves == 2 ? (h ^ sub) : 0;
                  w[n][h] = live ? *reinterpret_cast<const uint4*>(src + key * D + half * 64 + quad * 16) : make_uint4(0, 0, 0, 0);
                }
              }
            }
#pragma unroll
            for (int n = 0; n < kMine; ++n) {
              const int step = cw + n * C::kConvs, key = step * 8 + 2 * (lane >> 3) + sub;
              if (n < kMine - 1 || step < kKeys / 8) {
#pragma unroll
                for (int h = 0; h < C::kHalves; ++h) {
                  const int half = C::kHalves == 2 ? (h ^ sub) : 0;
                  const uint4 v = w[n][h];
                  uint8_t* row = dst + half * kSub + key * 128;
                  *reinterpret_cast<uint4*>(row + (((2 * quad) ^ (key & 7)) << 4)) =
                      make_uint4(e4m3x2_to_f16x2(v.x), e4m3x2_to_f16x2(v.x >> 16), e4m3x2_to_f16x2(v.y), e4m3x2_to_f16x2(v.y >> 16));
                  *reinterpret_cast<uint4*>(row + (((2 * quad + 1) ^ (key & 7)) << 4)) =
                      make_uint4(e4m3x2_to_f16x2(v.z), e4m3x2_to_f16x2(v.z >> 16), e4m3x2_to_f16x2(v.w), e4m3x2_to_f16x2(v.w >> 16));
                }
              }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              mbar_arrive(rawempty + st);
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
        for (int kt = it.kt0; kt < it.kt1; ++kt, ++t) {
          const int seg = kt * per_tile;
          if (sb.seg0 < 0 || seg >= sb.seg0 + 32) sb = load_segs(a, it, seg, P);
          const int l0 = seg - sb.seg0;
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
      while (ok && walk_next(walk)) {
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
        commit(odone);
        if (lane == 0) wait_bar_final(odone, item & 1, a.err);
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
  if (*abort_flag && threadIdx.x == 0) {
    const long long c = blockIdx.x, u0 = run_start(c, scan), u1 = run_start(c + 1, scan);
    while (walks->next_cut(u0, u1)) {
      const int c0 = owner_of(walks->it.ub, scan), c1 = owner_of(walks->it.ue - 1, scan);
      if (add_acq_rel(a.tickets + c0, 1u) == static_cast<unsigned int>(c1 - c0)) a.tickets[c0] = 0;
    }
  }
}

}  // namespace att
}  // namespace qspec
