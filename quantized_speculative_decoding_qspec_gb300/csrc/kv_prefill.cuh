// Attention for many query rows per key head (prompt chunks, wide trees) on the tcgen05 tensor cores.
//
// A CTA owns an item of 256 rows as two tiles X = 0, 1 of 128, and streams 128 keys at a time:
//   S_X = Q_X K^T (both from shared memory), P_X = 2^(S_X c + ev - m) by one thread per row, O_X += P_X V
// with S, P and O in TMEM (S 2 x 128 columns, P over the S it came from, O 2 x D).  The two tiles alternate
// on the tensor core, PV_0 S_0' PV_1 S_1', so that the softmax of one tile runs under the products of the other.
//  * The cache's codes arrive by bulk copies in a ring of raw tiles; four warps turn them into fp16 (exact) in
//    the 128-byte swizzled layout.  Keys are read along channels (K-major); the same layout of the values is
//    read along tokens (N-major B operand), so nothing is transposed.  Their lane mapping (two keys, opposite
//    halves of the channels per quarter warp) keeps loads and stores free of bank conflicts.
//  * Scales as in the decode kernel: 2^ek on the scores, 2^ev in the exponent, l = sum P 2^-ev.
//  * m moves only when a score exceeds it by 2^8; then the row's O and the tile's earlier P are rescaled in
//    TMEM (S of a tile is complete only after the tile's last PV, so O is at rest).
// Warps: 0-7 softmax (thread = row), 8-11 converters, 12 copies, 13 MMA issue.  Stages change hands by
// mbarriers; every wait is bounded and ends the CTA in order (kErrTimeout) when it runs out.
#pragma once

#include "kv_sched.cuh"

namespace qspec {
namespace att {

template <int D>
struct PrefillCfg {
  static constexpr int kRows = 256, kKeys = 128;
  static constexpr int kThreads = 14 * 32;
  static constexpr int kRaw = kKeys * D;          // one side of a tile, codes
  static constexpr int kConv = kKeys * D * 2;     // the same in fp16
  static constexpr int kHalves = D / 64;          // 128-byte wide sub-tiles
  static constexpr int kQ = 128 * D * 2;          // one tile of queries
  static constexpr int kNR = 3 * (128 / D), kNC = 3, kMeta = 8;
  static constexpr int kSmem = 1024 + 2 * kQ + kNC * kConv + kNR * kRaw + 4096;
};

struct TileMeta {
  int ek[8], ev[8];  // per 16 keys; ek = kBadGroup: no keys there
};

template <int D>
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
  int2* seq = reinterpret_cast<int2*>(scan + 1) + 2;
  volatile int* abort_flag = flags;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kNR; ++i) {
      mbar_init(rawfull + i, 1);
      mbar_init(rawempty + i, 4);
    }
    for (int i = 0; i < kNC; ++i) {
      mbar_init(convfull + i, 4);
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
  if (warp == 13) {
    tmem_alloc(tmem_base, kCols);
    tmem_relinquish();
  }
  grid_launch_dependents();
  grid_dependency_wait();
  Walk<kRows, kKeys> walk;
  tc_fence_before();
  share_out<C::kThreads>(a, seq, scan, walk);  // (barriers inside)
  tc_fence_after();
  const uint32_t tmem = *tmem_base;
  const long long run0 = walk.u;

  if (warp == 12) {
    // ------------------------------------------------------------------ copies
    const int P = a.c.page, per_tile = kKeys / P;
    const uint32_t seg_bytes = P * D;
    int t = 0, issued = 0;
    while (walk.next()) {
      const Item& it = walk.it;
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
            if (lane < 8) md.ek[lane] = kBadGroup;
            __syncwarp();
            if (mine) {
              const int g0 = (lane - l0) * (P / 16);
              for (int g = g0; g < g0 + P / 16; ++g) {
                md.ek[g] = sb.ek;
                md.ev[g] = sb.ev;
              }
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
  } else if (warp >= 8 && warp < 12) {
    // ------------------------------------------------------------------ converters
    const int cw = warp - 8;
    int i = 0;
    bool ok = true;
    while (ok && walk.next()) {
      const Item& it = walk.it;
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
#pragma unroll
          for (int step = 0; step < kKeys / 32; ++step) {  // 8 keys of this warp's 32
            const int key = cw * 32 + step * 8 + 2 * (lane >> 3) + sub;
            const bool live = md.ek[key >> 4] != kBadGroup && key < kv_in;
#pragma unroll
            for (int h = 0; h < C::kHalves; ++h) {
              const int half = C::kHalves == 2 ? (h ^ sub) : 0;
              uint4 w = *reinterpret_cast<const uint4*>(src + key * D + half * 64 + quad * 16);
              if (!live) w = make_uint4(0, 0, 0, 0);
              uint4 lo, hi;
              lo.x = e4m3x2_to_f16x2(w.x);
              lo.y = e4m3x2_to_f16x2(w.x >> 16);
              lo.z = e4m3x2_to_f16x2(w.y);
              lo.w = e4m3x2_to_f16x2(w.y >> 16);
              hi.x = e4m3x2_to_f16x2(w.z);
              hi.y = e4m3x2_to_f16x2(w.z >> 16);
              hi.z = e4m3x2_to_f16x2(w.w);
              hi.w = e4m3x2_to_f16x2(w.w >> 16);
              uint8_t* row = dst + half * kSub + key * 128;
              *reinterpret_cast<uint4*>(row + (((2 * quad) ^ (key & 7)) << 4)) = lo;
              *reinterpret_cast<uint4*>(row + (((2 * quad + 1) ^ (key & 7)) << 4)) = hi;
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
  } else if (warp == 13) {
    // ------------------------------------------------------------------ MMA issue
    if (lane == 0) {
      const uint32_t idesc_s = idesc_f16_f32(128, kKeys);
      const uint32_t idesc_o = idesc_f16_f32(128, D) | kIdescBMajorMN;
      const uint32_t q_addr = smem_u32(qs), c_addr = smem_u32(conv);
      int t = 0;             // tiles so far
      uint32_t item = 0, np[2] = {0, 0};
      bool ok = true;
      auto scores = [&](int X, uint32_t k_addr) {
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          const uint32_t off = (ks >> 2) * kSub + (ks & 3) * 32;
          mma_f16_ss(tmem + X * 128, smem_desc_sw128(q_addr + X * C::kQ + off), smem_desc_sw128(k_addr + off), idesc_s, ks > 0);
        }
        mma_commit(sfull + X);
      };
      auto values = [&](int X, uint32_t v_addr, bool first) {
#pragma unroll
        for (int ks = 0; ks < kKeys / 16; ++ks)
          mma_bf16_ts(tmem + kOCol + X * D, tmem + X * 128 + ks * 8, smem_desc_sw128_mn(v_addr + ks * 2048, kSub), idesc_o,
                      !(first && ks == 0));
      };
      while (ok && walk.next()) {
        const Item& it = walk.it;
        const int tiles = it.rows > 128 ? 2 : 1;
        ok = wait_bar(qfull, item & 1, abort_flag, a.err);
        auto conv_wait = [&](int i) {
          ok = ok && wait_bar(convfull + i % kNC, (i / kNC) & 1, abort_flag, a.err);
          return c_addr + (i % kNC) * C::kConv;
        };
        uint32_t k_addr = conv_wait(2 * t);
        if (!ok) break;
        tc_fence_after();
        for (int X = 0; X < tiles; ++X) scores(X, k_addr);
        mma_commit(convempty + (2 * t) % kNC);
        for (int kt = it.kt0; ok && kt < it.kt1; ++kt, ++t) {
          const bool more = kt + 1 < it.kt1;
          const uint32_t v_addr = conv_wait(2 * t + 1);
          if (kt == it.kt0 && item > 0) ok = ok && wait_bar(ofree, (item - 1) & 1, abort_flag, a.err);
          for (int X = 0; ok && X < tiles; ++X) {
            ok = wait_bar(pfull + X, np[X]++ & 1, abort_flag, a.err);
            if (X == 0 && more) k_addr = conv_wait(2 * t + 2);
            if (!ok) break;
            tc_fence_after();
            values(X, v_addr, kt == it.kt0);
            if (X == tiles - 1) mma_commit(convempty + (2 * t + 1) % kNC);
            if (more) scores(X, k_addr);
          }
          if (ok && more) mma_commit(convempty + (2 * t + 2) % kNC);
        }
        if (ok) {
          mma_commit(odone);
          ++item;
        }
      }
      // every MMA issued has finished before the CTA gives its TMEM and shared memory back: odone or, after
      // a wait ran out, one more commit
      if (!ok) {
        *abort_flag = 1;
        mma_commit(odone);
        wait_bar_final(odone, item & 1, a.err);
      }
    }
    __syncwarp();
  } else if (warp < 8) {
    // ------------------------------------------------------------------ softmax: thread = row
    const int X = warp >> 2, row = threadIdx.x;  // row of the item
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + lane_base + X * 128, to = tmem + lane_base + kOCol + X * D;
    int t = 0;
    uint32_t item = 0, ns = 0;
    bool ok = true;
    while (walk.next()) {
      const Item& it = walk.it;
      const bool active = X * 128 < it.rows, there = row < it.rows;
      const int packed = it.row0 + (there ? row : 0), i = packed / a.group;
      const int hq = it.head * a.group + packed - i * a.group;
      const int base = it.kv - it.n;
      // ---- the row's query: largest value to 2^14, rounded to nothing (fp16 holds all bits of bf16)
      bool odd = false;
      float mult = 0.0f;
      if (active) {
        const uint4* qp = reinterpret_cast<const uint4*>(a.q + static_cast<int64_t>(it.tok0 + i) * a.q_token + static_cast<int64_t>(hq) * D);
        uint32_t amax = 0;
#pragma unroll 4
        for (int k = 0; k < D / 8; ++k) {
          const uint4 w = qp[k];
          const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) amax = max(amax, max(v[e] & 0x7FFFu, (v[e] >> 16) & 0x7FFFu));
        }
        odd = amax >= 0x7F80u;
        const float shrink = copysignf(row_shrink(amax), a.scale_log2);
        mult = row_mult(amax, fabsf(a.scale_log2));
        uint8_t* q_row = qs + X * C::kQ + (row & 127) * 128;
#pragma unroll 4
        for (int k = 0; k < D / 8; ++k) {
          const uint4 w = qp[k];
          const uint32_t v[4] = {w.x, w.y, w.z, w.w};
          uint32_t f[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) f[e] = odd || !there ? 0u : pack_f16(bf16_lo(v[e]) * shrink, bf16_hi(v[e]) * shrink);
          *reinterpret_cast<uint4*>(q_row + (k >> 3) * kSub + (((k & 7) ^ (row & 7)) << 4)) = make_uint4(f[0], f[1], f[2], f[3]);
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(qfull);
      int lim, low;
      unsigned long long bits = 0;
      if (a.tree) {
        lim = it.kv;
        low = 0;
        bits = there ? a.tree[it.tok0 + i] : 0ull;
      } else {
        lim = min(max(base + i + 1, 0), it.kv);
        low = a.window > 0 ? max(base + i + 1 - a.window, 0) : 0;
      }
      int all_lo, all_hi;  // positions that every row of the item sees
      {
        const int i0 = it.row0 / a.group, i1 = (it.row0 + it.rows - 1) / a.group;
        all_hi = a.tree ? max(base, 0) : min(max(base + i0 + 1, 0), it.kv);
        all_lo = a.window > 0 ? max(base + i1 + 1 - a.window, 0) : 0;
      }
      float m = kNoMax, l = 0.0f;
      bool far = false;  // a maximum of the warp's rows is so large that its rounding matters in an exponent
      if (active) {
        for (int kt = it.kt0; kt < it.kt1; ++kt) {
          const int tt = t + kt - it.kt0;
          ok = ok && wait_bar(metafull + tt % kMeta, (tt / kMeta) & 1, abort_flag, a.err);
          ok = ok && wait_bar(sfull + X, ns & 1, abort_flag, a.err);
          ok = __all_sync(0xFFFFFFFFu, ok);
          if (!ok) break;
          ++ns;
          tc_fence_after();
          const TileMeta& md = meta[tt % kMeta];
          const int key0 = kt * kKeys;
          bool masks = key0 + kKeys > all_hi || key0 < all_lo;
#pragma unroll
          for (int g = 0; g < 8; ++g) masks |= md.ek[g] == kBadGroup;
#pragma unroll 1
          for (int ch = 0; ch < 4; ++ch) {  // 32 keys
            uint32_t s[32];
            tmem_ld32(ts + ch * 32, s);
            const int ek0 = md.ek[2 * ch], ek1 = md.ek[2 * ch + 1];
            const int ev0 = ek0 == kBadGroup ? 0 : md.ev[2 * ch], ev1 = ek1 == kBadGroup ? 0 : md.ev[2 * ch + 1];
            const float mk0 = ek0 == kBadGroup ? 0.0f : score_mult(mult, ek0), mk1 = ek1 == kBadGroup ? 0.0f : score_mult(mult, ek1);
            tmem_wait_ld();
            if (masks) {
#pragma unroll
              for (int e = 0; e < 32; ++e) {
                const int j = key0 + ch * 32 + e;
                bool see = j < lim && j >= low && (e < 16 ? ek0 : ek1) != kBadGroup;
                if (a.tree && j >= base) see = see && j - base < 64 && (bits >> (j - base) & 1ull);
                if (!see) s[e] = 0xFF800000u;  // -inf
              }
            }
            float g0 = __uint_as_float(s[0]), g1 = __uint_as_float(s[16]);
#pragma unroll
            for (int e = 1; e < 16; ++e) {
              g0 = fmaxf(g0, __uint_as_float(s[e]));
              g1 = fmaxf(g1, __uint_as_float(s[16 + e]));
            }
            // (a product of -inf and a factor 0 would be NaN: a group that nobody sees stays out)
            const float z0 = g0 == -INFINITY ? -INFINITY : fmaf(g0, mk0, static_cast<float>(ev0));
            const float z1 = g1 == -INFINITY ? -INFINITY : fmaf(g1, mk1, static_cast<float>(ev1));
            const float top = fmaxf(z0, z1);
            if (__any_sync(0xFFFFFFFFu, top > m + 8.0f)) {
              const float m1 = ceilf(fmaxf(m, top));  // whole, so the factor is a power of two: exact on P and O
              const float keep = ex2(m - m1);
              m = m1;
              l *= keep;
              far = __any_sync(0xFFFFFFFFu, fabsf(m) > 4194304.0f);
              tmem_wait_st();
              if (kt > it.kt0) {
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
#pragma unroll 1
              for (int c = 0; c < ch; ++c) {
                uint32_t p[16];
                tmem_ld16(ts + c * 16, p);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                  const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&p[e]));
                  p[e] = pack_f16(v.x * keep, v.y * keep);
                }
                tmem_st16(ts + c * 16, p);
              }
            }
            uint32_t p[16];
            const float b0 = static_cast<float>(ev0) - m, b1 = static_cast<float>(ev1) - m;
            float l0 = 0.0f, l1 = 0.0f;
            if (masks || far) {  // scores rounded as the maximum was; factors may be 0
#pragma unroll
              for (int e = 0; e < 32; ++e) {
                const float z = fmaf(__uint_as_float(s[e]), e < 16 ? mk0 : mk1, static_cast<float>(e < 16 ? ev0 : ev1));
                s[e] = s[e] == 0xFF800000u ? 0u : __float_as_uint(ex2(z - m));
              }
            } else {
#pragma unroll
              for (int e = 0; e < 32; ++e) s[e] = __float_as_uint(ex2(fmaf(__uint_as_float(s[e]), e < 16 ? mk0 : mk1, e < 16 ? b0 : b1)));
            }
#pragma unroll
            for (int e = 0; e < 16; e += 2) {
              l0 += __uint_as_float(s[e]) + __uint_as_float(s[e + 1]);
              l1 += __uint_as_float(s[16 + e]) + __uint_as_float(s[17 + e]);
              p[e / 2] = pack_f16(__uint_as_float(s[e]), __uint_as_float(s[e + 1]));
              p[8 + e / 2] = pack_f16(__uint_as_float(s[16 + e]), __uint_as_float(s[17 + e]));
            }
            l = fmaf(l0, exp2_int(-ev0), l);
            l = fmaf(l1, exp2_int(-ev1), l);
            tmem_st16(ts + ch * 16, p);
          }
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(pfull + X);
        }
      }
      t += it.kt1 - it.kt0;
      if (odd && l > 0.0f) l = NAN;
      ok = ok && wait_bar(odone, item & 1, abort_flag, a.err);
      ok = __all_sync(0xFFFFFFFFu, ok);
      if (!ok) *abort_flag = 1;
      ++item;
      tc_fence_after();
      const int64_t tok = it.tok0 + i;
      uint16_t* op = a.out + tok * a.out_token + static_cast<int64_t>(hq) * D;
      const bool whole = it.ub >= run0 && it.ue <= walk.u1;
      constexpr int kSlot = kRows * (D + 2);
      float* slot = a.partial + (static_cast<int64_t>(blockIdx.x) * 2 + (it.ub >= run0 ? 1 : 0)) * kSlot;
      if (ok && active) {
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll 1
        for (int c = 0; c < D; c += 16) {
          uint32_t o[16];
          __syncwarp();
          tmem_ld16(to + c, o);
          tmem_wait_ld();
          if (there && whole) {
            uint32_t w[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) w[e] = pack_bf16(__uint_as_float(o[2 * e]) * inv, __uint_as_float(o[2 * e + 1]) * inv);
            *reinterpret_cast<uint4*>(op + c) = make_uint4(w[0], w[1], w[2], w[3]);
            *reinterpret_cast<uint4*>(op + c + 8) = make_uint4(w[4], w[5], w[6], w[7]);
          } else if (there) {
#pragma unroll
            for (int e = 0; e < 4; ++e)  // [channel / 4][row]: consecutive rows are consecutive addresses
              *reinterpret_cast<uint4*>(slot + (static_cast<int64_t>(c / 4 + e) * kRows + row) * 4) =
                  make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
          }
        }
        if (!whole && there) *reinterpret_cast<float2*>(slot + kRows * D + 2 * row) = make_float2(m, l);
        if (whole && there && a.lse) a.lse[tok * a.heads_q + hq] = l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.693147180559945f;
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(ofree);
      if (!whole) {
        const int c0 = owner_of(it.ub, scan), c1 = owner_of(it.ue - 1, scan);
        __threadfence();
        named_bar_sync(1, 256);
        if (threadIdx.x == 0) {
          const bool last = atomicAdd(a.tickets + c0, 1u) == static_cast<unsigned int>(c1 - c0);
          if (last) a.tickets[c0] = 0;
          flags[1] = last;
          flags[2] = *abort_flag;  // (one reading for all warps: they leave together)
        }
        named_bar_sync(1, 256);
        if (flags[2]) break;
        if (flags[1] && there) {
          __threadfence();
          float mm = kNoMax, ll = 0.0f;
          for (int k = c0; k <= c1; ++k)
            mm = fmaxf(mm, __ldcg(a.partial + (static_cast<int64_t>(k) * 2 + (k == c0 ? 1 : 0)) * kSlot + kRows * D + 2 * row));
          for (int k = c0; k <= c1; ++k) {
            const float2 x = __ldcg(reinterpret_cast<const float2*>(a.partial + (static_cast<int64_t>(k) * 2 + (k == c0 ? 1 : 0)) * kSlot + kRows * D + 2 * row));
            ll = fmaf(x.y, ex2(x.x - mm), ll);
          }
          const float inv = ll == 0.0f ? 0.0f : 1.0f / ll;
#pragma unroll 1
          for (int c = 0; c < D; c += 16) {
            float4 acc[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[e] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            for (int k = c0; k <= c1; ++k) {
              const float* p = a.partial + (static_cast<int64_t>(k) * 2 + (k == c0 ? 1 : 0)) * kSlot;
              const float f = ex2(__ldcg(p + kRows * D + 2 * row) - mm);
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float4 v = __ldcg(reinterpret_cast<const float4*>(p + (static_cast<int64_t>(c / 4 + e) * kRows + row) * 4));
                acc[e].x = fmaf(v.x, f, acc[e].x);
                acc[e].y = fmaf(v.y, f, acc[e].y);
                acc[e].z = fmaf(v.z, f, acc[e].z);
                acc[e].w = fmaf(v.w, f, acc[e].w);
              }
            }
            uint32_t w[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              w[2 * e] = pack_bf16(acc[e].x * inv, acc[e].y * inv);
              w[2 * e + 1] = pack_bf16(acc[e].z * inv, acc[e].w * inv);
            }
            *reinterpret_cast<uint4*>(op + c) = make_uint4(w[0], w[1], w[2], w[3]);
            *reinterpret_cast<uint4*>(op + c + 8) = make_uint4(w[4], w[5], w[6], w[7]);
          }
          if (a.lse) a.lse[tok * a.heads_q + hq] = ll == 0.0f ? -INFINITY : (mm + log2f(ll)) * 0.693147180559945f;
        }
      } else {
        // the queries' shared memory and the flags are taken up again by the next item, in step
        named_bar_sync(1, 256);
        if (threadIdx.x == 0) flags[2] = *abort_flag;
        named_bar_sync(1, 256);
        if (flags[2]) break;
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 13) {
    tc_fence_after();
    tmem_dealloc(tmem, kCols);
  }
}

}  // namespace att
}  // namespace qspec
