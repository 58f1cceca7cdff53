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
//    z = score + ev and m = max z, P = 2^(z - m) weights the bare codes and l = sum P 2^-ev is the softmax sum,
//    so pages of different scales share one accumulator and fp16 rounds relative to the largest weight.
//  * m only moves when a score exceeds it by more than 2^15 (fp16 has the room), which one vote per 16
//    keys decides; the common step has no shuffles.
//  * A producer warp streams tiles of 64 keys through a ring with bulk copies (a page and head is one
//    contiguous run of bytes), page ids and exponents fetched 32 segments at a time.
// Four warps share a tile (16 keys each); with more than 16 rows a second set of four takes the next 16.
// Each warp sums its own keys; the sums meet in shared memory once per item.
#pragma once

#include "kv_sched.cuh"

namespace qspec {
namespace att {

template <int D, int RG>
struct DecodeCfg {
  static constexpr int kRows = 16 * RG;
  static constexpr int kKeys = 64;
  static constexpr int kConsumers = 128 * RG;
  static constexpr int kThreads = kConsumers + 32;
  static constexpr int kCtas = RG == 1 ? 2 : 1;              // resident per SM
  static constexpr int kSide = kKeys * D;                    // bytes of a tile's keys or values
  static constexpr int kStages = (RG == 1 ? 4 : 8) * (128 / D);
  static constexpr int kRowPad = D + (D / 32) * 4 * (D == 128 ? 1 : 2);  // floats of a merge row: conflict-free
  static constexpr int kMerge = 4 * RG * 16 * kRowPad * 4;   // bytes
  static constexpr int kSmem = 128 + kStages * 2 * kSide + kMerge + kStages * 64 + 4096;
};

struct StageMeta {
  int ek[4], ev[4];  // per 16 keys; ek = kBadGroup: nothing there
};

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <int D, int RG>
__global__ void __launch_bounds__(DecodeCfg<D, RG>::kThreads, DecodeCfg<D, RG>::kCtas) decode_kernel(const AttArgs a) {
  using C = DecodeCfg<D, RG>;
  using namespace ptx;
  constexpr int kRows = C::kRows, kKeys = C::kKeys, kS = C::kStages, kSide = C::kSide, kPad = C::kRowPad;
  constexpr int kSteps = D / 16;   // k16 steps of a score
  constexpr int kTiles = D / 8;    // n8 tiles of the output
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = smem_raw + ((128u - (smem_u32(smem_raw) & 127u)) & 127u);
  float* merge = reinterpret_cast<float*>(ring + kS * 2 * kSide);  // [4 RG warps][16][kPad]
  StageMeta* meta = reinterpret_cast<StageMeta*>(merge + 4 * RG * 16 * kPad);
  uint64_t* full = reinterpret_cast<uint64_t*>(meta + kS);
  uint64_t* empty = full + kS;
  float2* ml = reinterpret_cast<float2*>(empty + kS);  // [4 RG][16] running maximum and sum of each warp's rows
  ScanShared* scan = reinterpret_cast<ScanShared*>(ml + 4 * RG * 16);
  volatile int* flags = reinterpret_cast<volatile int*>(scan + 1);  // abort, last to arrive, abort as the item ended
  int2* seq = reinterpret_cast<int2*>(scan + 1) + 2;
  volatile int* abort_flag = flags;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kS; ++i) {
      mbar_init(full + i, 1);
      mbar_init(empty + i, 4 * RG);
    }
    flags[0] = 0;
    fence_mbar_init();
  }
  grid_launch_dependents();
  grid_dependency_wait();
  Walk<kRows, kKeys> walk;
  share_out<C::kThreads>(a, seq, scan, walk);
  const long long run0 = walk.u;

  if (warp == 4 * RG) {
    // ------------------------------------------------------------------ producer
    const int seg_keys = min(a.c.page, kKeys), per_tile = kKeys / seg_keys;
    const uint32_t seg_bytes = seg_keys * D;
    int s = 0;
    while (walk.next()) {
      const Item& it = walk.it;
      SegBatch sb;
      for (int kt = it.kt0; kt < it.kt1; ++kt, ++s) {
        const int seg = kt * per_tile;
        if (sb.seg0 < 0 || seg >= sb.seg0 + 32) sb = load_segs(a, it, seg, seg_keys);
        const int st = s % kS;
        const bool ok = s < kS || wait_bar(empty + st, ((s / kS) - 1) & 1, abort_flag, a.err);
        if (!__all_sync(0xFFFFFFFFu, ok)) break;
        const int l0 = seg - sb.seg0;
        const bool mine = lane >= l0 && lane < l0 + per_tile && sb.page >= 0;
        if (lane < 4) meta[st].ek[lane] = kBadGroup;
        __syncwarp();
        if (mine) {
          const int g0 = (lane - l0) * (seg_keys / 16);
          for (int g = g0; g < g0 + seg_keys / 16; ++g) {
            meta[st].ek[g] = sb.ek;
            meta[st].ev[g] = sb.ev;
          }
        }
        const uint32_t who = __ballot_sync(0xFFFFFFFFu, mine);
        __syncwarp();
        if (lane == 0) mbar_arrive_expect_tx(full + st, __popc(who) * 2 * seg_bytes);
        __syncwarp();
        if (mine) {
          const long long key = static_cast<long long>(seg + lane - l0) * seg_keys;
          const int64_t at = ((static_cast<int64_t>(sb.page) * a.c.heads + it.head) * a.c.page + key % a.c.page) * D;
          uint8_t* dst = ring + st * 2 * kSide + (lane - l0) * seg_bytes;
          bulk_load(dst, a.c.k + at, seg_bytes, full + st);
          bulk_load(dst + kSide, a.c.v + at, seg_bytes, full + st);
        }
      }
      if (__any_sync(0xFFFFFFFFu, *abort_flag)) break;
    }
    // nothing may still be copying into shared memory when the CTA exits
    __syncwarp();
    for (int t = s > kS ? s - kS : 0; t < s; ++t) wait_bar_final(full + t % kS, (t / kS) & 1, a.err);
    return;
  }

  // -------------------------------------------------------------------- consumers
  const int g = lane >> 2, c = lane & 3;
  const int rg = warp >> 2, kw = warp & 3;  // row group, key group
  constexpr int kHalves = D / 64;
  int s = 0;
  while (walk.next()) {
    const Item& it = walk.it;
    // ---- query fragments and what each of the thread's two rows sees
    uint32_t qf[kSteps][4];
    float mult[2];
    int lim[2], low[2];
    unsigned long long bits[2];
    const int base = it.kv - it.n;
    bool odd[2];  // rows with a NaN or an infinity
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int row = rg * 16 + g + 8 * r;
      const bool there = row < it.rows;
      const int packed = it.row0 + (there ? row : 0);
      const int i = packed / a.group, hq = it.head * a.group + packed - i * a.group;
      const uint16_t* qp = a.q + static_cast<int64_t>(it.tok0 + i) * a.q_token + static_cast<int64_t>(hq) * D + 16 * c;
      uint32_t w[kHalves][8];
      uint32_t amax = 0;
#pragma unroll
      for (int h = 0; h < kHalves; ++h) {
        const uint4 x = there ? *reinterpret_cast<const uint4*>(qp + 64 * h) : make_uint4(0, 0, 0, 0);
        const uint4 y = there ? *reinterpret_cast<const uint4*>(qp + 64 * h + 8) : make_uint4(0, 0, 0, 0);
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
#pragma unroll
      for (int h = 0; h < kHalves; ++h)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const uint32_t f = odd[r] ? 0u : pack_f16(bf16_lo(w[h][e]) * shrink, bf16_hi(w[h][e]) * shrink);
          qf[4 * h + e / 2][r + 2 * (e & 1)] = f;
        }
      if (a.tree) {
        lim[r] = it.kv;
        low[r] = 0;
        bits[r] = there ? a.tree[it.tok0 + i] : 0ull;
      } else {
        lim[r] = min(max(base + i + 1, 0), it.kv);
        low[r] = a.window > 0 ? max(base + i + 1 - a.window, 0) : 0;
        bits[r] = 0;
      }
    }
    // positions that every row of the item sees: no masks there
    int all_lo, all_hi;
    {
      const int i0 = it.row0 / a.group, i1 = (it.row0 + it.rows - 1) / a.group;
      all_hi = a.tree ? max(base, 0) : min(max(base + i0 + 1, 0), it.kv);
      all_lo = a.window > 0 ? max(base + i1 + 1 - a.window, 0) : 0;
    }

    float o[kTiles][4];
#pragma unroll
    for (int j = 0; j < kTiles; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.0f;
    float m[2] = {kNoMax, kNoMax}, l[2] = {0.0f, 0.0f};

    for (int kt = it.kt0; kt < it.kt1; ++kt, ++s) {
      const int st = s % kS;
      const bool ok = __all_sync(0xFFFFFFFFu, wait_bar(full + st, (s / kS) & 1, abort_flag, a.err));
      const int ek = meta[st].ek[kw];
      const int key0 = kt * kKeys + 16 * kw;
      if (ok && ek != kBadGroup && key0 < it.hi && key0 + 16 > it.lo) {
        const int ev = meta[st].ev[kw];
        const uint8_t* kp = ring + st * 2 * kSide + (16 * kw + g) * D + 16 * c;
        float sc[2][2][4];  // [n tile][chain]
#pragma unroll
        for (int t = 0; t < 2; ++t) {
#pragma unroll
          for (int e = 0; e < 4; ++e) sc[t][0][e] = sc[t][1][e] = 0.0f;
#pragma unroll
          for (int h = 0; h < kHalves; ++h) {
            const uint4 x = *reinterpret_cast<const uint4*>(kp + 8 * t * D + 64 * h);
            const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int e = 0; e < 4; ++e)
              mma_f16(sc[t][e & 1], qf[4 * h + e], e4m3x2_to_f16x2(w[e]), e4m3x2_to_f16x2(w[e] >> 16));
          }
        }
        // ---- scores: element e of tile t is row g + 8 (e / 2), key key0 + 8 t + 2 c + (e & 1)
        float z[2][4];
        const float mk[2] = {score_mult(mult[0], ek), score_mult(mult[1], ek)};
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) z[t][e] = fmaf(sc[t][0][e] + sc[t][1][e], mk[e >> 1], static_cast<float>(ev));
        if (key0 + 16 > all_hi || key0 < all_lo) {
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int j = key0 + 8 * t + 2 * c + (e & 1), r = e >> 1;
              bool see = j < lim[r] && j >= low[r];
              if (a.tree && j >= base) see = see && j - base < 64 && (bits[r] >> (j - base) & 1ull);
              if (!see) z[t][e] = -INFINITY;
            }
        }
        const float top0 = fmaxf(fmaxf(z[0][0], z[0][1]), fmaxf(z[1][0], z[1][1]));
        const float top1 = fmaxf(fmaxf(z[0][2], z[0][3]), fmaxf(z[1][2], z[1][3]));
        if (__any_sync(0xFFFFFFFFu, top0 > m[0] + kSlack || top1 > m[1] + kSlack)) {
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            float top = r == 0 ? top0 : top1;
            top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
            const float m1 = fmaxf(m[r], top);
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
        uint32_t pf[4];
        {
          float p[2][4];
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) p[t][e] = ex2(z[t][e] - m[e >> 1]);
          const float unit = exp2_int(-ev);
          l[0] = fmaf(p[0][0] + p[0][1] + p[1][0] + p[1][1], unit, l[0]);
          l[1] = fmaf(p[0][2] + p[0][3] + p[1][2] + p[1][3], unit, l[1]);
          pf[0] = pack_f16(p[0][0], p[0][1]);
          pf[1] = pack_f16(p[0][2], p[0][3]);
          pf[2] = pack_f16(p[1][0], p[1][1]);
          pf[3] = pack_f16(p[1][2], p[1][3]);
        }
        // ---- values: channels [g * kTiles, + kTiles) of keys 2c, 2c + 1, 2c + 8, 2c + 9
        const uint8_t* vp = ring + st * 2 * kSide + kSide + (16 * kw + 2 * c) * D + g * kTiles;
        uint32_t v[4][kTiles / 4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint8_t* at = vp + ((k & 1) + 8 * (k >> 1)) * D;
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
        if (key0 + 16 > it.kv) {  // slots behind the end hold anything, NaN codes included
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (key0 + 2 * c + (k & 1) + 8 * (k >> 1) >= it.kv)
#pragma unroll
              for (int w = 0; w < kTiles / 4; ++w) v[k][w] = 0;
        }
#pragma unroll
        for (int w = 0; w < kTiles / 4; ++w) {
          // bytes (key 0, key 1) of two channels per word
          const uint32_t a0 = __byte_perm(v[0][w], v[1][w], 0x5140), a1 = __byte_perm(v[0][w], v[1][w], 0x7362);
          const uint32_t b0 = __byte_perm(v[2][w], v[3][w], 0x5140), b1 = __byte_perm(v[2][w], v[3][w], 0x7362);
          mma_f16(o[4 * w + 0], pf, e4m3x2_to_f16x2(a0), e4m3x2_to_f16x2(b0));
          mma_f16(o[4 * w + 1], pf, e4m3x2_to_f16x2(a0 >> 16), e4m3x2_to_f16x2(b0 >> 16));
          mma_f16(o[4 * w + 2], pf, e4m3x2_to_f16x2(a1), e4m3x2_to_f16x2(b1));
          mma_f16(o[4 * w + 3], pf, e4m3x2_to_f16x2(a1 >> 16), e4m3x2_to_f16x2(b1 >> 16));
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(empty + st);
      if (!ok) break;
    }

    // ---- the four key groups of each row meet in shared memory
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
    named_bar_sync(1, C::kConsumers);
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
    const long long end = walk.u1;
    if (it.ub < run0 || it.ue > end) {
      // ---- part of an item: leave it in the workspace; the last part to arrive adds all of them
      constexpr int kSlot = kRows * (D + 2);
      const int c0 = owner_of(it.ub, scan), c1 = owner_of(it.ue - 1, scan);
      float* slot = a.partial + (static_cast<int64_t>(blockIdx.x) * 2 + (it.ub >= run0 ? 1 : 0)) * kSlot;
      if (row < it.rows) {
#pragma unroll
        for (int k = 0; k < kChunks; ++k) *reinterpret_cast<float4*>(slot + row * D + 4 * (part + 8 * k)) = acc[k];
        if (part == 0) *reinterpret_cast<float2*>(slot + kRows * D + 2 * row) = make_float2(mm, ll);
      }
      __threadfence();
      named_bar_sync(1, C::kConsumers);
      if (threadIdx.x == 0) {
        const unsigned int n = static_cast<unsigned int>(c1 - c0);
        const bool last = atomicAdd(a.tickets + c0, 1u) == n;
        if (last) a.tickets[c0] = 0;
        flags[1] = last;
        flags[2] = *abort_flag;  // (one reading for all warps: they leave together)
      }
      named_bar_sync(1, C::kConsumers);
      done = flags[1] != 0;
      if (done && row < it.rows) {
        __threadfence();
        mm = kNoMax;
        for (int k = c0; k <= c1; ++k) {
          const float* p = a.partial + (static_cast<int64_t>(k) * 2 + (k == c0 ? 1 : 0)) * kSlot;
          mm = fmaxf(mm, __ldcg(p + kRows * D + 2 * row));
        }
        ll = 0.0f;
#pragma unroll
        for (int k = 0; k < kChunks; ++k) acc[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
        for (int k = c0; k <= c1; ++k) {
          const float* p = a.partial + (static_cast<int64_t>(k) * 2 + (k == c0 ? 1 : 0)) * kSlot;
          const float2 x = __ldcg(reinterpret_cast<const float2*>(p + kRows * D + 2 * row));
          const float f = ex2(x.x - mm);
          ll = fmaf(x.y, f, ll);
#pragma unroll
          for (int e = 0; e < kChunks; ++e) {
            const float4 v = __ldcg(reinterpret_cast<const float4*>(p + row * D + 4 * (part + 8 * e)));
            acc[e].x = fmaf(v.x, f, acc[e].x);
            acc[e].y = fmaf(v.y, f, acc[e].y);
            acc[e].z = fmaf(v.z, f, acc[e].z);
            acc[e].w = fmaf(v.w, f, acc[e].w);
          }
        }
      }
    } else {
      if (threadIdx.x == 0) flags[2] = *abort_flag;
      named_bar_sync(1, C::kConsumers);  // the merge buffer is read: the next item may fill it
    }
    if (flags[2]) break;
    if (done && row < it.rows) {
      const int packed = it.row0 + row, i = packed / a.group;
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
  }
}

}  // namespace att
}  // namespace qspec
