// Attention over the key/value cache for units of more than 32 query rows (of an
// e4m3 cache more than 16): tensor memory's lanes are query rows, 128 / kRep of them
// per CTA.  A unit of more than 128 rows (kPair: up to 256) belongs to two
// neighbouring CTAs, 128 rows each, which walk the same run of tiles side by side: the
// second finds K and V in L2.  (With the second 128 rows as units of their own further
// down the list, both halves of 61-token trees over 16 K bf16 keys read the cache from
// memory, and 125 us were twice its size at the memory's rate.)
//
// Per tile, as in the d = 128 forward kernel: S = Q K^T (128 x 128 keys) into one of
// two score buffers in tensor memory, softmax by two warpgroups (h owns keys
// [64h, 64h + 64) and its own m, l and accumulator O_h), P V from tensor memory.  With
// at most 64 (32) rows half (three quarters) of the lanes would idle, so Q is written
// kRep = 2 (4) times, once per lane block, and block i of a warpgroup's lanes takes
// only the i-th part of its 64 keys (the other parts of its P rows are zero): the
// exponentials spread over all warps, and each lane block ends with its own m, l and
// O, joined in the epilogue.  The tensor core's work does not grow.
//
// A tile takes about 1600 cycles (bf16, 61-token trees: 105 us, 56% of the memory's
// rate), the chain of a tile's scores, exponentials and products.
//
// e4m3: S from the bytes themselves, Q as an e4m3 and an e5m2 term.  P and V are f16:
// four more warps scale and convert V on its way, into two buffers of its own.  Its
// scales are taken relative to 2^k, the power of two below the tile's largest, and 2^k
// enters the exponents: the values are rounded twice by 2^-11, and a weight that f16
// cannot hold is off by 2^-24 of the row's largest (weight times scale).  A factor per
// key that every warp reads costs shared memory a cycle, so the softmax reads one (the
// score's): 512 cycles a tile, next to the products' 770, the copies' 256 and the
// conversion's 384; a tile takes 1900 to 2300.  With P as two e4m3 terms and three
// factors per key (value scales in the exponents) it was 3600.  Slow tiles, with drafted
// rows or scales more than 64 times apart, do read three: each key's scale stands in its
// own exponent, as in the other kernel, and V is converted as it is.  The loops are kept
// short: with the conversion and the scales' loop unrolled, warps waited for instructions
// three times as often as they issued one, and nothing else counted.
#pragma once

#include "fa_cache_fwd.cuh"

namespace fa {

// Writes kWords words of lane block `part` of kRep, zeros in the others'.
template <int kWords, int kRep>
__device__ __forceinline__ void store_part(uint32_t taddr, const uint32_t* r, int part) {
  uint32_t z[kWords];
#pragma unroll
  for (int i = 0; i < kWords; ++i) z[i] = 0u;
#pragma unroll
  for (int c = 0; c < kRep; ++c) {
    const uint32_t at = taddr + c * kWords;
    if (kRep == 1 || c == part) {  // warp-uniform
      if constexpr (kWords == 32) FA_TMEM_ST32(at, r);
      if constexpr (kWords == 16) FA_TMEM_ST16(at, r);
      if constexpr (kWords == 8) FA_TMEM_ST8(at, r);
    } else {
      if constexpr (kWords == 16) FA_TMEM_ST16(at, z);
      if constexpr (kWords == 8) FA_TMEM_ST8(at, z);
    }
  }
}

template <int kD, bool kE4m3_>
struct CacheRowsCfg : CacheTile<kD, kE4m3_> {
  static constexpr bool kE4m3 = kE4m3_;
  using T = CacheTile<kD, kE4m3>;
  // 128 to 160 KB of K and V in flight or in use per SM: the SM's share of the
  // memory bandwidth (23 bytes a cycle) times about 2000 cycles needs 47 KB
  static constexpr int kKStages = kE4m3 ? 65536 / T::kTileBytes : kD == 128 ? 3 : 5;
  static constexpr int kVStages = kE4m3 ? 32768 / T::kTileBytes : kD == 128 ? 2 : 5;
  static constexpr int kV16Bytes = 256 * kD;  // a V tile as f16
  // Q: 128 rows of bf16, or of two 8-bit terms; the epilogue joins lane blocks in it
  static constexpr int kQTerm = 128 * kD;  // bytes of one 8-bit term
  static constexpr int kOffQ = 0;
  static constexpr int kQBytes = 32768;
  static constexpr int kOffK = kQBytes;
  static constexpr int kOffV = kOffK + kKStages * T::kTileBytes;
  static constexpr int kOffV16 = kOffV + kVStages * T::kTileBytes;
  // e4m3: Q's rows on their way, four 16-byte pieces per softmax thread
  static constexpr int kOffStage = kOffV16 + (kE4m3 ? 2 * kV16Bytes : 0);
  static constexpr int kSmem = kOffStage + (kE4m3 ? 16384 : 0) + 1024;  // + alignment slack
  static constexpr int kTmemCols = 512;
  static constexpr uint32_t kColS = 0, kColO = 256;
  static constexpr int kProducerWarp = 8, kSIssuerWarp = 9, kPvIssuerWarp = 10;
  // 12 warps leave 168 registers each.  The last: bf16, V's producer (one warp for
  // K and V would hold back the next K behind a V whose stage is still in use);
  // e4m3, whose rings are deeper, the scaler.  e4m3 has four converting warps
  // behind them, and 128 registers.
  static constexpr int kLastWarp = 11, kConvertWarp = 12;
  static constexpr int kThreads = kE4m3 ? 512 : 384;
  // exponent of a row's largest weight when its reference is set, and how far above
  // that it may grow before the reference is set anew: f16 weights reach 2^14
  static constexpr float kTop = kE4m3 ? 6.f : 0.f;
  static constexpr float kGrow = 8.f;
  static_assert(2 * 128 * kD <= kQBytes, "Q fits its region");
};

// Bits e of keys key0 + e, e < kKeys, that token t of sequence b sees.
template <int kKeys>
__device__ __forceinline__ uint64_t visible_keys(const CacheFwdParams& p, int b, int start, int klen,
                                                 int t, int key0) {
  constexpr uint64_t kAll = kKeys == 64 ? ~0ull : (1ull << (kKeys & 63)) - 1;
  const int n = klen - key0;
  if (n <= 0) return 0;
  const uint64_t in = n >= kKeys ? kAll : (1ull << n) - 1;
  const int pre = start - key0;  // keys of the sequence itself
  if (pre >= kKeys) return in;
  if (!p.mask) {
    const int last = pre + t;  // >= -kKeys... the last visible key
    return last < 0 ? 0 : last >= 63 ? in : in & ((2ull << last) - 1);
  }
  const uint32_t* words = p.mask + ((long long)b * p.T + t) * p.W;
  uint64_t bits;
  if (pre > 0) {
    const uint64_t lo = words[0], hi = p.W > 1 ? words[1] : 0;
    bits = ((lo | hi << 32) << pre) | ((1ull << pre) - 1);
  } else {
    const int u = -pre, i = u >> 5, sh = u & 31;
    uint32_t x[3];
#pragma unroll
    for (int k = 0; k < 3; ++k) x[k] = i + k < p.W ? words[i + k] : 0u;
    bits = (uint64_t)__funnelshift_r(x[0], x[1], sh) |
           (uint64_t)__funnelshift_r(x[1], x[2], sh) << 32;
  }
  return in & bits;
}

// What the softmax warps share of a tile.
template <typename C, bool kE4m3>
struct RowsShared {
  // pv_done[h][x]: O_h has P_h V of buffer x's tile
  uint64_t p_full[2][2], pv_done[2][2], v_full[C::kVStages], v16_full[2], scl_empty[2];
  // per key of a tile: factor of its scores, value scale over 2^k (twice, as f16), and
  // in a slow tile (2^-k told as 0) the scale's log2 and inverse; per tile: k, 2^-k
  __align__(16) float scl[kE4m3 ? 2 : 1][4][kE4m3 ? 128 : 4];
  float k[2][2];
  int abort_flag, any_bad;
  uint32_t bad[32];  // drafted rows with non-finite values (T <= 1024)
};

// The softmax of one tile whose scores are there: S(n) to P, m, l and, where m grows,
// O_h.  token: of this thread's row, negative without one.  kSlow: an e4m3 tile whose
// value scales stand in the exponents, all with drafted rows or the sequence's end among
// them.  False after a wait that gave up.
template <typename C, bool kE4m3, int kRep, bool kSlow>
__device__ __forceinline__ bool tile_step(const CacheFwdParams& p, int b, int start, int klen, bool first,
                                          RowsShared<C, kE4m3>& sh, uint8_t* smem, int tile, int n,
                                          uint32_t tmem, float rowf, int token, float& m, float& l) {
  constexpr int kRows = 128 / kRep, kKeys = 64 / kRep;  // keys of a tile per softmax thread
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, h = warp >> 2, x = n & 1;
  const int part = (threadIdx.x & 127) / kRows;  // warp-uniform
  const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
  const uint32_t tO = tmem + C::kColO + C::D * h + lane_off;
  const uint32_t tS = tmem + C::kColS + 128 * x + 64 * h + lane_off;
  tc_fence_after();
  uint32_t r[kKeys];
  if constexpr (kKeys == 64) FA_TMEM_LD64_SYNC(tS, r);
  if constexpr (kKeys == 32) FA_TMEM_LD32_SYNC(tS + 32 * part, r);
  if constexpr (kKeys == 16) FA_TMEM_LD16_SYNC(tS + 16 * part, r);
  const int koff = 64 * h + kKeys * part;  // the thread's keys in the tile
  if constexpr (kE4m3) {
#pragma unroll
    for (int g = 0; g < kKeys; g += 4) {
      const float4 a = *reinterpret_cast<const float4*>(&sh.scl[kE4m3 ? x : 0][0][koff + g]);
      float2 t0 = mul2(make_float2(__uint_as_float(r[g]), __uint_as_float(r[g + 1])), make_float2(a.x, a.y));
      float2 t1 = mul2(make_float2(__uint_as_float(r[g + 2]), __uint_as_float(r[g + 3])), make_float2(a.z, a.w));
      if constexpr (kSlow) {  // the value scales stand in the exponents
        const float4 lv = *reinterpret_cast<const float4*>(&sh.scl[kE4m3 ? x : 0][2][koff + g]);
        t0 = fma2(t0, make_float2(rowf, rowf), make_float2(lv.x, lv.y));
        t1 = fma2(t1, make_float2(rowf, rowf), make_float2(lv.z, lv.w));
      }
      r[g] = __float_as_uint(t0.x);
      r[g + 1] = __float_as_uint(t0.y);
      r[g + 2] = __float_as_uint(t1.x);
      r[g + 3] = __float_as_uint(t1.y);
    }
  }
  if (kE4m3 ? kSlow : (tile + 1) * 128 > start) {  // drafted rows, and the sequence's end
    const uint64_t vis = token >= 0 ? visible_keys<kKeys>(p, b, start, klen, token, tile * 128 + koff) : ~0ull;
#pragma unroll
    for (int e = 0; e < kKeys; ++e)
      if (!((vis >> e) & 1)) r[e] = 0xff800000u;
    const int st = kE4m3 ? x : n % C::kVStages;
    const bool ok =
        kE4m3 ? cache_wait_warp(&sh.v16_full[x], (n >> 1) & 1, &sh.abort_flag, p.status, 2524)
              : cache_wait_warp(&sh.v_full[st], (n / C::kVStages) & 1, &sh.abort_flag, p.status, 2524);
    if (!ok) return false;
    const int row0 = 64 * h + 16 * (warp & 3);
    if (tile * 128 + row0 + 16 > start)
      clean_rows<C, 16, false, kE4m3>(
          smem + (kE4m3 ? C::kOffV16 + st * C::kV16Bytes : C::kOffV + st * C::kTileBytes), start, klen,
          row0, tile * 128, sh.bad, &sh.any_bad);
  }
  // the scale (positive) multiplies in the exponent; e4m3: the row's factor
  const float exp_scale = !kE4m3 ? p.scale_log2 : kSlow ? 1.f : rowf;
  const float k = kE4m3 && !kSlow ? sh.k[x][0] : 0.f;
  float tmax = __uint_as_float(r[0]);
  if constexpr (kKeys == 64) tmax = fmaxf(max32(r), max32(r + 32));
  if constexpr (kKeys == 32) tmax = max32(r);
  if constexpr (kKeys == 16) {
#pragma unroll
    for (int e = 1; e < 15; e += 2)
      tmax = max3(tmax, __uint_as_float(r[e]), __uint_as_float(r[e + 1]));
    tmax = fmaxf(tmax, __uint_as_float(r[15]));
  }
  const float top = tmax * exp_scale + (k - C::kTop);
  const bool grow = top > m + C::kGrow;  // true when m = -inf, top finite
  float alpha = 1.f;
  if (grow) {
    alpha = (m == -INFINITY) ? 0.f : ex2(m - top);
    m = top;
  }
  if (!first && __any_sync(0xffffffffu, grow)) {
    // O_h holds the tiles before this one once the last P_h V is done
    const bool ok = cache_wait_warp(&sh.pv_done[h][x ^ 1], ((n - 1) >> 1) & 1, &sh.abort_flag, p.status, 2525 + h);
    if (!ok) return false;
    tc_fence_after();
#pragma unroll 1
    for (int c = 0; c < C::D / 32; ++c) {
      uint32_t o[32];
      FA_TMEM_LD32_SYNC(tO + 32 * c, o);
#pragma unroll
      for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
      FA_TMEM_ST32(tO + 32 * c, o);
    }
  }
  const float nm = (m == -INFINITY) ? 0.f : k - m;
  const float2 c2 = make_float2(exp_scale, exp_scale), nm2 = make_float2(nm, nm);
  float2 acc[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
  // P rounded to bf16 (2^-8 of each weight), as in the forward kernels, or f16;
  // signalling its first half early, as the d = 128 forward does, gained nothing here
  uint32_t pk[kKeys / 2];
#pragma unroll
  for (int e = 0; e < kKeys; e += 4) {
    float4 inv = make_float4(1.f, 1.f, 1.f, 1.f);
    if constexpr (kE4m3 && kSlow)
      inv = *reinterpret_cast<const float4*>(&sh.scl[kE4m3 ? x : 0][3][koff + e]);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float2 s = make_float2(__uint_as_float(r[e + 2 * i]), __uint_as_float(r[e + 2 * i + 1]));
      const float2 t = fma2(s, c2, nm2);
      const float2 pv = make_float2(ex2(t.x), ex2(t.y));
      if constexpr (kE4m3 && kSlow)
        acc[i] = fma2(pv, i ? make_float2(inv.z, inv.w) : make_float2(inv.x, inv.y), acc[i]);
      else
        acc[i] = add2(acc[i], pv);
      pk[e / 2 + i] = kE4m3 ? pack_f16(pv.x, pv.y) : pack_bf16(pv.x, pv.y);
    }
  }
  store_part<kKeys / 2, kRep>(tS, pk, part);
  const float2 sum = add2(acc[0], acc[1]);
  l = l * alpha + (sum.x + sum.y) * (kE4m3 && !kSlow ? sh.k[x][1] : 1.f);
  tmem_wait_st();
  tc_fence_before();
  mbar_arrive_warp(&sh.p_full[x][h]);
  if (kE4m3 && lane == 0) mbar_arrive(&sh.scl_empty[x]);
  return true;
}

// The slow tiles' softmax, out of line: in the others' loop its code made long e4m3
// calls 15 % longer.
struct RowState {
  float m, l;
  bool ok;
};
template <typename C, int kRep>
__device__ __noinline__ RowState slow_tile(const CacheFwdParams& p, int b, int start, int klen, bool first,
                                           RowsShared<C, C::kE4m3>& sh, uint8_t* smem, int tile, int n,
                                           uint32_t tmem, float rowf, int token, float m, float l) {
  const bool ok = tile_step<C, C::kE4m3, kRep, C::kE4m3>(p, b, start, klen, first, sh, smem, tile, n, tmem,
                                                         rowf, token, m, l);
  return RowState{m, l, ok};
}

// The factors of four keys of a slow tile.
static __device__ __noinline__ void slow_factors(float* at, float4 v) {
  const float s[4] = {v.x, v.y, v.z, v.w};
  float a[4], b[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const KeyFactors f = key_factors(make_float2(0.f, s[e]), 0.f);
    a[e] = f.log2v;
    b[e] = f.inv;
  }
  const float one = __uint_as_float(0x3c003c00u);  // 1 twice, as f16
  *reinterpret_cast<float4*>(at + 128) = make_float4(one, one, one, one);
  *reinterpret_cast<float4*>(at + 256) = make_float4(a[0], a[1], a[2], a[3]);
  *reinterpret_cast<float4*>(at + 384) = make_float4(b[0], b[1], b[2], b[3]);
}

template <int kD, bool kE4m3, int kRep, bool kPair>
__global__ void __launch_bounds__(CacheRowsCfg<kD, kE4m3>::kThreads, 1)
    fa_cache_rows_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                        const __grid_constant__ CacheFwdParams p) {
  using C = CacheRowsCfg<kD, kE4m3>;
  constexpr int kRows = 128 / kRep;            // query rows of this CTA
  constexpr int kUnit = kPair ? 256 : kRows;   // of a unit
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  // A commit costs its thread some 200
  // cycles, so barriers that tell the same are one: k_empty[st] is a tile's scores done,
  // pv_done[1] a V buffer free where there are two.
  __shared__ RowsShared<C, kE4m3> sh;
  auto& p_full = sh.p_full;
  auto& pv_done = sh.pv_done;
  auto& v_full = sh.v_full;
  auto& scl_empty = sh.scl_empty;
  auto& v16_full = sh.v16_full;
  auto& abort_flag = sh.abort_flag;
  auto& s_scl = sh.scl;
  __shared__ uint64_t q_full, drain[2], scl_full[2];
  __shared__ uint64_t k_full[C::kKStages], k_empty[C::kKStages], v_empty[C::kVStages];
  __shared__ uint32_t tmem_slot;
  __shared__ float s_m[2][128], s_l[2][128], s_rowf[kE4m3 ? 128 : 1];

  // barriers and tensor memory need nothing of the kernel before
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    mbar_init(&q_full, 1);
    for (int x = 0; x < 2; ++x) mbar_init(&drain[x], 1);
    for (int x = 0; x < 2; ++x) {
      mbar_init(&scl_full[x], 1);
      mbar_init(&scl_empty[x], 12);  // softmax and converting warps
      mbar_init(&v16_full[x], 4);
      for (int h = 0; h < 2; ++h) {
        mbar_init(&p_full[x][h], 4);
        mbar_init(&pv_done[x][h], 1);
      }
    }
    for (int s = 0; s < C::kKStages; ++s) {
      mbar_init(&k_full[s], 1);
      mbar_init(&k_empty[s], 1);
    }
    for (int s = 0; s < C::kVStages; ++s) {
      mbar_init(&v_full[s], 1);
      mbar_init(&v_empty[s], kE4m3 ? 4 : 1);  // the converting warps; the P V issuer's commit
    }
    abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == C::kProducerWarp && lane == 0) {
    prefetch_tensormap(&tmK);
    prefetch_tensormap(&tmV);
  }
  if (warp == C::kSIssuerWarp) tmem_alloc(&tmem_slot, C::kTmemCols);
  pdl_wait();
  // kPair: CTAs 2i and 2i + 1 take the same run, 128 rows of each unit apiece
  const int base = kPair ? 128 * (blockIdx.x & 1) : 0;
  PieceWalk<kUnit> walk(p, kPair ? blockIdx.x >> 1 : blockIdx.x, kPair ? gridDim.x >> 1 : gridDim.x,
                        base);  // every warp follows the same list
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  pdl_launch_dependents();
  if (walk.left == 0) {
    if (warp == C::kSIssuerWarp) tmem_dealloc(tmem, C::kTmemCols);
    return;
  }
  const CacheRing kring{smem + C::kOffK, k_full, k_empty, &tmK};
  // whether a tile's V is free with its pv_done[1] (same count of buffers, same phases)
  constexpr bool kTwoV = kE4m3 || C::kVStages == 2;
  const CacheRing vring{smem + C::kOffV, v_full, !kE4m3 && kTwoV ? pv_done[1] : v_empty, &tmV};
  Piece w;

  if (warp == C::kProducerWarp) {
    cache_producer<C, true, kE4m3, 1>(p, walk, kring, vring, 0, &abort_flag, 2501, [](const Piece&) {},
                                   [](const Piece&, int) { return true; });
  } else if (!kE4m3 && warp == C::kLastWarp) {
    cache_producer<C, false, true, 1>(p, walk, kring, vring, 0, &abort_flag, 2501, [](const Piece&) {},
                                   [](const Piece&, int) { return true; });
  } else if (warp == C::kSIssuerWarp) {
    // ------------------------------------------------------------ S issuer
    if (lane == 0) {
      const uint32_t sQ = smem_addr(smem + C::kOffQ), sK = smem_addr(smem + C::kOffK);
      bool ok = true;
      int n = 0;
      for (int piece = 0; ok && walk.next(w); ++piece) {
        ok = cache_wait(&q_full, piece & 1, &abort_flag, p.status, 2511);
        for (int tile = w.t0; ok && tile < w.t1; ++tile, ++n) {
          const int st = n % C::kKStages, x = n & 1;
          ok = cache_wait(&k_full[st], (n / C::kKStages) & 1, &abort_flag, p.status, 2512);
          // S(n) overwrites buffer x, where P of tile n - 2 sits
          if (ok && n >= 2) ok = cache_wait(&pv_done[0][x], ((n - 2) >> 1) & 1, &abort_flag, p.status, 2513);
          if (ok && n >= 2) ok = cache_wait(&pv_done[1][x], ((n - 2) >> 1) & 1, &abort_flag, p.status, 2514);
          if (!ok) break;
          tc_fence_after();
          const uint32_t k = sK + st * C::kTileBytes, tS = tmem + C::kColS + 128 * x;
          if constexpr (kE4m3) {
#pragma unroll
            for (int term = 0; term < 2; ++term) {
              const uint32_t idesc = idesc_e4m3(128, 128, false, false, term > 0);
#pragma unroll
              for (int ks = 0; ks < C::D / 32; ++ks) {
                const uint32_t a = sQ + term * C::kQTerm + 32 * ks, b = k + 32 * ks;
                mma8_ss(tS, C::D == 64 ? sdesc_sw64(a) : sdesc_sw128(a, 16, 1024),
                        C::D == 64 ? sdesc_sw64(b) : sdesc_sw128(b, 16, 1024), idesc,
                        term + ks > 0 ? 1u : 0u);
              }
            }
          } else {
            constexpr uint32_t idesc = idesc_bf16(128, 128, false, false);
            const uint64_t dQ = sdesc_sw128(sQ, 16, 1024), dK = sdesc_sw128(k, 16, 1024);
#pragma unroll
            for (int ks = 0; ks < C::D / 16; ++ks) {
              const uint32_t off = ((ks >> 2) * C::kChunkBytes + (ks & 3) * 32) >> 4;
              mma_ss(tS, dQ + off, dK + off, idesc, ks > 0 ? 1u : 0u);
            }
          }
          mma_commit(&k_empty[st]);
        }
      }
      mma_commit(&drain[0]);
      mbar_drain(&drain[0], 0);
    }
  } else if (warp == C::kPvIssuerWarp) {
    // ------------------------------------------------------------ P_h V issuer
    if (lane == 0) {
      const uint32_t sV = smem_addr(smem + (kE4m3 ? C::kOffV16 : C::kOffV));
      constexpr int kStages = kE4m3 ? 2 : C::kVStages, kBytes = kE4m3 ? C::kV16Bytes : C::kTileBytes;
      uint64_t* const full = kE4m3 ? v16_full : v_full;
      bool ok = true;
      int n = 0;
      while (ok && walk.next(w)) {
        for (int tile = w.t0; ok && tile < w.t1; ++tile, ++n) {
          const int st = n % kStages, x = n & 1;
          const uint32_t first = tile == w.t0 ? 0u : 1u;
          ok = cache_wait(&full[st], (n / kStages) & 1, &abort_flag, p.status, 2515);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (ok) ok = cache_wait(&p_full[x][h], (n >> 1) & 1, &abort_flag, p.status, 2516 + h);
            if (!ok) break;
            tc_fence_after();
            const uint32_t tO = tmem + C::kColO + C::D * h, tP = tmem + C::kColS + 128 * x + 64 * h;
            constexpr uint32_t idesc =
                kE4m3 ? idesc_f16(128, C::D, false, true) : idesc_bf16(128, C::D, false, true);
            const uint64_t dV = sdesc_sw128(sV + st * kBytes, 16384, 1024);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma_ts(tO, tP + 8 * kk, dV + (4 * h + kk) * (2048 >> 4), idesc, kk > 0 ? 1u : first);
            mma_commit(&pv_done[h][x]);
            if (!kTwoV && h == 1) mma_commit(&v_empty[st]);
          }
        }
      }
      mma_commit(&drain[1]);
      mbar_drain(&drain[1], 0);
    }
  } else if (kE4m3 && warp >= C::kConvertWarp) {
    // ------------------------------------------------------------ converters
    // V's bytes to f16, 32 rows per warp, 8 at a time; a lane has 16 bytes of each of
    // its kU rows.  Which half of them it takes first is chosen so that neither its
    // 8-byte loads nor its 16-byte stores meet others' in a bank.
    constexpr int kLanes = C::D / 16, kPer = 32 / kLanes, kU = 8 / kPer;
    const int j = lane % kLanes;
    uint32_t from[kU], to[kU], half[kU];
    int row[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      row[u] = 32 * (warp - C::kConvertWarp) + u * kPer + lane / kLanes;
      half[u] = C::D == 128 ? (j >> 2) ^ (row[u] & 1) : (row[u] >> 1) & 1;
      from[u] = e4m3_row_offset<C::D>(row[u], 2 * j);
      to[u] = (j >> 2) * 16384 + sw128_offset(row[u], 16 * (j & 3));
    }
    bool ok = true;
    int n = 0, st = 0;
    uint32_t parity = 0;
    while (ok && walk.next(w)) {
#pragma unroll 1
      for (int tile = w.t0; tile < w.t1; ++tile, ++n) {
        const int x = n & 1;
        ok = cache_wait_warp(&v_full[st], parity, &abort_flag, p.status, 2541) &&
             cache_wait_warp(&scl_full[x], (n >> 1) & 1, &abort_flag, p.status, 2543) &&
             cache_wait_warp(&pv_done[1][x], ((n >> 1) & 1) ^ 1, &abort_flag, p.status, 2542);
        if (!ok) break;
        const uint8_t* src = smem + C::kOffV + st * C::kTileBytes;
        uint8_t* dst = smem + C::kOffV16 + x * C::kV16Bytes;
        const float* scale = s_scl[kE4m3 ? x : 0][1];
#pragma unroll 1
        for (int i = 0; i < 4; ++i, src += 8 * C::D, dst += 1024, scale += kE4m3 ? 8 : 0) {
          uint2 v[kU][2];
          uint32_t s[kU];
#pragma unroll
          for (int u = 0; u < kU; ++u) {
            v[u][0] = *reinterpret_cast<const uint2*>(src + from[u] + 8 * half[u]);
            v[u][1] = *reinterpret_cast<const uint2*>(src + from[u] + 8 * (half[u] ^ 1));
            s[u] = __float_as_uint(scale[kE4m3 ? row[u] : 0]);
          }
#pragma unroll
          for (int u = 0; u < kU; ++u)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              *reinterpret_cast<uint4*>(dst + (to[u] ^ (16 * (half[u] ^ e)))) =
                  make_uint4(scaled_f16(v[u][e].x, s[u]), scaled_f16(v[u][e].x >> 16, s[u]),
                             scaled_f16(v[u][e].y, s[u]), scaled_f16(v[u][e].y >> 16, s[u]));
        }
        mbar_arrive_warp(&v_empty[st]);
        if (lane == 0) mbar_arrive(&scl_empty[x]);
        fence_proxy_async_smem();
        mbar_arrive_warp(&v16_full[x]);
        if (++st == C::kVStages) {
          st = 0;
          parity ^= 1;
        }
      }
    }
  } else if (kE4m3 && warp == C::kLastWarp) {
    // ------------------------------------------------------------ scaler
    // turns a tile's scales into the two factors per key, two tiles ahead of the
    // softmax at most; lane i's keys are 4i .. 4i + 3 (one page: its size is a
    // multiple of 4).  The scales are read a tile, their page two tiles ahead.
    bool ok = true;
    int n = 0;
    while (ok && walk.next(w)) {
      float4 sk, sv;
      int key = w.t0 * 128 + 4 * lane;
      key_scales4(p.c, w, key, key_page(p.c, w, key), &sk, &sv);
      int page = key_page(p.c, w, key + 128);
#pragma unroll 1
      for (int tile = w.t0; tile < w.t1; ++tile, ++n, key += 128) {
        const int x = n & 1;
        ok = cache_wait_warp(&scl_empty[x], ((n >> 1) & 1) ^ 1, &abort_flag, p.status, 2533);
        if (!ok) break;
        const float k4[4] = {sk.x, sk.y, sk.z, sk.w};
        const float v4[4] = {sv.x, sv.y, sv.z, sv.w};
        float a[4], v[4];
        uint32_t most = 0, least = 0x7f800000u;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const bool in = key + e < w.klen;  // else: whatever the page holds
          a[e] = in ? k4[e] * p.scale_log2 : 0.f;
          v[e] = in ? v4[e] : 0.f;
          const uint32_t bits = __float_as_uint(fmaxf(v[e], 0.f));  // ordered as the values
          if (v[e] < INFINITY) most = max(most, bits);
          least = min(least, bits);
        }
        most = __reduce_max_sync(0xffffffffu, most);
        least = __reduce_min_sync(0xffffffffu, least);
        float* const at = &s_scl[kE4m3 ? x : 0][0][kE4m3 ? 4 * lane : 0];
        *reinterpret_cast<float4*>(at) = make_float4(a[0], a[1], a[2], a[3]);
        // the largest scale becomes 64 to 128: times 448 it is below f16's 65504
        int k = max((int)(most >> 23) - 133, -64);
        float down = __uint_as_float((uint32_t)(127 - k) << 23);
        // Drafted rows' scales must not reach the rows that do not see them, as they
        // would through k; and where the key of k's scale is not the one that counts, k
        // would raise the rows' references and push the other tiles' weights below what
        // f16 holds.  Such tiles keep their values as they are (f16 holds e4m3) and every
        // scale in its key's exponent.
        if ((tile + 1) * 128 > w.start || __uint_as_float(most) > 64.f * __uint_as_float(least)) {
          slow_factors(at, make_float4(v[0], v[1], v[2], v[3]));
          k = 0;
          down = 0.f;
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            // (scales that are not finite: not this far)
            const float s = fmaxf(fminf(v[e] * down, 128.f), 0.f);
            v[e] = __uint_as_float(pack_f16(s, s));
          }
          *reinterpret_cast<float4*>(at + (kE4m3 ? 128 : 0)) = make_float4(v[0], v[1], v[2], v[3]);
        }
        if (lane < 2) sh.k[x][lane] = lane ? down : (float)k;
        mbar_arrive_warp(&scl_full[x]);
        key_scales4(p.c, w, key + 128, page, &sk, &sv);
        page = key_page(p.c, w, key + 256);
      }
    }
  } else {
    // ------------------------------------------------------------ softmax
    const int h = warp >> 2;  // key half
    const int tq = tid & 127;
    const int row = tq & (kRows - 1);
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    // After a wait that gave up, a warp still passes every barrier of its piece
    // (the others may be waiting there); the piece's last barrier stops all.
    bool ok = true;
    int n = 0;
    while (walk.next(w)) {
      // ---- Q of the unit, kRep times: 16 (D = 64: 8) lanes per row
      if (tid < 32) sh.bad[tid] = 0u;
      if (tid == 0) sh.any_bad = 0;
      {
        // The loops are not unrolled: these are a call's first instructions, and
        // fetching them takes longer than the loads.
        constexpr int kLanes = C::D / 8, kPer = 32 / kLanes, kSteps = kRows / (8 * kPer);
        const int c8 = lane % kLanes;
        auto q_row = [&](int i) { return (8 * i + warp) * kPer + lane / kLanes; };
        auto q_copy = [&](int i, uint8_t* dst) {
          const int r = q_row(i), g = w.rt * kUnit + base + r;
          const int t = row_token(p, g), hq = w.h * p.group + g - t * p.group;
          const bool in = base + r < w.rows;
          const __nv_bfloat16* const src = p.q + (in ? row_offset(p.lq, w.b, hq, t) + 8 * c8 : 0);
          copy16(dst, src, in);
        };
        if constexpr (kE4m3) {
          uint8_t* const stage = smem + C::kOffStage + 16 * tid;  // 4 KB per piece
          constexpr int kAhead = kSteps < 4 ? kSteps : 4;
#pragma unroll 1
          for (int i = 0; i < kAhead; ++i) {
            q_copy(i, stage + 4096 * i);
            asm volatile("cp.async.commit_group;" ::: "memory");
          }
#pragma unroll 1
          for (int i = 0; i < kSteps; ++i) {
            asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 1) : "memory");
            uint8_t* const mine = stage + 4096 * (i % kAhead);
            const SplitQ f = split_q<kLanes, false>(*reinterpret_cast<const uint4*>(mine));
            if (i + kAhead < kSteps) q_copy(i + kAhead, mine);  // read by this thread alone
            asm volatile("cp.async.commit_group;" ::: "memory");
            const int r = q_row(i);
#pragma unroll
            for (int c = 0; c < kRep; ++c) {
              const int rr = r + c * kRows;
              uint8_t* at = smem + C::kOffQ + e4m3_row_offset<C::D>(rr, c8);
              *reinterpret_cast<uint2*>(at) = f.hi;
              *reinterpret_cast<uint2*>(at + C::kQTerm) = f.lo;
              if (c8 == 0) s_rowf[kE4m3 ? rr : 0] = f.factor;
            }
          }
        } else {
#pragma unroll 1
          for (int i = 0; i < kSteps * kRep; ++i) {
            const int r = q_row(i % kSteps) + i / kSteps * kRows;
            q_copy(i % kSteps, smem + C::kOffQ + (c8 >> 3) * C::kChunkBytes + sw128_offset(r, (c8 & 7) * 8));
          }
          asm volatile("cp.async.wait_all;" ::: "memory");
        }
      }
      fence_proxy_async_smem();
      asm volatile("bar.sync 1, 256;" ::: "memory");
      if (tid == 0) mbar_arrive(&q_full);
      const float rowf = kE4m3 ? s_rowf[kE4m3 ? tq : 0] : 1.f;
      const int token = base + row < w.rows ? row_token(p, w.rt * kUnit + base + row) : -1;

      float m = -INFINITY, l = 0.f;
      for (int tile = w.t0; tile < w.t1; ++tile, ++n) {
        const int x = n & 1;
        bool slow = false;
        if (kE4m3) {  // (there long before the scores)
          ok = cache_wait_warp(&scl_full[x], (n >> 1) & 1, &abort_flag, p.status, 2523);
          slow = sh.k[x][1] == 0.f;
        }
        // (the phase stays until S(n + kKStages), behind this tile's P)
        if (ok)
          ok = cache_wait_warp(&k_empty[n % C::kKStages], (n / C::kKStages) & 1, &abort_flag, p.status,
                               2521 + h);
        if (!ok) break;
        if (slow) {
          const RowState y = slow_tile<C, kRep>(p, w.b, w.start, w.klen, tile == w.t0, sh, smem, tile, n,
                                                tmem, rowf, token, m, l);
          m = y.m;
          l = y.l;
          ok = y.ok;
        } else {
          ok = tile_step<C, kE4m3, kRep, false>(p, w.b, w.start, w.klen, tile == w.t0, sh, smem, tile, n, tmem,
                                                rowf, token, m, l);
        }
        if (!ok) break;
      }

      // ---- epilogue: join the two key halves and the lane blocks
      const int xl = (n - 1) & 1;
      if (ok)
        ok = cache_wait_warp(&pv_done[0][xl], ((n - 1) >> 1) & 1, &abort_flag, p.status, 2527) &&
             cache_wait_warp(&pv_done[1][xl], ((n - 1) >> 1) & 1, &abort_flag, p.status, 2528);
      tc_fence_after();
      s_m[h][tq] = m;
      s_l[h][tq] = l;
      asm volatile("bar.sync 1, 256;" ::: "memory");
      // maximum and sum of query row r over its 2 kRep parts
      auto row_max = [&](int r) {
        float mm = -INFINITY;
#pragma unroll
        for (int c = 0; c < kRep; ++c) mm = fmaxf(mm, fmaxf(s_m[0][r + c * kRows], s_m[1][r + c * kRows]));
        return mm;
      };
      auto weight = [&](float mi, float mm) { return mi == -INFINITY ? 0.f : ex2(mi - mm); };
      const float mrow = row_max(row);
      const float w0 = weight(s_m[0][tq], mrow), w1 = weight(s_m[1][tq], mrow);
      // this thread writes columns cg .. cg + 32 / kRep of row orow of each chunk
      constexpr int kCols = 32 / kRep;
      const int orow = tq / kRep, cg = (tq % kRep) * kCols;
      const float mout = row_max(orow);
      float lout = 0.f;
#pragma unroll
      for (int i = 0; i < 2 * kRep; ++i) {
        const int at = orow + (i >> 1) * kRows;
        lout += s_l[i & 1][at] * weight(s_m[i & 1][at], mout);
      }
      const bool empty = lout == 0.f;
      const float inv = empty ? 0.f : 1.f / lout;
      const int urow = base + orow;  // row of the unit
      const bool write = ok && urow < w.rows;
      const int g = w.rt * kUnit + urow, t = row_token(p, g), hq = w.h * p.group + g - t * p.group;
      float* const slot = w.slot < 0 ? nullptr : p.ws + (size_t)w.slot * slot_floats<kD, kUnit>();
      float* const red = reinterpret_cast<float*>(smem + C::kOffQ) + h * 128 * 32;
#pragma unroll 1
      for (int c = 0; c < C::D / 64; ++c) {
        const int col = (C::D / 2) * h + 32 * c;
        // lanes that write nothing must not run ahead to the next (warp-wide) load
        __syncwarp();
        uint32_t r0[32], r1[32];
        if (ok) {  // warp-uniform
          FA_TMEM_LD32_SYNC(tmem + C::kColO + col + lane_off, r0);
          FA_TMEM_LD32_SYNC(tmem + C::kColO + C::D + col + lane_off, r1);
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) r0[e] = r1[e] = 0u;
        }
        float v[32];
#pragma unroll
        for (int e = 0; e < 32; ++e)
          v[e] = __uint_as_float(r0[e]) * w0 + __uint_as_float(r1[e]) * w1;
        if constexpr (kRep > 1) {
          // row tq of 32 floats, its 16-byte pieces XORed with the row
#pragma unroll
          for (int i = 0; i < 8; ++i)
            *reinterpret_cast<float4*>(red + tq * 32 + 4 * (i ^ (tq & 7))) =
                make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
          asm volatile("bar.sync %0, 128;" ::"r"(2 + h) : "memory");
#pragma unroll
          for (int i = 0; i < kCols / 4; ++i) {
            float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int k = 0; k < kRep; ++k) {
              const int at = orow + k * kRows;
              const float4 y = *reinterpret_cast<const float4*>(
                  red + at * 32 + 4 * ((cg / 4 + i) ^ (at & 7)));
              s.x += y.x; s.y += y.y; s.z += y.z; s.w += y.w;
            }
            v[4 * i] = s.x; v[4 * i + 1] = s.y; v[4 * i + 2] = s.z; v[4 * i + 3] = s.w;
          }
          asm volatile("bar.sync %0, 128;" ::"r"(2 + h) : "memory");
        }
        if (write) {
          if (sh.any_bad) {
            float extra[kCols];
#pragma unroll
            for (int e = 0; e < kCols; ++e) extra[e] = 0.f;
            add_nonfinite<kE4m3>(p, w.b, w.h, w.start, sh.bad, t, col + cg, kCols, extra);
#pragma unroll
            for (int e = 0; e < kCols; ++e) v[e] += extra[e];
          }
          if (slot) {
            float4* dst = reinterpret_cast<float4*>(slot + urow * C::D + col + cg);
#pragma unroll
            for (int i = 0; i < kCols / 4; ++i)
              dst[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
          } else {
            uint4* dst = reinterpret_cast<uint4*>(p.o + row_offset(p.lo, w.b, hq, t) + col + cg);
#pragma unroll
            for (int e = 0; e < kCols; ++e) v[e] *= inv;
#pragma unroll
            for (int i = 0; i < kCols / 8; ++i) dst[i] = pack8(v + 8 * i);
          }
        }
      }
      if (write && h == 0 && cg == 0) {
        if (slot) {
          slot[kUnit * C::D + urow] = mout;
          slot[kUnit * C::D + kUnit + urow] = lout;
        } else {
          p.lse[((size_t)w.b * p.Hq + hq) * p.T + t] =
              empty ? -INFINITY : (mout + log2f(lout)) * kLn2;
        }
      }
      // the accumulators, the statistics and the Q region are read: the next
      // unit may overwrite them
      tc_fence_before();
      if (barrier_any(1, 256, !ok)) break;
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == C::kSIssuerWarp) {
    __syncwarp();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

template <bool kE4m3>
cudaError_t launch_cache_rows(const CacheMaps& m, const CacheFwdParams& p, cudaStream_t s) {
  const int rows = cache_fwd_rows(p.T * p.group);
  auto go = [&](auto d) {
    constexpr int kD = decltype(d)::value;
    using C = CacheRowsCfg<kD, kE4m3>;
    if constexpr (kE4m3)
      if (rows == 32)
        return launch_cache_pair<kD, 32, fa_cache_rows_kernel<kD, kE4m3, 4, false>>(C::kThreads, C::kSmem, 1, m, p, s);
    return rows == 64 ? launch_cache_pair<kD, 64, fa_cache_rows_kernel<kD, kE4m3, 2, false>>(C::kThreads, C::kSmem, 1, m, p, s)
           : rows == 128
               ? launch_cache_pair<kD, 128, fa_cache_rows_kernel<kD, kE4m3, 1, false>>(C::kThreads, C::kSmem, 1, m, p, s)
               : launch_cache_pair<kD, 256, fa_cache_rows_kernel<kD, kE4m3, 1, true>>(C::kThreads, C::kSmem, 2, m, p, s);
  };
  return p.c.d == 64 ? go(std::integral_constant<int, 64>{}) : go(std::integral_constant<int, 128>{});
}

}  // namespace fa
