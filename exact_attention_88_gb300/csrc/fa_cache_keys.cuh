// Attention over the key/value cache for units of up to 32 query rows, of an e4m3
// cache up to 16 (single tokens, small trees): tensor memory's lanes are keys, its columns query rows.
//
//   S^T = K Q^T   (M = 128 keys, N = the rows; A = the K tile as TMA wrote it)
//   P'  = 2^(S - m)   one key per thread, its rows in registers
//   O^T += V^T P^T    (M = d, N = the rows; A = the V tile read transposed)
// With query rows as M, as in the forward kernels, a few rows would still cost
// the tensor core 128 x 128 products and the softmax warps idle lanes; here a
// product with N <= 32 takes 44 cycles per 4 KB of tile (its reads from shared
// memory), 350 cycles per e4m3 tile and 700 per bf16 tile of d = 128, and every
// softmax thread has a key.  The memory needs 1400 and 2800 cycles for them.
//
// kG groups of four warps take the tiles in turn.  A group is on its own: two of its
// threads issue its products (one S, one P V: by one thread they took 1700 of a tile's
// 4500 cycles, and d = 64 e4m3 tiles 8 % more), it has its reference m and sum l per row,
// its score and P buffer and its accumulators.  A tile's chain (S, scores, vote,
// exponentials, P, P V) is some 3000 cycles of latency; four groups (two beyond 16
// rows, whose registers do not suffice for more, and for bf16 at d = 128, which
// needs no more) overlap theirs.  Issuing from one warp for all groups instead cost
// 1450 cycles a tile in waits and commits alone.
// A reference belongs to all 128 keys of a group, so it cannot follow each
// thread's maximum: it stays until some score passes it by kGrow (one vote per
// tile), and only then are the rows' maxima formed (warp reductions, joined in
// shared memory), the references raised and the accumulator's columns rescaled.  A
// row that has seen no key yet has reference -2^128 (kept negated): its first
// visible key raises it.
// P goes to shared memory (keys contiguous: the B operand), one element (e4m3: three
// terms, two keys' bytes of each) per thread and row.
// At the end of a piece each group leaves its m and l in shared memory, and the
// group of the last tile joins the accumulators of all; the others go on with the
// next piece (statistics and accumulators are double-buffered by piece).
// At d = 64 the V tile is read as if it had two equal halves (the stride between
// them is 0), so lanes 64..127 of O^T repeat lanes 0..63.
//
// Roles: warps 0 .. 4 kG - 1 softmax, then four that load K and V (TMA) and a
// quarter of Q's rows each (two buffers).  A load costs its warp 400 cycles, 900 for
// eight pages of 16 rows, and another 400 per tile; an e4m3 tile's memory time is
// 700 (d = 64) or 1400.  So each of the four loads K and V for one group, or (two
// groups) K or V for one; one warp each for K and V bound d = 64 and small pages.
// A softmax thread reads its key's scales from global memory itself, a tile of its
// group ahead, and their page two tiles ahead: as TMA boxes they cost the producers as
// much as the data.
#pragma once

#include "fa_cache_fwd.cuh"

namespace fa {

template <int kD, bool kE4m3, int kR>
struct CacheKeysCfg : CacheTile<kD, kE4m3> {
  using T = CacheTile<kD, kE4m3>;
  // columns of S^T: the rows (at least the 16 of an MMA), or two e4m3 terms of each;
  // of O^T: the same, or three e5m2 terms (24 make it 32: a multiple of 16)
  static constexpr int kN = kE4m3 ? 2 * kR : (kR < 16 ? 16 : kR);
  static constexpr int kNO = kE4m3 ? (3 * kR + 15) / 16 * 16 : kN;
  static constexpr int kQBytes = kN * T::kRowBytes < 1024 ? 1024 : kN * T::kRowBytes;
  static constexpr int kPRow = kE4m3 ? 128 : 256;  // bytes of a row of P: 128 keys
  static constexpr int kPBytes = kNO * kPRow;
  // softmax groups: bf16 tiles of d = 128 take the memory longer than one group
  // takes for two
  static constexpr int kG = kR <= 16 && T::kTileBytes < 32768 ? 4 : 2;
  // A multiple of kG stages each, so that a stage serves one group: only a waiter
  // that has seen a barrier's last phase can tell the next by its parity.  128 KB
  // in flight or in use per SM; the SM's share of the memory bandwidth (23 bytes a
  // cycle) times about 2000 cycles needs 47 KB.
  static constexpr int kKStages = 65536 / T::kTileBytes, kVStages = kKStages;
  static_assert(kKStages % kG == 0, "");
  static constexpr int kOffQ = 0;              // two buffers
  static constexpr int kOffP = kOffQ + 2 * kQBytes;
  static constexpr int kOffK = kOffP + kG * kPBytes;
  static constexpr int kOffV = kOffK + kKStages * T::kTileBytes;
  static constexpr int kSmem = kOffV + kVStages * T::kTileBytes + 1024;  // + alignment slack
  static constexpr int kTmemCols = 512;
  // scores of group e at kN e; accumulator of group e in pieces of parity y at
  // kColO + kNO (e + kG y)
  static constexpr uint32_t kColS = 0, kColO = 128;
  // exponent of a row's largest weight when its reference is set, and how far above
  // that it may grow before the reference is set anew: 2^8 (bf16), 2^15.75 = 55000 of
  // e5m2's 57344
  static constexpr float kTop = kE4m3 ? 13.f : 0.f;
  static constexpr float kGrow = kE4m3 ? 2.75f : 8.f;
  static constexpr int kProducerWarp = 4 * kG;  // the first of four
  static constexpr int kThreads = 32 * (kProducerWarp + 4);
  static_assert(kN * kG <= 128 && 2 * kNO * kG <= 384 && kQBytes % 1024 == 0 && kPBytes % 1024 == 0, "");
};

// negated reference of a row that has seen no key: the largest float, so that every
// score raises it
constexpr float kUnset = 0x1.fffffep127f;

__device__ __forceinline__ float warp_max(float x) {
  float y;
  asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}

#define FA_TMEM_LD8_SYNC(taddr, r)                                                             \
  asm volatile(                                                                                \
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n"               \
      "tcgen05.wait::ld.sync.aligned;"                                                         \
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),   \
        "=r"(r[7])                                                                             \
      : "r"(taddr)                                                                             \
      : "memory")

// Sums of kR values over the warp: lane i (mod kR) gets value i's.  Each step
// halves the values a lane holds instead of reducing every value by itself.
template <int kR>
__device__ __forceinline__ float sum_to_lanes(float* v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int h = kR / 2; h >= 1; h >>= 1) {
#pragma unroll
    for (int i = 0; i < h; ++i) {
      const bool up = (lane & h) != 0;
      const float give = up ? v[i] : v[i + h];
      v[i] = (up ? v[i + h] : v[i]) + __shfl_xor_sync(0xffffffffu, give, h);
    }
  }
  float s = v[0];
#pragma unroll
  for (int o = kR; o < 32; o <<= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}

// S^T = K Q^T of one tile, by one thread.  `done`, which frees the K tile, tells the
// softmax too: a commit costs its thread some 200 cycles.
template <typename C, bool kE4m3>
__device__ __noinline__ void issue_scores(uint32_t tS, uint32_t k, uint32_t q, uint64_t* done) {
  tc_fence_after();
  if constexpr (kE4m3) {
    constexpr uint32_t idesc = idesc_e4m3(128, C::kN, false, false);
    const uint64_t dk = C::D == 64 ? sdesc_sw64(k) : sdesc_sw128(k, 16, 1024);
    const uint64_t dq = C::D == 64 ? sdesc_sw64(q) : sdesc_sw128(q, 16, 1024);
#pragma unroll
    for (int ks = 0; ks < C::D / 32; ++ks)  // 32 bytes on
      mma8_ss(tS, dk + 2 * ks, dq + 2 * ks, idesc, ks > 0 ? 1u : 0u);
  } else {
    constexpr uint32_t idesc = idesc_bf16(128, C::kN, false, false);
    const uint64_t dk = sdesc_sw128(k, 16, 1024), dq = sdesc_sw128(q, 16, 1024);
#pragma unroll
    for (int ks = 0; ks < C::D / 16; ++ks)
      mma_ss(tS, dk + (((ks >> 2) * C::kChunkBytes + (ks & 3) * 32) >> 4),
             dq + (((ks >> 2) * C::kN * 128 + (ks & 3) * 32) >> 4), idesc, ks > 0 ? 1u : 0u);
  }
  mma_commit(done);
}

// O^T (+)= V^T P^T of one tile, likewise.
template <typename C, bool kE4m3>
__device__ __noinline__ void issue_values(uint32_t tO, uint32_t v, uint32_t pb, uint32_t accumulate,
                                          uint64_t* done) {
  tc_fence_after();
  const uint64_t dp = sdesc_sw128(pb, 16, 1024);
  if constexpr (kE4m3) {
    constexpr uint32_t idesc = idesc_e4m3(128, C::kNO, true, false, false, true);
    const uint64_t dv = C::D == 64 ? sdesc_sw64(v, 0) : sdesc_sw128(v, 1024, 1024);
#pragma unroll
    for (int ks = 0; ks < 4; ++ks)  // 32 keys each
      mma8_ss(tO, dv + ((32 * C::kRowBytes * ks) >> 4), dp + 2 * ks, idesc, ks > 0 ? 1u : accumulate);
  } else {
    constexpr uint32_t idesc = idesc_bf16(128, C::kNO, true, false);
    const uint64_t dv = sdesc_sw128(v, C::D == 64 ? 0 : C::kChunkBytes, 1024);
#pragma unroll
    for (int ks = 0; ks < 8; ++ks)  // 16 keys each
      mma_ss(tO, dv + 128 * ks, dp + (((ks >> 2) * C::kNO * 128 + (ks & 3) * 32) >> 4), idesc,
             ks > 0 ? 1u : accumulate);
  }
  mma_commit(done);
}

template <int kD, bool kE4m3, int kR>
__global__ void __launch_bounds__(CacheKeysCfg<kD, kE4m3, kR>::kThreads, 1)
    fa_cache_keys_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                         const __grid_constant__ CacheFwdParams p) {
  using C = CacheKeysCfg<kD, kE4m3, kR>;
  constexpr int kG = C::kG;
  constexpr int kRows = 32;  // the list's row tile: a unit has at most kR rows
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ uint64_t q_full[2], q_empty[2], drain[kG];
  // per piece parity: every group's statistics and products are done; joined
  __shared__ uint64_t done[2], joined[2];
  __shared__ uint64_t k_full[C::kKStages], k_empty[C::kKStages];
  __shared__ uint64_t v_full[C::kVStages], v_empty[C::kVStages];
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag, any_bad[2];
  __shared__ uint32_t bad[2][32];  // drafted rows with non-finite values (T <= 1024)
  // per group and row: negated reference, rescale factor; per Q buffer and row:
  // factor of the scores
  __shared__ __align__(16) float s_nm[kG][kR], s_alpha[kG][kR], s_rowf[2][kE4m3 ? kR : 4];
  __shared__ float s_red[kG][4][kR];  // maxima of a group's warps
  // per piece parity: the groups' negated references, their warps' sums of l,
  // the weights of their accumulators
  __shared__ float s_pm[2][kG][kR], s_pl[2][kG][4][kR], s_w[2][kG][kR];
  __shared__ long long s_out[2][kR];  // per piece parity: where a row's output starts

  // barriers and tensor memory need nothing of the kernel before
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int x = 0; x < 2; ++x) {
      mbar_init(&q_full[x], 4);
      mbar_init(&q_empty[x], 4 * kG);
      mbar_init(&done[x], 5 * kG);  // a group's warps, and its last product
      mbar_init(&joined[x], 4);
    }
    for (int x = 0; x < kG; ++x) mbar_init(&drain[x], 2);
    for (int s = 0; s < C::kKStages; ++s) {
      mbar_init(&k_full[s], 1);
      mbar_init(&k_empty[s], 1);
    }
    for (int s = 0; s < C::kVStages; ++s) {
      mbar_init(&v_full[s], 1);
      mbar_init(&v_empty[s], 1);
    }
    abort_flag = 0;
    any_bad[0] = any_bad[1] = 0;
    fence_mbar_init();
  }
  if (tid < 64) bad[tid >> 5][lane] = 0u;
  if (!kE4m3 && kR < C::kN) {  // rows of P behind the query rows: zero throughout
    for (int i = tid; i < kG * C::kPBytes / 16; i += C::kThreads)
      *reinterpret_cast<uint4*>(smem + C::kOffP + 16 * i) = make_uint4(0u, 0u, 0u, 0u);
    fence_proxy_async_smem();
  }
  if (warp == C::kProducerWarp) {
    if (lane == 0) prefetch_tensormap(&tmK);
    tmem_alloc(&tmem_slot, C::kTmemCols);
  }
  if (warp == C::kProducerWarp + 1 && lane == 0) prefetch_tensormap(&tmV);
  pdl_wait();
  PieceWalk<kRows> walk(p, blockIdx.x, gridDim.x);  // every warp follows the same list
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  pdl_launch_dependents();
  if (walk.left == 0) {
    if (warp == C::kProducerWarp) tmem_dealloc(tmem, C::kTmemCols);
    return;
  }
  const CacheRing kring{smem + C::kOffK, k_full, k_empty, &tmK};
  const CacheRing vring{smem + C::kOffV, v_full, v_empty, &tmV};
  Piece w;

  if (warp >= C::kProducerWarp) {
    // ------------------------------------------------------------ producers
    const int pw = warp - C::kProducerWarp;
    constexpr int kLanes = C::D / 8, kPer = 32 / kLanes;  // lanes of a row of Q, rows at once
    constexpr int kLoads = kR / (4 * kPer) > 0 ? kR / (4 * kPer) : 1;  // per lane
    const int c8 = lane % kLanes, sub = lane / kLanes;
    uint4 q8[kLoads];
    // Q's rows are on their way while the piece's first tile is asked for
    auto q_load = [&](const Piece& w) {
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int r = (4 * i + pw) * kPer + sub;
        q8[i] = make_uint4(0u, 0u, 0u, 0u);
        if (r < w.rows) {
          const int t = row_token(p, r), hq = w.h * p.group + r - t * p.group;
          q8[i] = __ldg(reinterpret_cast<const uint4*>(p.q + row_offset(p.lq, w.b, hq, t)) + c8);
        }
      }
    };
    auto q_store = [&](const Piece&, int piece) {
      const int x = piece & 1;
      uint8_t* const q = smem + C::kOffQ + x * C::kQBytes;
      if (!cache_wait_warp(&q_empty[x], ((piece >> 1) & 1) ^ 1, &abort_flag, p.status, 2641))
        return false;
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int r = (4 * i + pw) * kPer + sub;
        if constexpr (kE4m3) {
          const SplitQ f = split_q<kLanes, true>(q8[i]);
          if (r < kR) {
            *reinterpret_cast<uint2*>(q + e4m3_row_offset<C::D>(r, c8)) = f.hi;
            *reinterpret_cast<uint2*>(q + e4m3_row_offset<C::D>(kR + r, c8)) = f.lo;
            if (c8 == 0) s_rowf[x][r] = f.factor;
          }
        } else if (r < kR) {
          uint8_t* at = q + (c8 >> 3) * C::kN * 128;
          *reinterpret_cast<uint4*>(at + sw128_offset(r, (c8 & 7) * 8)) = q8[i];
          if (kR < C::kN)  // an MMA has 16 columns at least
            *reinterpret_cast<uint4*>(at + sw128_offset(r + 8, (c8 & 7) * 8)) =
                make_uint4(0u, 0u, 0u, 0u);
        }
      }
      fence_proxy_async_smem();
      mbar_arrive_warp(&q_full[x]);
      return true;
    };
    if constexpr (kG == 4) {
      cache_producer<C, true, true, 4>(p, walk, kring, vring, pw, &abort_flag, 2601, q_load, q_store);
    } else if (pw < 2) {
      cache_producer<C, true, false, 2>(p, walk, kring, vring, pw, &abort_flag, 2601, q_load, q_store);
    } else {
      cache_producer<C, false, true, 2>(p, walk, kring, vring, pw - 2, &abort_flag, 2601, q_load,
                                        q_store);
    }
  } else {
    // ------------------------------------------------------------ softmax
    const int e = warp >> 2, wq = warp & 3;  // group, warp of the group
    const int kk = tid & 127;                // key of the tile; lane of O^T
    // P V is issued by a thread of the group's first warp, S by one of its second
    const bool issuer = kk == 0, s_issuer = kk == 32;
    const uint32_t lane_off = (uint32_t)(wq * 32) << 16;
    const uint32_t sQ = smem_addr(smem + C::kOffQ), sP = smem_addr(smem + C::kOffP);
    const uint32_t sK = smem_addr(smem + C::kOffK), sV = smem_addr(smem + C::kOffV);
    // S(n) from Q buffer qx; the issuer alone, its operands landed
    auto issue_s = [&](int n, int qx) {
      const int st = n % C::kKStages;
      issue_scores<C, kE4m3>(tmem + C::kColS + C::kN * e, sK + st * C::kTileBytes,
                             sQ + qx * C::kQBytes, &k_empty[st]);
    };
    // O += P(n) V(n); likewise
    auto issue_pv = [&](int n, uint32_t tO, uint32_t accumulate) {
      const int st = n % C::kVStages;
      issue_values<C, kE4m3>(tO, sV + st * C::kTileBytes, sP + e * C::kPBytes, accumulate, &v_empty[st]);
    };
    // waits for S(n); for O += P(n) V(n).  (Until the group's next one on the stage
    // the barrier's phase stays, and that is issued behind both.)
    auto scores_done = [&](int n) {
      return cache_wait(&k_empty[n % C::kKStages], (n / C::kKStages) & 1, &abort_flag, p.status, 2621);
    };
    auto values_done = [&](int n) {
      return cache_wait(&v_empty[n % C::kVStages], (n / C::kVStages) & 1, &abort_flag, p.status, 2628);
    };
    auto k_ready = [&](int n) { return mbar_try(smem_addr(&k_full[n % C::kKStages]), (n / C::kKStages) & 1); };

    // After a wait that gave up, a warp still passes every barrier of its group;
    // a vote then stops the group.
    bool ok = true;
    int n0 = 0;  // tiles before the piece
    // e4m3: the scales of the group's next tile, the page of the one after
    float2 scales = make_float2(0.f, 0.f);
    int page = 0;
    bool more = walk.next(w);
    if (kE4m3) {
      const int key = (w.t0 + e) * 128 + kk;
      page = key_page(p.c, w, key);
      scales = key_scales(p.c, w, key, page);
    }
    for (int piece = 0; more; ++piece) {
      const int y = piece & 1;
      const uint32_t tO = tmem + C::kColO + C::kNO * (e + kG * y);
      const int tiles = w.t1 - w.t0;
      if (wq == 0 && lane < kR) s_nm[e][lane] = lane < w.rows ? kUnset : -INFINITY;  // unused: weight 0
      // the statistics, flags and accumulators of the piece before last are free
      if (ok && piece >= 2)
        ok = cache_wait_warp(&joined[y], ((piece >> 1) & 1) ^ 1, &abort_flag, p.status, 2617);
      if (ok) ok = cache_wait_warp(&q_full[y], (piece >> 1) & 1, &abort_flag, p.status, 2620);
      asm volatile("bar.sync %0, 128;" ::"r"(2 + e) : "memory");
      float l[kR];
#pragma unroll
      for (int r = 0; r < kR; ++r) l[r] = 0.f;
      const int i0 = (e - n0) & (kG - 1);
      bool issued = false;  // S of the coming tile (the issuer's)
      if (kE4m3) page = key_page(p.c, w, (w.t0 + i0 + kG) * 128 + kk);
      for (int i = i0; i < tiles; i += kG) {  // the group's tiles
        const int n = n0 + i, tile = w.t0 + i;
        const bool tail = (tile + 1) * 128 > w.start;  // drafted rows, the sequence's end
        if (s_issuer && !issued) {
          if (ok)
            ok = cache_wait(&k_full[n % C::kKStages], (n / C::kKStages) & 1, &abort_flag, p.status, 2612);
          if (ok) issue_s(n, y);
        }
        if (ok) ok = scores_done(n);
        // (the stage's last V first, which this warp has not waited for: were it still on
        // its way, its phase's parity would pass for this one's)
        if (ok && tail && n >= kG) ok = values_done(n - kG);
        if (ok && tail)
          ok = cache_wait(&v_full[n % C::kVStages], (n / C::kVStages) & 1, &abort_flag, p.status, 2626);
        ok = __all_sync(0xffffffffu, ok);
        const int key = tile * 128 + kk;
        float t[kR];
        float inv = 0.f;
        if (ok) {  // warp-uniform
          tc_fence_after();
          uint32_t s[C::kN];
          const uint32_t tS = tmem + C::kColS + C::kN * e + lane_off;
          if constexpr (C::kN == 32) FA_TMEM_LD32_SYNC(tS, s);
          if constexpr (C::kN == 16) FA_TMEM_LD16_SYNC(tS, s);
          if constexpr (kE4m3) {
            const KeyFactors f = key_factors(scales, p.scale_log2);
            scales = key_scales(p.c, w, key + 128 * kG, page);
            page = key_page(p.c, w, key + 256 * kG);
            inv = f.inv;
            const float2 a2 = make_float2(f.score, f.score), b2 = make_float2(f.log2v, f.log2v);
            const float2 sixteenth = make_float2(0.0625f, 0.0625f);
#pragma unroll
            for (int r = 0; r < kR; r += 4) {
              const float4 rf = *reinterpret_cast<const float4*>(&s_rowf[y][kE4m3 ? r : 0]);
#pragma unroll
              for (int j = 0; j < 4; j += 2) {
                const float2 sum = fma2(make_float2(__uint_as_float(s[(C::kN / 2 + r + j) % C::kN]),
                                                    __uint_as_float(s[(C::kN / 2 + r + j + 1) % C::kN])),
                                        sixteenth,
                                        make_float2(__uint_as_float(s[r + j]), __uint_as_float(s[r + j + 1])));
                const float2 z = fma2(sum, mul2(a2, j ? make_float2(rf.z, rf.w) : make_float2(rf.x, rf.y)), b2);
                t[r + j] = z.x;
                t[r + j + 1] = z.y;
              }
            }
          } else {
#pragma unroll
            for (int r = 0; r < kR; ++r) t[r] = __uint_as_float(s[r]) * p.scale_log2;
          }
          tc_fence_before();
          if (tail) {
            const int u = key - w.start;
            if (u >= 0) {
              uint32_t sees = 0;  // bit r: row r sees the key
              if (key < w.klen)
#pragma unroll 1
                for (int r = 0, tok = 0; r < w.rows; r += p.group, ++tok)
                  if (token_sees(p, w.b, tok, u))
                    sees |= (p.group < 32 ? (1u << p.group) - 1u : ~0u) << r;
#pragma unroll
              for (int r = 0; r < kR; ++r)
                if (!((sees >> r) & 1u)) t[r] = -INFINITY;
            }
            if (tile * 128 + 32 * wq + 32 > w.start)
              clean_rows<C, 32, kE4m3>(smem + C::kOffV + (n % C::kVStages) * C::kTileBytes, w.start,
                                       w.klen, 32 * wq, tile * 128, bad[y], &any_bad[y]);
          }
        } else {
#pragma unroll
          for (int r = 0; r < kR; ++r) t[r] = -INFINITY;
        }
        // ---- do all scores stay within reach of their references?
        float over = -INFINITY;
#pragma unroll
        for (int r = 0; r < kR; r += 4) {
          const float4 nm = *reinterpret_cast<const float4*>(&s_nm[e][r]);
          over = max3(max3(over, t[r] + nm.x, t[r + 1] + nm.y), t[r + 2] + nm.z, t[r + 3] + nm.w);
        }
        const bool raise = barrier_any(2 + e, 128, over > C::kTop + C::kGrow || !ok);
        if (raise) {
          if (barrier_any(2 + e, 128, !ok)) {
            ok = false;
            break;
          }
          // the rows' maxima over the tile
          float mine = -INFINITY;
#pragma unroll
          for (int r = 0; r < kR; ++r) {
            const float m = warp_max(t[r]);
            if (lane == r) mine = m;
          }
          if (lane < kR) s_red[e][wq][lane] = mine;
          asm volatile("bar.sync %0, 128;" ::"r"(2 + e) : "memory");
          if (wq == 0 && lane < kR) {
            const float m = fmaxf(fmaxf(s_red[e][0][lane], s_red[e][1][lane]),
                                  fmaxf(s_red[e][2][lane], s_red[e][3][lane]));
            const float nm = s_nm[e][lane];
            float alpha = 1.f;
            if (m + nm > C::kTop + C::kGrow) {
              alpha = nm == kUnset ? 0.f : ex2(C::kTop - m - nm);
              s_nm[e][lane] = C::kTop - m;
            }
            s_alpha[e][lane] = alpha;
          }
          asm volatile("bar.sync %0, 128;" ::"r"(2 + e) : "memory");
#pragma unroll
          for (int r = 0; r < kR; ++r) l[r] *= s_alpha[e][r];
          if (i >= kG) {
            // the accumulator holds the group's earlier tiles once the last is done
            ok = __all_sync(0xffffffffu, values_done(n - kG));
            if (ok) {
              tc_fence_after();
#pragma unroll 1
              for (int c = 0; c < C::kNO; c += 16) {
                uint32_t o[16];
                FA_TMEM_LD16_SYNC(tO + lane_off + c, o);
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                  const int r = (c + j) & (kR - 1);
                  o[j] = __float_as_uint(__uint_as_float(o[j]) * s_alpha[e][r]);
                }
                FA_TMEM_ST16(tO + lane_off + c, o);
              }
              tmem_wait_st();
            }
          }
        }
        // ---- P of this key, once the group's last product has read its P
        if (ok && n >= kG) ok = __all_sync(0xffffffffu, values_done(n - kG));
        uint8_t* const pb = smem + C::kOffP + e * C::kPBytes;
        if constexpr (kE4m3) {
          // Neighbouring keys exchange rows, so that a store has both keys' bytes of a row
          // (by one byte the stores took 5 % of a call with 16 rows): the even lane takes
          // rows 4 j and 4 j + 1, the odd one 4 j + 2 and 4 j + 3, in other banks.
          const int odd = lane & 1;
          uint8_t* const at = pb + (kk & 14) + odd * 256;
          const uint32_t c16 = (kk >> 4) ^ (2 * odd);
          const uint32_t sel0 = odd ? 0x1054 : 0x5410, sel1 = odd ? 0x3276 : 0x7632;
#pragma unroll
          for (int r = 0; r < kR; r += 4) {
            uint32_t x[2];  // rows r, r + 1; r + 2, r + 3 as f16
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const int i = r + 2 * j;
              const float2 nm = *reinterpret_cast<const float2*>(&s_nm[e][i]);
              const float2 z = add2(make_float2(t[i], t[i + 1]), nm);
              const float2 pv = make_float2(ex2(z.x), ex2(z.y));
              const float2 sum = fma2(pv, make_float2(inv, inv), make_float2(l[i], l[i + 1]));
              l[i] = sum.x;
              l[i + 1] = sum.y;
              x[j] = pack_f16(pv.x, pv.y);
            }
            const uint32_t mine = odd ? x[1] : x[0];
            const uint32_t other = __shfl_xor_sync(0xffffffffu, odd ? x[0] : x[1], 1);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              uint32_t term[3];
              split_p(__byte_perm(mine, other, j ? sel1 : sel0), term);
              uint8_t* const a0 = at + (r + j) * 128 + ((c16 ^ ((r + j) & 7)) << 4);
#pragma unroll
              for (int i = 0; i < 3; ++i)  // kR is a multiple of 8: the same swizzle
                *reinterpret_cast<uint16_t*>(a0 + i * kR * 128) =
                    (uint16_t)__byte_perm(term[i], 0, 0x31);
            }
          }
        } else {
          uint8_t* const at = pb + (kk >> 6) * C::kN * 128 + (kk & 7) * 2;
          const uint32_t c16 = (kk & 63) >> 3;
#pragma unroll
          for (int r = 0; r < kR; r += 2) {
            const float2 nm = *reinterpret_cast<const float2*>(&s_nm[e][r]);
            const float2 z = add2(make_float2(t[r], t[r + 1]), nm);
            const float2 pv = make_float2(ex2(z.x), ex2(z.y));
            const float2 sum = add2(pv, make_float2(l[r], l[r + 1]));
            l[r] = sum.x;
            l[r + 1] = sum.y;
            const uint32_t two = pack_bf16(pv.x, pv.y);  // 2^-8 of each weight
            *reinterpret_cast<uint16_t*>(at + r * 128 + ((c16 ^ (r & 7)) << 4)) = (uint16_t)two;
            *reinterpret_cast<uint16_t*>(at + (r + 1) * 128 + ((c16 ^ ((r + 1) & 7)) << 4)) =
                (uint16_t)(two >> 16);
          }
        }
        fence_proxy_async_smem();
        tc_fence_before();
        if (wq == 0) {
          asm volatile("bar.sync %0, 128;" ::"r"(6 + e) : "memory");
          if (issuer && ok) {
            ok = cache_wait(&v_full[n % C::kVStages], (n / C::kVStages) & 1, &abort_flag, p.status, 2614);
            if (ok) issue_pv(n, tO, i >= kG ? 1u : 0u);
          }
          ok = __shfl_sync(0xffffffffu, ok, 0);
        } else {
          asm volatile("bar.arrive %0, 128;" ::"r"(6 + e) : "memory");
          // the group has read S(n) (the vote): S of its next tile replaces it, if its
          // keys have landed
          issued = s_issuer && ok && i + kG < tiles && k_ready(n + kG);
          if (issued) issue_s(n + kG, y);
          __syncwarp();
        }
      }

      // ---- leave the group's statistics, and its last product's completion
      const float ls = sum_to_lanes<kR>(l);
      if (lane < kR) {
        s_pl[y][e][wq][lane] = ls;
        if (wq == 0) s_pm[y][e][lane] = s_nm[e][lane];
      }
      if (issuer) {
        if (ok && i0 < tiles)
          mma_commit(&done[y]);
        else
          mbar_arrive(&done[y]);
      }
      mbar_arrive_warp(&done[y]);
      if (lane == 0) mbar_arrive(&q_empty[y]);
      const Piece last = w;
      n0 += tiles;
      more = walk.next(w);
      if (kE4m3 && more) {
        const int key = (w.t0 + ((e - n0) & (kG - 1))) * 128 + kk;
        page = key_page(p.c, w, key);
      }

      // ---- the group of the piece's last tile joins all groups
      if (e == ((n0 - 1) & (kG - 1))) {
        if (ok) ok = cache_wait_warp(&done[y], (piece >> 1) & 1, &abort_flag, p.status, 2627);
        tc_fence_after();
        // groups with a tile in the piece (the others' accumulators are old)
        auto has = [&](int g) { return ((g - (n0 - tiles)) & (kG - 1)) < tiles; };
        float* const slot = last.slot < 0 ? nullptr : p.ws + (size_t)last.slot * slot_floats<kD, kRows>();
        if (kk < kR) {
          float m[kG], mm = -INFINITY, lt = 0.f;
#pragma unroll
          for (int g = 0; g < kG; ++g) {
            const float nm = s_pm[y][g][kk];
            m[g] = nm == kUnset || kk >= last.rows ? -INFINITY : -nm;
            mm = fmaxf(mm, m[g]);
          }
#pragma unroll
          for (int g = 0; g < kG; ++g) {
            m[g] = m[g] == -INFINITY ? 0.f : ex2(m[g] - mm);  // now the group's weight
            lt += (s_pl[y][g][0][kk] + s_pl[y][g][1][kk] + s_pl[y][g][2][kk] + s_pl[y][g][3][kk]) * m[g];
          }
          const bool empty = lt == 0.f;
          const float scale = slot ? 1.f : empty ? 0.f : 1.f / lt;
#pragma unroll
          for (int g = 0; g < kG; ++g) s_w[y][g][kk] = m[g] * scale;
          const int t = row_token(p, kk), hq = last.h * p.group + kk - t * p.group;
          s_out[y][kk] = slot ? kk * C::D : row_offset(p.lo, last.b, hq, t);
          if (ok && kk < last.rows) {
            if (slot) {
              slot[kRows * C::D + kk] = mm;
              slot[kRows * C::D + kRows + kk] = lt;
            } else {
              p.lse[((size_t)last.b * p.Hq + hq) * p.T + t] = empty ? -INFINITY : (mm + log2f(lt)) * kLn2;
            }
          }
        }
        asm volatile("bar.sync %0, 128;" ::"r"(2 + e) : "memory");
        // lane kk of O^T holds element kk of every row
        if (ok && (C::D == 128 || wq < 2)) {
          const uint32_t tall = tmem + C::kColO + C::kNO * kG * y + lane_off;
#pragma unroll 1
          for (int r0 = 0; r0 < last.rows; r0 += 8) {
            __syncwarp();  // the loads below are warp-wide
            float o[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) o[j] = 0.f;
#pragma unroll
            for (int g = 0; g < kG; ++g) {
              if (!has(g)) continue;
              uint32_t a[8];
              FA_TMEM_LD8_SYNC(tall + C::kNO * g + r0, a);
              if constexpr (kE4m3) {
                uint32_t b[8], c[8];
                FA_TMEM_LD8_SYNC(tall + C::kNO * g + kR + r0, b);
                FA_TMEM_LD8_SYNC(tall + C::kNO * g + 2 * kR + r0, c);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                  o[j] = fmaf(__uint_as_float(a[j]) + (__uint_as_float(b[j]) + __uint_as_float(c[j])),
                              s_w[y][g][r0 + j], o[j]);
              } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) o[j] = fmaf(__uint_as_float(a[j]), s_w[y][g][r0 + j], o[j]);
              }
            }
            if (any_bad[y]) {
#pragma unroll 1
              for (int j = 0; j < 8 && r0 + j < last.rows; ++j) {
                float extra = 0.f;
                add_nonfinite<kE4m3>(p, last.b, last.h, last.start, bad[y], row_token(p, r0 + j), kk, 1,
                                     &extra);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                  if (i == j) o[i] += extra;
              }
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              if (r0 + j >= last.rows) break;
              const long long at = s_out[y][r0 + j] + kk;
              if (slot)
                slot[at] = o[j];
              else
                p.o[at] = __float2bfloat16(o[j]);
            }
          }
        }
        tc_fence_before();
        asm volatile("bar.sync %0, 128;" ::"r"(2 + e) : "memory");
        if (wq == 0) {
          bad[y][lane] = 0u;
          if (lane == 0) any_bad[y] = 0;
        }
        mbar_arrive_warp(&joined[y]);
      }
      if (kE4m3 && more) scales = key_scales(p.c, w, (w.t0 + ((e - n0) & (kG - 1))) * 128 + kk, page);
      if (barrier_any(2 + e, 128, !ok)) break;
    }
    // the group's products are complete once its drain flips (after an abort one of S
    // may still run)
    if (issuer || s_issuer) {
      mma_commit(&drain[e]);
      mbar_drain(&drain[e], 0);
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == C::kProducerWarp) {
    __syncwarp();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

template <bool kE4m3>
cudaError_t launch_cache_keys(const CacheMaps& m, const CacheFwdParams& p, cudaStream_t s) {
  const int rows = p.T * p.group;
  auto go = [&](auto d) {
    constexpr int kD = decltype(d)::value;
    auto with = [&](auto r) {
      constexpr int kR = decltype(r)::value;
      using C = CacheKeysCfg<kD, kE4m3, kR>;
      return launch_cache_pair<kD, 32, fa_cache_keys_kernel<kD, kE4m3, kR>>(C::kThreads, C::kSmem, 1,
                                                                            m, p, s);
    };
    if constexpr (!kE4m3)
      if (rows > 16) return with(std::integral_constant<int, 32>{});
    return rows <= 8 ? with(std::integral_constant<int, 8>{}) : with(std::integral_constant<int, 16>{});
  };
  return p.c.d == 64 ? go(std::integral_constant<int, 64>{}) : go(std::integral_constant<int, 128>{});
}

}  // namespace fa
