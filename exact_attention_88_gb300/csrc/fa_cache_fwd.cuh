// What the kernels of attention over the key/value cache share.
//
// Work.  A unit is one sequence, one cache head and a tile of query rows (row =
// token * group + head within the group: all query heads that share the cache
// head are rows of one matrix product, so each cached row is read once for all
// of them).  A unit's keys are walked in tiles of 128.  The tiles of all units
// form one list, cut into equal runs, one per CTA (one persistent CTA per SM):
// lengths on the device decide the cut, so ragged batches and a single long
// sequence both load every SM alike (and where whole units do nearly as well, none
// is cut).  A unit cut by a run's border leaves
// partial results (O, m, l in fp32) that a second kernel joins; every other
// unit is finished by its CTA.  All sums have a fixed order: results are the
// same bit for bit from run to run.
//
// e4m3.  S is formed from the cache's 8-bit values (kind::f8f6f4, fp32 accumulation,
// exact products): Q, scaled by a power of two per row, is the sum of two 8-bit terms,
// exact down to 2^-13 of the row's largest element, and the keys' scales multiply the
// scores.  For few query rows P V is too: P as three e5m2 terms keeps 8 to 9 bits, and
// the values' scales s_v enter the exponent: P' = 2^(s + log2 s_v - m) with m following
// the maximum of that sum, so that a row's largest *contribution* sits at 2^13 ..
// 2^15.75 of the terms' range whatever the scales are; l sums P' / s_v.  For more rows P
// is f16 and V is scaled and converted to f16 on its way.
//
// Rows behind the sequence and drafted tokens that a query row does not see may
// hold anything, and 0 * NaN is NaN in a matrix product: in the tiles that
// reach past start[b] the softmax warps zero the V rows behind the sequence and
// the non-finite elements of drafted rows in shared memory, and the epilogue
// adds the latter back to the rows that see them.
#pragma once

#include <type_traits>

#include "fa_cache.cuh"

namespace fa {

constexpr int kCacheMaxCtas = 160;

struct CacheFwdParams {
  const __nv_bfloat16* q;
  __nv_bfloat16* o;
  float* lse;
  Layout lq, lo;
  CacheView c;
  const int32_t* start;
  const int32_t* q_len;
  const uint32_t* mask;
  float* ws;
  int B, Hq, T, W;  // W: mask words of a token
  int group;        // query heads per cache head
  uint32_t group_inv;  // 2^32 / group, rounded up: row / group by one multiplication
  int box_rows;     // rows of one TMA box
  float scale_log2;
  int whole;    // no unit is cut (else the lengths decide)
  float slack;  // tiles above the average that a CTA may have before units are cut
  int* status;
};

// Token of a unit's row g < 2^26, g / group: the product with the inverse, less than
// 2^-32 too large, is at most one too large (from g group > 2^32 on it can be).
__device__ __forceinline__ int row_token(const CacheFwdParams& p, int g) {
  if (p.group == 1) return g;
  const int t = (int)__umulhi((uint32_t)g, p.group_inv);
  return t - (t * p.group > g ? 1 : 0);
}

// A wait on an mbarrier whose first try is inline and whose loop is not: the
// kernels have some twenty waits, and short calls spend much of their time on
// fetching instructions.
static __device__ __noinline__ bool cache_wait_loop(uint64_t* bar, uint32_t parity, int* abort_flag,
                                             int* status, int site) {
  return mbar_wait(bar, parity, abort_flag, status, site);
}
__device__ __forceinline__ bool cache_wait(uint64_t* bar, uint32_t parity, int* abort_flag,
                                           int* status, int site) {
  return mbar_try(smem_addr(bar), parity) || cache_wait_loop(bar, parity, abort_flag, status, site);
}
__device__ __forceinline__ bool cache_wait_warp(uint64_t* bar, uint32_t parity, int* abort_flag,
                                                int* status, int site) {
  return __all_sync(0xffffffffu, cache_wait(bar, parity, abort_flag, status, site));
}

// ---------------------------------------------------------------------------
// the list of tiles, shared by the main and the joining kernel
// ---------------------------------------------------------------------------
struct SeqInfo {
  int start, q, klen, tiles, row_tiles;
};

// (Out of line with its arguments in registers: a reference to the parameters would
// be read through memory.)
template <int kRows>
__device__ __noinline__ SeqInfo seq_info(const int32_t* start, const int32_t* q_len, int b, int T,
                                         int capacity, int group) {
  SeqInfo s;
  s.q = clamped_len(q_len, b, T);
  s.start = min(max(__ldg(start + b), 0), capacity);
  s.klen = min(s.start + min(s.q, capacity), capacity);  // capacity < 2^31 - 2^16
  s.tiles = s.q > 0 ? (s.klen + 127) >> 7 : 0;
  s.row_tiles = (s.q * group + kRows - 1) / kRows;  // kRows: a power of two
  return s;
}
template <int kRows>
__device__ __forceinline__ SeqInfo seq_info(const CacheFwdParams& p, int b) {
  return seq_info<kRows>(p.start, p.q_len, b, p.T, p.c.capacity, p.group);
}

// (Tiles fit 31 bits: checked on the host.)
struct TileList {
  int total;       // tiles of all units
  int ctas;        // CTAs with work (at most kCacheMaxCtas): each takes at least one tile
  int each, more;  // total = each * ctas + more
  uint32_t inv;    // 2^32 / ctas, rounded up
  __device__ TileList(int tiles, int grid) : total(tiles), ctas(min(tiles, grid)), each(0), more(0), inv(0) {
    if (ctas == 0) return;
    each = total / ctas;
    more = total - each * ctas;
    inv = 0xffffffffu / ctas + 1u;
  }
  // total c / ctas (more c < 2^16: the product with the inverse is exact)
  __device__ int begin(int c) const {
    return each * c + (ctas == 1 ? more * c : (int)__umulhi((uint32_t)(more * c), inv));
  }
  __device__ int cta_of(int g) const {  // the largest c with begin(c) <= g
    int c = min((int)((float)g * ((float)ctas / (float)total)), ctas - 1);
#pragma unroll 1
    while (c + 1 < ctas && begin(c + 1) <= g) ++c;
#pragma unroll 1
    while (begin(c) > g) --c;
    return c;
  }
};

// Tiles of sequence b's units (whole: its units).
template <int kRows>
__device__ __forceinline__ int seq_weight(const CacheFwdParams& p, const SeqInfo& s, bool whole) {
  return (whole ? min(s.tiles, 1) : s.tiles) * s.row_tiles * p.c.heads;
}

// Cutting every unit where a run ends balances the CTAs to a tile, but each cut costs
// a partial result, its joining, and Q and an epilogue once more: as much as five
// tiles, of bf16 and few rows four.  So units stay whole where the CTA with the most
// would have at most that much (slack) more than the average.  (8 sequences, 8 heads,
// 500 keys, e4m3: 9.7 us whole, 13.7 cut; with 64 rows 13 and 20; one sequence of 760
// keys: 11.2 and 10.6; 8 bf16 sequences of 1000 keys: 16.1 and 15.8.)  With no more
// tiles than CTAs nobody has two pieces, and three tiles are the limit (one sequence of
// 630 keys, 32 rows: 14.4 and 11.2).
// (Rounded operations by name: both kernels must decide alike.)
__device__ __forceinline__ bool keep_whole(int tiles, int units, int most, int grid,
                                           float slack) {
  const float inv = __frcp_rn((float)grid);
  const float runs = ceilf(__fmul_rn((float)units, inv));
  return __fsub_rn(__fmul_rn(runs, (float)most), __fmul_rn((float)tiles, inv)) <=
         (tiles <= grid ? fminf(slack, 3.f) : slack);
}

// Whole warp: the list of all sequences' units, and the tiles of those below `before`
// in *prefix.
struct WholeOrTiles {
  int total;
  bool whole;
};
template <int kRows>
__device__ __forceinline__ WholeOrTiles list_of(const CacheFwdParams& p, int grid, int before, int* prefix) {
  int tiles = 0, units = 0, most = 0, pre = 0;
#pragma unroll 1
  for (int b = threadIdx.x & 31; b < p.B; b += 32) {
    const SeqInfo s = seq_info<kRows>(p, b);
    const int w = seq_weight<kRows>(p, s, false);
    tiles += w;
    units += seq_weight<kRows>(p, s, true);
    most = max(most, s.tiles);
    if (b < before) pre += w;
  }
  if (prefix) *prefix = __reduce_add_sync(0xffffffffu, pre);
  tiles = __reduce_add_sync(0xffffffffu, tiles);
  units = __reduce_add_sync(0xffffffffu, units);
  most = __reduce_max_sync(0xffffffffu, most);
  const bool whole = p.whole || keep_whole(tiles, units, most, grid, p.slack);
  return WholeOrTiles{whole ? units : tiles, whole};
}

// Whole warp: the sequence that holds tile (whole: unit) g of the list (g < its total),
// its first, and what is known of it.
template <int kRows>
__device__ __forceinline__ int find_seq(const CacheFwdParams& p, int g, bool whole, int* first,
                                        SeqInfo* info) {
  const int lane = threadIdx.x & 31;
  int acc = 0;
#pragma unroll 1
  for (int base = 0;; base += 32) {
    SeqInfo s{};
    if (base + lane < p.B) s = seq_info<kRows>(p, base + lane);
    const int w = seq_weight<kRows>(p, s, whole);
    int incl = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += x;
    }
    const unsigned past = __ballot_sync(0xffffffffu, acc + incl > g);
    if (past || base + 32 >= p.B) {
      const int at = past ? __ffs(past) - 1 : 0;
      *first = __shfl_sync(0xffffffffu, acc + incl - w, at);
      info->start = __shfl_sync(0xffffffffu, s.start, at);
      info->q = __shfl_sync(0xffffffffu, s.q, at);
      info->klen = __shfl_sync(0xffffffffu, s.klen, at);
      info->tiles = __shfl_sync(0xffffffffu, s.tiles, at);
      info->row_tiles = __shfl_sync(0xffffffffu, s.row_tiles, at);
      return base + at;
    }
    acc += __shfl_sync(0xffffffffu, incl, 31);
  }
}

// One CTA's part of a unit: tiles [t0, t1) of `tiles`.
struct Piece {
  int b, h, rt, t0, t1;
  int start, klen, rows;  // rows: query rows of the unit
  int slot;               // workspace slot of a partial result; -1: the whole unit
};

template <int kRows>
struct PieceWalk {
  const CacheFwdParams& p;
  const int row0;  // pieces of units with at most row0 rows are passed over
  int left;
  int b, h, rt, tile, slot;
  SeqInfo s;

  __device__ PieceWalk(const CacheFwdParams& params, int cta, int grid, int skip_rows = 0)
      : p(params), row0(skip_rows) {  // whole warp
    const WholeOrTiles all = list_of<kRows>(p, grid, 0, nullptr);
    const TileList list(all.total, grid);
    left = 0;
    if (cta >= list.ctas) return;
    const int lo = list.begin(cta);
    left = list.begin(cta + 1) - lo;
    int first;
    b = find_seq<kRows>(p, lo, all.whole, &first, &s);
    const int in = lo - first, unit = all.whole ? in : in / s.tiles;
    tile = all.whole ? 0 : in - unit * s.tiles;
    h = s.row_tiles == 1 ? unit : unit / s.row_tiles;
    rt = unit - h * s.row_tiles;
    slot = all.whole ? -1 : 2 * cta;  // (-1 throughout)
  }
  __device__ bool next(Piece& w) {
#pragma unroll 1
    while (left > 0) {
      step(w);
      if (w.rows > row0) return true;
    }
    return false;
  }
  __device__ void step(Piece& w) {
#pragma unroll 1
    while (s.tiles == 0) {
      if (++b >= p.B) {  // only if the lengths changed under the kernel
        left = w.rows = 0;
        return;
      }
      s = seq_info<kRows>(p, b);
    }
    const int run = slot < 0 ? s.tiles : min(left, s.tiles - tile);
    w.b = b;
    w.h = h;
    w.rt = rt;
    w.t0 = tile;
    w.t1 = tile + run;
    w.start = s.start;
    w.klen = s.klen;
    w.rows = min(kRows, s.q * p.group - rt * kRows);
    w.slot = run == s.tiles ? -1 : slot;
    slot |= 1;
    left -= slot < 0 ? 1 : run;
    tile = 0;
    if (++rt == s.row_tiles) {
      rt = 0;
      if (++h == p.c.heads) {
        h = 0;
        s.tiles = 0;  // the next call takes the next sequence
      }
    }
  }
};

template <int kD, int kRows>
__host__ __device__ constexpr int slot_floats() { return kRows * (kD + 2); }  // O, then m, then l

// ---------------------------------------------------------------------------
// tensor-core pieces, tiles in shared memory
// ---------------------------------------------------------------------------
__device__ __forceinline__ void mma8_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                        uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Instruction descriptor, kind::f8f6f4 with A and B e4m3 (format 0; a5, b5: e5m2), D fp32.
__host__ __device__ constexpr uint32_t idesc_e4m3(int M, int N, bool a_mn, bool b_mn, bool a5 = false,
                                                  bool b5 = false) {
  return (1u << 4) | ((a5 ? 1u : 0u) << 7) | ((b5 ? 1u : 0u) << 10) | ((a_mn ? 1u : 0u) << 15) |
         ((b_mn ? 1u : 0u) << 16) |
         ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
// Instruction descriptor of kind::f16 for f16 x f16 -> fp32.
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, bool a_mn, bool b_mn) {
  return idesc_bf16(M, N, a_mn, b_mn) & ~((1u << 7) | (1u << 10));
}
// Matrix descriptor of the 64-byte-swizzled layout (8 rows x 64 bytes per
// 512-byte atom, 16-byte chunk index XOR (row / 2) % 4).
__device__ __forceinline__ uint64_t sdesc_sw64(uint32_t saddr, uint32_t lbo = 512) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | (uint64_t)(lbo >> 4) << 16 |
         (uint64_t)(512 >> 4) << 32 | (uint64_t)1 << 46 | (uint64_t)4 << 61;
}

// Barrier `id` of n threads that tells all of them whether any passed true.
__device__ __forceinline__ bool barrier_any(int id, int n, bool mine) {
  uint32_t any;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n"
      " barrier.cta.red.or.pred q, %2, %3, p;\n selp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(any)
      : "r"((uint32_t)mine), "r"(id), "r"(n)
      : "memory");
  return any != 0;
}

// A K or V tile of 128 keys in shared memory.
template <int kD, bool kE4m3>
struct CacheTile {
  static constexpr int D = kD;
  static constexpr int kRowBytes = D * (kE4m3 ? 1 : 2);
  static constexpr int kTileBytes = 128 * kRowBytes;
  static constexpr int kChunks = kRowBytes > 128 ? 2 : 1;  // 128-byte columns of a tile
  static constexpr int kChunkRow = kRowBytes / kChunks;    // 64 or 128 bytes
  static constexpr int kChunkBytes = kTileBytes / kChunks;
};

struct CacheMaps {
  CUtensorMap k, v;
};

// A ring of K or V tiles.
struct CacheRing {
  uint8_t* tiles;
  uint64_t *full, *empty;
  const CUtensorMap* map;
};

// A producer warp: loads the K tiles, the V tiles, or both (K before V of each
// tile) of the CTA's list in order, of every kStep tiles the one numbered first.
// Lane i loads box i of a tile (a page of up to 128 rows each).  The block table
// is read 32 entries at a time, a block ahead of its use.  before(w) runs before
// each piece, behind(w, piece) once in it, behind its first tile's loads.
template <typename C, bool kK, bool kV, int kStep, typename Walk, typename Before, typename Behind>
__device__ __forceinline__ void cache_producer(const CacheFwdParams& p, Walk& walk,
                                               const CacheRing& k, const CacheRing& v, int first,
                                               int* abort_flag, int site, Before before,
                                               Behind behind) {
  static_assert(C::kKStages % kStep == 0 && C::kVStages % kStep == 0, "");
  const int lane = threadIdx.x & 31;
  const bool mine = lane * p.box_rows < 128;  // this lane has a box of each tile
  const uint32_t box_bytes = p.box_rows * C::kRowBytes;
  const uint32_t dst0 = lane * p.box_rows * C::kChunkRow;
  const bool paged = p.c.table != nullptr;
  bool ok = true;
  int n0 = 0, ks = first, vs = first;
  uint32_t kparity = 1, vparity = 1;
  Piece w;
  for (int piece = 0; ok && walk.next(w); ++piece) {
    const int32_t* table = paged ? p.c.table + w.b * p.c.table_stride : nullptr;
    const int need = paged ? (w.klen + p.c.page_size - 1) >> p.c.page_shift : 0;
    auto entry = [&](int i) { return i < need ? __ldg(table + i) : 0; };
    int tile = w.t0 + ((first - n0) & (kStep - 1));
    n0 += w.t1 - w.t0;
    int base = (tile * 128) >> p.c.page_shift, ids = 0, ahead = 0;
    if (paged) {
      ids = entry(base + lane);
      ahead = entry(base + 32 + lane);
    }
    before(w);
    bool pending = true;
    int key = tile * 128 + lane * p.box_rows;  // first key of this lane's box
#pragma unroll 1
    for (;; tile += kStep, key += 128 * kStep) {
      if (tile < w.t1) {
        const bool live = mine && key < w.klen;
        const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, live)) * box_bytes;
        int page = w.b, y = key;
        if (paged) {
          if (((tile * 128) >> p.c.page_shift) - base >= 32) {
            // a tile has at most 8 entries: none straddles, no block is skipped
            base += 32;
            ids = ahead;
            ahead = entry(base + 32 + lane);
          }
          page = __shfl_sync(0xffffffffu, ids, ((key >> p.c.page_shift) - base) & 31);
          y = key & (p.c.page_size - 1);
        }
        auto load = [&](const CacheRing& r, int st, uint32_t parity, int which) {
          if (!cache_wait_warp(&r.empty[st], parity, abort_flag, p.status, which)) return false;
          if (lane == 0) mbar_expect_tx(&r.full[st], bytes);
          __syncwarp();
          if (live) {
            uint8_t* dst = r.tiles + st * C::kTileBytes + dst0;
#pragma unroll
            for (int c = 0; c < C::kChunks; ++c)
              tma_load_4d(r.map, &r.full[st], dst + c * C::kChunkBytes, c * 64, y, w.h, page);
          }
          return true;
        };
        if (kK) {
          ok = load(k, ks, kparity, site);
          if ((ks += kStep) >= C::kKStages) {
            ks = first;
            kparity ^= 1;
          }
        }
        if (kV && ok) {
          ok = load(v, vs, vparity, site + 1);
          if ((vs += kStep) >= C::kVStages) {
            vs = first;
            vparity ^= 1;
          }
        }
        // a page outside the cache reads as zeros
        if (live && (unsigned)page >= (unsigned)p.c.pages) report_page(p.status, 3003);
      }
      if (pending) {
        pending = false;
        if (ok) ok = behind(w, piece);
      }
      if (!ok || tile + kStep >= w.t1) break;
    }
  }
  // every issued copy must have landed before the CTA may exit (after an abort
  // the last round may lack one: the drain is bounded)
  if (kK)
#pragma unroll 1
    for (int i = first; i < C::kKStages; i += kStep) {
      const int used = (n0 + C::kKStages - 1 - i) / C::kKStages;
      if (used) mbar_drain(&k.full[i], (used - 1) & 1);
    }
  if (kV)
#pragma unroll 1
    for (int i = first; i < C::kVStages; i += kStep) {
      const int used = (n0 + C::kVStages - 1 - i) / C::kVStages;
      if (used) mbar_drain(&v.full[i], (used - 1) & 1);
    }
}

// The scales of key `key` of a piece's sequence (K's, V's); a bad page's read as
// 0.  page: the key's entry of the block table (without one: unused).
__device__ __forceinline__ float2 key_scales(const CacheView& c, const Piece& w, int key, int page) {
  if (!c.table) page = w.b;
  if (key >= w.klen || (unsigned)page >= (unsigned)c.pages) return make_float2(0.f, 0.f);
  const int row = c.table ? key & (c.page_size - 1) : key;
  const long long at = (long long)page * c.sb + w.h * c.sh + row;
  return make_float2(__ldg(c.ks + at), __ldg(c.vs + at));
}
// The same for the four keys key .. key + 3 (key a multiple of 4, so one page and
// 16-byte aligned); unread past the sequence.
__device__ __forceinline__ void key_scales4(const CacheView& c, const Piece& w, int key, int page,
                                            float4* k, float4* v) {
  *k = *v = make_float4(0.f, 0.f, 0.f, 0.f);
  if (!c.table) page = w.b;
  if (key >= w.klen || (unsigned)page >= (unsigned)c.pages) return;
  const long long at = (long long)page * c.sb + w.h * c.sh + (c.table ? key & (c.page_size - 1) : key);
  *k = __ldg(reinterpret_cast<const float4*>(c.ks + at));
  *v = __ldg(reinterpret_cast<const float4*>(c.vs + at));
}
// The block table's entry for a key (0 past the sequence, or without a table).
__device__ __forceinline__ int key_page(const CacheView& c, const Piece& w, int key) {
  return c.table && key < w.klen ? __ldg(c.table + w.b * c.table_stride + (key >> c.page_shift)) : 0;
}

// Factors of a key: of its scores, log2 of its value scale, 1 / value scale.
// Keys behind the sequence and bad pages (scales 0) get harmless ones.
struct KeyFactors {
  float score, log2v, inv;
};
__device__ __forceinline__ KeyFactors key_factors(float2 scales, float scale_log2) {
  const float s = fmaxf(scales.y, kMinScale);
  return KeyFactors{scales.x * scale_log2, __log2f(s), __frcp_rn(s)};  // 2^-22 is enough
}

// Two f16 as e4m3, and back.
__device__ __forceinline__ uint32_t e4m3_of(__half2 x) {
  return __nv_cvt_halfraw2_to_fp8x2(x, __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ __half2 half_of(uint32_t e) {
  return __half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)e, __NV_E4M3));
}
// Two weights (f16, below 2^15.8) as three e5m2 terms each, in bytes 1 and 3 of t: e5m2
// is the upper byte of f16, so a term is cut off and the rest, exact, goes on; the last
// is rounded.  The sum is within 2^-8.6 of the weight, or 2^-17, that is 2^-30 of the
// row's largest (kTop).  (Two e4m3 terms dropped what was below 2^-16 of it: next
// to one key of weight 2^16, 28000 of 1 left O 14 % off.  Three cost conversions: 16
// rows 7 % longer.)
__device__ __forceinline__ void split_p(uint32_t x, uint32_t* t) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    t[i] = x & 0xff00ff00u;
    asm("sub.f16x2 %0, %0, %1;" : "+r"(x) : "r"(t[i]));
  }
  t[2] = x + 0x00800080u;  // NaN (0x7fff) carries nowhere
}

// Splits 8 elements of a Q row (kLanes lanes hold the row) into two terms of the row
// times 2^k; factor: 2^-k.  2^k is the largest power of two that keeps the row within
// 448 = 1.75 2^8.  The first term is e4m3.  What it leaves has three bits where it is
// normal (2^-6 and up); the second term holds it as e5m2, where the terms' products add
// up in one accumulator, or times 16 as e4m3 (kTimes16), where they are apart.  Either
// way the sum is exact from 2^-6 up, 2^-13 of the row's largest (224 to 448), and at
// most 2^-14 off below.  (With a second term of the first's type and scale 2^-10: rows
// with one channel 1000 times the others lost bits of those.)  A row with infinities or
// NaN has no finite score: its factor is NaN.  Called by the whole warp.
struct SplitQ {
  uint2 hi, lo;
  float factor;
};
template <int kLanes, bool kTimes16>
__device__ __noinline__ SplitQ split_q(uint4 v) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  // magnitudes compare as integers; infinities and NaN are the largest
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) top = __vmaxu2(top, w[i] & 0x7fff7fffu);
#pragma unroll
  for (int o = 1; o < kLanes; o <<= 1) top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, o));
  const int bits = max(top & 0xffffu, top >> 16);  // bf16
  int k = 8 - ((bits >> 7) - 127) - ((bits & 0x7f) > 0x60 ? 1 : 0);
  k = bits ? min(max(k, -120), 100) : 0;
  const float up = __uint_as_float((uint32_t)(127 + k) << 23);
  uint32_t hi[4], lo[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 x = __floats2half2_rn(__uint_as_float(w[i] << 16) * up,
                                        __uint_as_float(w[i] & 0xffff0000u) * up);
    hi[i] = e4m3_of(x);
    const __half2 rest = __hsub2(x, half_of(hi[i]));
    lo[i] = kTimes16 ? e4m3_of(__hmul2(rest, __float2half2_rn(16.f)))
                     : __nv_cvt_halfraw2_to_fp8x2(rest, __NV_SATFINITE, __NV_E5M2);
  }
  return SplitQ{make_uint2(hi[0] | hi[1] << 16, hi[2] | hi[3] << 16),
                make_uint2(lo[0] | lo[1] << 16, lo[2] | lo[3] << 16),
                __uint_as_float(bits < 0x7f80 ? (uint32_t)(127 - k) << 23 : 0x7fc00000u)};
}

// Byte offset of 8 bytes `c8` (elements 8 c8 ..) of e4m3 row `r`, rows of kD.
template <int kD>
__device__ __forceinline__ uint32_t e4m3_row_offset(int r, int c8) {
  const int c16 = c8 >> 1;
  return (kD == 64 ? r * 64 + ((c16 ^ ((r >> 1) & 3)) << 4) : r * 128 + ((c16 ^ (r & 7)) << 4)) +
         8 * (c8 & 1);
}

__device__ __forceinline__ bool token_sees(const CacheFwdParams& p, int b, int t, int u) {
  if (!p.mask) return u <= t;
  return (p.mask[((long long)b * p.T + t) * p.W + (u >> 5)] >> (u & 31)) & 1u;
}

// Adds to x (columns [col, col + n) of token t) the non-finite elements of the
// drafted rows flagged in `bad` that t sees.  Rare: only where a drafted row
// of this piece holds one.
template <bool kE4m3>
__device__ __noinline__ void add_nonfinite(const CacheFwdParams& p, int b, int h, int start,
                                           const uint32_t* bad, int t, int col, int n, float* x) {
  for (int i = 0; i < p.W; ++i)
    for (uint32_t m = bad[i]; m; m &= m - 1) {
      const int u = 32 * i + __ffs(m) - 1;
      if (!token_sees(p, b, t, u)) continue;
      const CacheRow at = cache_row(p.c, b, (long long)start + u);
      if (at.page < 0) continue;
      const long long off = (long long)at.page * p.c.l.b + h * p.c.l.h + at.row * p.c.l.n + col;
      for (int e = 0; e < n; ++e) {
        if (kE4m3) {
          const uint8_t v = static_cast<const uint8_t*>(p.c.v)[off + e];
          if ((v & 0x7f) == 0x7f) x[e] = __uint_as_float(0x7fc00000u);
        } else {
          const float v = __bfloat162float(static_cast<const __nv_bfloat16*>(p.c.v)[off + e]);
          if (!(fabsf(v) < INFINITY)) x[e] += v;
        }
      }
    }
}

// Makes V rows of a tile that reaches past start[b] safe to multiply by zero: kRows rows
// of the tile from row0 on, by this warp.  Rows behind the sequence become zero;
// non-finite elements of drafted rows too, and the rows are flagged.  The tile is of
// bf16, or f16 converted from e4m3 (kF16), or (kBytes) e4m3 itself.  Where no row is
// behind the sequence a look without branches mostly finds that there is nothing to do
// (1024 tokens over an empty e4m3 cache 82 -> 68 us, bf16 50 -> 38; unrolled further 67
// and 36, but then the code that the main loops share a cache with makes them 2 % slower).
template <typename C, int kRows, bool kBytes, bool kF16 = false>
__device__ __noinline__ void clean_rows(uint8_t* tile, int start, int klen, int row0, int key_base,
                                        uint32_t* bad, int* any_bad) {
  constexpr int kChunkRow = kF16 ? 128 : C::kChunkRow, kChunks = kF16 ? C::D / 64 : C::kChunks;
  constexpr int kPieces = kChunkRow / 16;  // 16-byte pieces of a chunk's row
  // all-ones exponent fields (bf16: 8 bits, f16: 5; e4m3's NaN: 7 bits); one more
  // there carries into the sign's place
  constexpr uint32_t kAll = kBytes ? 0x7f7f7f7fu : kF16 ? 0x7c007c00u : 0x7f807f80u;
  constexpr uint32_t kOne = kBytes ? 0x01010101u : kF16 ? 0x04000400u : 0x00800080u;
  const int first = max(row0, start - key_base), row1 = row0 + kRows;
  if (key_base + row1 <= klen) {
    uint32_t found = 0;
#pragma unroll 1
    for (int c = 0; c < kChunks; ++c) {
      const uint4* const at = reinterpret_cast<const uint4*>(tile + c * 128 * kChunkRow);
#pragma unroll 2
      for (int j = 0; j < kRows * kPieces / 32; ++j) {
        const int i = row0 * kPieces + 32 * j + (threadIdx.x & 31);
        if (i < first * kPieces) continue;
        const uint4 v = at[i];
        found |= ((v.x & kAll) + kOne) | ((v.y & kAll) + kOne) | ((v.z & kAll) + kOne) |
                 ((v.w & kAll) + kOne);
      }
    }
    if (!__any_sync(0xffffffffu, found & (kBytes ? 0x80808080u : 0x80008000u))) return;
  }
#pragma unroll 1
  for (int c = 0; c < kChunks; ++c) {
    uint4* const at = reinterpret_cast<uint4*>(tile + c * 128 * kChunkRow);
#pragma unroll 1
    for (int i = first * kPieces + (threadIdx.x & 31); i < row1 * kPieces; i += 32) {
      const int key = key_base + i / kPieces;
      uint4 v = make_uint4(0u, 0u, 0u, 0u);
      if (key < klen) {
        v = at[i];
        uint32_t* x = reinterpret_cast<uint32_t*>(&v);
        uint32_t found = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t m = kBytes ? __vcmpeq4(x[k] & kAll, kAll) : __vcmpeq2(x[k] & kAll, kAll);
          found |= m;
          x[k] &= ~m;
        }
        if (!found) continue;
        atomicOr(&bad[(key - start) >> 5], 1u << ((key - start) & 31));
        *any_bad = 1;
      }
      at[i] = v;
    }
  }
  fence_proxy_async_smem();
}

// ---------------------------------------------------------------------------
// Joining the partial results of a unit that several CTAs share: weights
// 2^(m_i - m), then O = sum w_i O_i / sum w_i l_i.  One warp per row, or four where
// a unit has many parts; grid.y, z: the units themselves when they are few, else the
// borders between runs (a unit is cut by at least one; its first border does the
// work).  Latency is what it costs: a row's first parts are asked for along with its
// statistics (one token over 1000 keys 10.6 -> 10.1 us).
// ---------------------------------------------------------------------------
constexpr int kJoinWarps = 4;

template <int kD, int kRows, int kShare>
__global__ void __launch_bounds__(32 * kJoinWarps)
    fa_cache_join_kernel(const __grid_constant__ CacheFwdParams p, int grid, int by_unit) {
  constexpr int kPer = kD / 32;                 // floats per lane
  constexpr int kMost = (kCacheMaxCtas + 31) / 32;  // parts per lane
  __shared__ float s_o[kShare > 1 ? kJoinWarps : 1][kShare > 1 ? kD : 1];
  __shared__ float s_wt[kJoinWarps][32 * kMost];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // start and q_len are older than the main kernel, which waited for their
  // writer before it let this one start; its results are waited for below, on
  // every path (a grid that ended earlier would let the next kernel pass)
  // grid: row blocks, heads x row tiles (or borders), sequences (or 1)
  constexpr int kRowsHere = kJoinWarps / kShare;
  constexpr int kAtOnce = 4;  // parts in flight
  const int share = kShare == 1 ? 0 : warp;
  int b, h = 0, rt = 0, c0 = 0, c1 = 0, rows = 0;
  bool first_odd = false;  // the first part is its CTA's last piece, not its first
  {
    int first, u0 = 0;
    SeqInfo s{};
    bool cut = false;
    b = blockIdx.z;
    const WholeOrTiles all = list_of<kRows>(p, grid, b, &first);
    const TileList list(all.whole ? 0 : all.total, grid);
    if (all.whole) {
      // nothing was cut
    } else if (by_unit) {
      s = seq_info<kRows>(p, b);
      cut = s.tiles > 0 && (int)blockIdx.y < p.c.heads * s.row_tiles;
      h = s.row_tiles <= 1 ? blockIdx.y : blockIdx.y / s.row_tiles;
      rt = blockIdx.y - h * s.row_tiles;
      u0 = first + blockIdx.y * s.tiles;
    } else if ((int)blockIdx.y + 1 < list.ctas) {
      const int border = list.begin(blockIdx.y + 1);
      b = find_seq<kRows>(p, border, false, &first, &s);
      const int unit = (border - first) / s.tiles;
      h = s.row_tiles <= 1 ? unit : unit / s.row_tiles;
      rt = unit - h * s.row_tiles;
      u0 = first + unit * s.tiles;
      cut = u0 < border && list.begin(blockIdx.y) <= u0;
    }
    if (cut) {
      c0 = list.cta_of(u0);
      c1 = list.cta_of(u0 + s.tiles - 1);
      rows = min(kRows, s.q * p.group - rt * kRows);
      first_odd = list.begin(c0) < u0;
    }
  }
  pdl_wait();
  pdl_launch_dependents();
  if (c0 == c1) return;
  // a CTA's first piece is in its even slot: only the unit's first part may not be
  auto slot = [&](int c) {
    return p.ws + (2 * c + (c == c0 && first_odd ? 1 : 0)) * slot_floats<kD, kRows>();
  };
#pragma unroll 1
  for (int row0 = blockIdx.x * kRowsHere; row0 < rows; row0 += gridDim.x * kRowsHere) {
    const int row = row0 + (kShare == 1 ? warp : 0);
    const bool on = row < rows;
    float o[kPer] = {}, mm = -INFINITY, lt = 0.f;
    if (on) {
      // kAtOnce parts are on their way ahead: the first while the statistics are
      constexpr int kStep = kShare * kAtOnce;
      float x[kAtOnce][kPer];
      [[maybe_unused]] float y[kAtOnce][kPer];
      auto fetch = [&](int c, float (*to)[kPer]) {
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
          if (c + i * kShare > c1) continue;
          const float* sl = slot(c + i * kShare) + row * kD + lane * kPer;
          if constexpr (kPer == 4)
            *reinterpret_cast<float4*>(to[i]) = *reinterpret_cast<const float4*>(sl);
          else
            *reinterpret_cast<float2*>(to[i]) = *reinterpret_cast<const float2*>(sl);
        }
      };
      auto add = [&](int c, const float (*from)[kPer]) {
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
          if (c + i * kShare > c1) continue;
          const float w = s_wt[warp][c + i * kShare - c0];
#pragma unroll
          for (int e = 0; e < kPer; ++e) o[e] = fmaf(w, from[i][e], o[e]);
        }
      };
      fetch(c0 + share, x);
      float m[kMost], l[kMost];
#pragma unroll
      for (int k = 0; k < kMost; ++k) {
        const int c = c0 + lane + 32 * k;
        m[k] = -INFINITY;
        l[k] = 0.f;
        if (c <= c1) {
          m[k] = slot(c)[kRows * kD + row];
          l[k] = slot(c)[kRows * kD + kRows + row];
        }
      }
#pragma unroll
      for (int k = 0; k < kMost; ++k) mm = fmaxf(mm, m[k]);
#pragma unroll
      for (int k = 16; k > 0; k >>= 1) mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, k));
#pragma unroll
      for (int k = 0; k < kMost; ++k) {
        const float w = m[k] == -INFINITY ? 0.f : ex2(m[k] - mm);
        lt += l[k] * w;  // NaN stays NaN
        s_wt[warp][lane + 32 * k] = w;
      }
#pragma unroll
      for (int k = 16; k > 0; k >>= 1) lt += __shfl_xor_sync(0xffffffffu, lt, k);
      __syncwarp();
      if constexpr (kShare > 1) {  // many parts
#pragma unroll 1
        for (int c = c0 + share; c <= c1; c += 2 * kStep) {
          const bool more = c + kStep <= c1;
          if (more) fetch(c + kStep, y);
          add(c, x);
          if (!more) break;
          fetch(c + 2 * kStep, x);
          add(c + kStep, y);
        }
      } else {
#pragma unroll 1
        for (int c = c0; c <= c1; c += kStep) {
          add(c, x);
          fetch(c + kStep, x);
        }
      }
      __syncwarp();
    }
    if constexpr (kShare > 1) {
      __syncthreads();  // the last row's sums are read
#pragma unroll
      for (int e = 0; e < kPer; ++e) s_o[warp][lane * kPer + e] = o[e];
      __syncthreads();
      if (share != 0) continue;
#pragma unroll
      for (int k = 1; k < kShare; ++k)
#pragma unroll
        for (int e = 0; e < kPer; ++e) o[e] += s_o[k][lane * kPer + e];
    }
    if (!on) continue;
    const int g = rt * kRows + row, t = row_token(p, g), hq = h * p.group + g - t * p.group;
    const bool empty = lt == 0.f;
    const float inv = empty ? 0.f : 1.f / lt;
    uint32_t* dst = reinterpret_cast<uint32_t*>(p.o + row_offset(p.lo, b, hq, t) + lane * kPer);
#pragma unroll
    for (int e = 0; e < kPer; e += 2) dst[e / 2] = pack_bf16(o[e] * inv, o[e + 1] * inv);
    if (lane == 0)
      p.lse[((size_t)b * p.Hq + hq) * p.T + t] = empty ? -INFINITY : (mm + log2f(lt)) * kLn2;
  }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
// Query rows of a unit: lanes hold keys up to 32 rows (8, 16 or 32 columns),
// query rows beyond (64, each twice; 128; or two CTAs' 128 each).
inline int cache_fwd_rows(int rows) {
  return rows <= 32 ? 32 : rows <= 64 ? 64 : rows <= 128 ? 128 : 256;
}

// Launches the main kernel and, unless no unit can be cut, the joining kernel behind it.
// Up to 512 rows of capacity (1024, where a third of the CTAs or more, and no CTA twice,
// would have one) units are never cut, whatever their lengths: without the second kernel
// a call is 1.4 us shorter.
template <int kD, int kRows, auto kKernel>
cudaError_t launch_cache_pair(int threads, int smem, int ctas_per_run, const CacheMaps& m,
                              CacheFwdParams p, cudaStream_t s) {
  const int sms = device_sm_count();
  if (sms <= 0) return cudaErrorInvalidDevice;
  const int ctas = (sms < kCacheMaxCtas ? sms : kCacheMaxCtas) / ctas_per_run * ctas_per_run;
  const int grid = ctas / ctas_per_run;  // runs
  if (grid < 1) return cudaErrorInvalidConfiguration;
  cudaError_t e = allow_smem_once<kKernel>(smem);
  if (e != cudaSuccess) return e;
  const int row_tiles = tiles_of(p.T * p.group, kRows);
  const long long units = (long long)p.B * p.c.heads * row_tiles;
  p.whole = p.c.capacity <= (3 * units >= grid && units <= grid ? 1024 : 512);
  if (p.whole)
    return launch_pdl(kKernel, dim3(units < grid ? (int)units * ctas_per_run : ctas), dim3(threads),
                      smem, s, m.k, m.v, p);
  e = launch_pdl(kKernel, dim3(ctas), dim3(threads), smem, s, m.k, m.v, p);
  if (e != cudaSuccess) return e;
  const int rows = p.T * p.group < kRows ? p.T * p.group : kRows;
  const bool by_unit = units < grid - 1;
  auto join = [&](auto kernel, int rows_here) {
    // about eight blocks per SM, each over the rows of one unit
    const int most = tiles_of(rows, rows_here);
    const int want = (int)(8ll * sms / (by_unit ? units : grid - 1)) + 1;
    return launch_pdl(kernel,
                      dim3(want < most ? want : most, by_unit ? p.c.heads * row_tiles : grid - 1,
                           by_unit ? p.B : 1),
                      dim3(32 * kJoinWarps), 0, s, p, grid, (int)by_unit);
  };
  // eight parts to a unit or more: four warps to a row
  return units * 8 <= grid ? join(fa_cache_join_kernel<kD, kRows, kJoinWarps>, 1)
                           : join(fa_cache_join_kernel<kD, kRows, 1>, kJoinWarps);
}

// One function per format and orientation, each in a file of its own.
cudaError_t launch_cache_keys_bf16(const CacheMaps& m, const CacheFwdParams& p, cudaStream_t s);
cudaError_t launch_cache_keys_e4m3(const CacheMaps& m, const CacheFwdParams& p, cudaStream_t s);
cudaError_t launch_cache_rows_bf16(const CacheMaps& m, const CacheFwdParams& p, cudaStream_t s);
cudaError_t launch_cache_rows_e4m3(const CacheMaps& m, const CacheFwdParams& p, cudaStream_t s);

}  // namespace fa
