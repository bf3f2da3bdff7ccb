// Writing new rows into the key/value cache and reading rows back.
//
// Write: a row's scale is its largest finite magnitude / 448 (the e4m3
// maximum), so the row uses the whole range of the format whatever its size:
// the rounding is 2^-4 relative at most down to 2^-15 of that magnitude.  Keys
// are rotated on the way in (fp32, rounded once), which saves writing and
// reading the rotated bf16 keys.  Both kernels are bound by memory: a bf16 row
// of 2 d bytes on one side, d + 4 bytes (e4m3) on the other.  d/16 neighbouring
// lanes hold a row, 16 elements each; a thread keeps its token, its slot and K or
// V, and steps through the heads, a few of them in flight.  The write of 23 K tokens
// (four prompts of up to 8 K) x 8 heads takes 33.8 us where the memory needs 21.5.
// Neither the issue (68 %: some 120 instructions per 16 elements) nor the memory
// (42 %) is full: 27 warps per SM each go through a row's chain of copy, rotation,
// largest magnitude over the lanes and conversion.  (With the place of every row
// looked up and divided out anew there were 390 instructions.)
#include "fa_cache.cuh"

namespace fa {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTokens = 32;  // of a block: 16 KB of angles at most

struct RwParams {
  CacheView c;
  const int32_t* start;
  const int32_t* len;
  const void* in[2];
  void* out[2];
  Layout l[2];
  RopeArgs r;
  int T, tokens;  // tokens: B T
  RowSplit split;
  int* status;
};

// A thread's token: its place in the cache and in the dense tensors.
struct Token {
  CacheRow at;  // page -1: no such row
  int b, n;
  bool on;  // one of the sequence's tokens
};
__device__ __forceinline__ Token thread_token(const RwParams& p, const TokenIndex& first, int nt, int t,
                                              int site) {
  Token k;
  const TokenIndex i(first, min(t, nt - 1), p.T);
  k.b = i.b;
  k.n = i.n;
  k.on = t < nt && k.n < clamped_len(p.len, k.b, p.T);
  k.at = CacheRow{-1, 0};
  if (k.on) {
    k.at = cache_row(p.c, k.b, (p.start ? (long long)__ldg(p.start + k.b) : 0ll) + k.n);
    if (k.at.page < 0) report_page(p.status, site);
  }
  return k;
}

// Largest magnitude of a row (NaN left out) from its S lanes' 16 elements each.
template <int S>
__device__ __forceinline__ float row_max(const float* x) {
  float m[2] = {0.f, 0.f};
#pragma unroll
  for (int e = 0; e < 16; e += 2) m[(e >> 1) & 1] = max3(m[(e >> 1) & 1], fabsf(x[e]), fabsf(x[e + 1]));
  float y = fmaxf(m[0], m[1]);
#pragma unroll
  for (int o = 1; o < S; o <<= 1) y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, o));
  return y;
}

constexpr int kDepth = 2;  // rows of a thread in flight (four: no faster)
using WriteRing = RowRing<2, kDepth, kThreads>;

template <bool kE4m3, int D>
__global__ void __launch_bounds__(kThreads, 4) cache_write_kernel(const RwParams p) {
  constexpr int S = D / 16;  // lanes of a row
  extern __shared__ __align__(16) float2 cs[];  // [token][pair], then the ring
  pdl_wait();
  pdl_launch_dependents();
  const int pairs = p.r.freq ? p.r.dim / 2 : 0;
  const int tok0 = blockIdx.x * p.split.tokens, nt = min(p.split.tokens, p.tokens - tok0);
  const int s = threadIdx.x % S, t = (threadIdx.x / S) & (p.split.tokens - 1);
  const int lane = threadIdx.x / S / p.split.tokens;
  // a block of padding alone has nothing to do
  const TokenIndex first_token(tok0, p.T);
  if (p.len && first_token.n + nt <= p.T && first_token.n >= clamped_len(p.len, first_token.b, p.T))
    return;
  const int side = lane & 1, first = lane >> 1, step = p.split.lanes >> 1;  // K or V; heads
  const int H = p.c.heads;
  const Token k = thread_token(p, first_token, nt, t, 3001);
  const Slot sl = slot_of(s, side ? 0 : 2 * pairs, D);
  const __nv_bfloat16* const in =
      static_cast<const __nv_bfloat16*>(p.in[side]) + row_offset(p.l[side], k.b, 0, k.n);
  const long long in_head = p.l[side].h;
  WriteRing ring(cs + p.split.tokens * pairs);
  auto ask = [&](int i, int h) {
    const __nv_bfloat16* const at = in + h * in_head;
    ring.ask(i, k.on && h < H, [&](int g) { return at + (g ? sl.second : sl.first); });
  };
#pragma unroll 1
  for (int i = 0; i < kDepth; ++i) ask(i, first + i * step);
  if (pairs)
    block_angles(cs, p.r, first_token, nt, p.T, [&](int b, int n) {
      return p.r.pos ? __ldg(p.r.pos + b * p.r.pos_stride + n) : __ldg(p.start + b) + n;
    });
  __syncthreads();
  SlotTurn a;
  if (sl.turned && t < nt) a.load(cs + t * pairs, sl, p.r.interleaved, 1.f);
  const bool on = k.on && k.at.page >= 0;
  const long long page = max(k.at.page, 0);
  uint8_t* const out = static_cast<uint8_t*>(side ? p.c.v : p.c.k) +
                       (page * p.c.l.b + k.at.row * p.c.l.n) * (kE4m3 ? 1 : 2);
  float* const out_scale = kE4m3 ? (side ? p.c.vs : p.c.ks) + page * p.c.sb + k.at.row : nullptr;
#pragma unroll 1
  for (int h0 = 0; h0 < H; h0 += step) {  // whole warps: a row's lanes shuffle
    const int h = h0 + first;
    const bool mine = on && h < H;
    ring.wait();
    float x[16];
    auto value = [&] {
      unpack8(ring.get(0), x);
      unpack8(ring.get(1), x + 8);
      if (sl.turned) a.turn(x, p.r.interleaved);
    };
    value();
    if constexpr (kE4m3) {
      float amax = row_max<S>(x);
      // infinities out of the scale (rare: the vote keeps the shuffles whole)
      const bool inf = __any_sync(0xffffffffu, !(amax < INFINITY));
      if (inf) {
#pragma unroll
        for (int e = 0; e < 16; ++e) x[e] = fabsf(x[e]) < INFINITY ? x[e] : 0.f;
        amax = row_max<S>(x);
        value();
      }
      // Both divisions, exact to the last bit, are products with an inverse and its rest
      // (23 K tokens of 8 heads take 33.8 us; with a division each 47; with the inverse
      // alone 33.2, 59 % of the scales in the last bit and a byte in a thousand a step off).
      constexpr float kInv = 1.f / kE4m3Max, kInvRest = (float)(1.0 / kE4m3Max - kInv);
      const float scale = fmaxf(fmaf(amax, kInv, amax * kInvRest), kMinScale);
      if (inf) {
#pragma unroll
        for (int e = 0; e < 16; ++e)
          if (fabsf(x[e]) == INFINITY) x[e] = copysignf(kE4m3Max * scale, x[e]);
      }
      if (mine) {
        const float up = __fdividef(1.f, scale), rest = fmaf(-up, scale, 1.f) * up;
        const float2 up2 = make_float2(up, up), rest2 = make_float2(rest, rest);
#pragma unroll
        for (int e = 0; e < 16; e += 2) {
          const float2 v = make_float2(x[e], x[e + 1]), y = fma2(v, up2, mul2(v, rest2));
          x[e] = y.x;
          x[e + 1] = y.y;
        }
        uint8_t* const at = out + h * p.c.l.h;
        *reinterpret_cast<uint2*>(at + sl.first) = make_uint2(e4m3x4(x), e4m3x4(x + 4));
        *reinterpret_cast<uint2*>(at + sl.second) = make_uint2(e4m3x4(x + 8), e4m3x4(x + 12));
        if (s == 0) out_scale[h * p.c.sh] = scale;
      }
    } else if (mine) {
      __nv_bfloat16* const at = reinterpret_cast<__nv_bfloat16*>(out) + h * p.c.l.h;
      *reinterpret_cast<uint4*>(at + sl.first) = pack8(x);
      *reinterpret_cast<uint4*>(at + sl.second) = pack8(x + 8);
    }
    ask(ring.at, h + kDepth * step);
    ring.next();
  }
}

template <bool kE4m3, int D, int kUnroll>
__global__ void __launch_bounds__(kThreads, 4) cache_read_kernel(const RwParams p) {
  constexpr int S = D / 16;
  pdl_wait();
  pdl_launch_dependents();
  const int tok0 = blockIdx.x * p.split.tokens, nt = min(p.split.tokens, p.tokens - tok0);
  const int s = threadIdx.x % S, t = (threadIdx.x / S) & (p.split.tokens - 1);
  const int lane = threadIdx.x / S / p.split.tokens;
  const int side = lane & 1, first = lane >> 1, step = p.split.lanes >> 1;  // K or V; heads
  const Token k = thread_token(p, TokenIndex(tok0, p.T), nt, t, 3002);
  if (!k.on) return;  // past the sequence's rows: left as it was
  const int H = p.c.heads;
  const bool there = k.at.page >= 0;  // else zeros
  const Slot sl = slot_of(s, 0, D);
  const long long page = max(k.at.page, 0);
  const uint8_t* const in = static_cast<const uint8_t*>(side ? p.c.v : p.c.k) +
                            (page * p.c.l.b + k.at.row * p.c.l.n) * (kE4m3 ? 1 : 2);
  const float* const in_scale = kE4m3 ? (side ? p.c.vs : p.c.ks) + page * p.c.sb + k.at.row : nullptr;
  __nv_bfloat16* const out =
      static_cast<__nv_bfloat16*>(p.out[side]) + row_offset(p.l[side], k.b, 0, k.n);
  const long long out_head = p.l[side].h;
  for (int h0 = first; h0 < H; h0 += step * kUnroll) {
    uint4 raw[kUnroll][kE4m3 ? 1 : 2];
    float scale[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int h = h0 + u * step;
      raw[u][0] = make_uint4(0u, 0u, 0u, 0u);
      if (!kE4m3) raw[u][kE4m3 ? 0 : 1] = raw[u][0];
      scale[u] = 0.f;
      if (there && h < H) {
        if constexpr (kE4m3) {
          const uint2 lo = __ldcs(reinterpret_cast<const uint2*>(in + h * p.c.l.h + sl.first));
          const uint2 hi = __ldcs(reinterpret_cast<const uint2*>(in + h * p.c.l.h + sl.second));
          raw[u][0] = make_uint4(lo.x, lo.y, hi.x, hi.y);
          scale[u] = __ldg(in_scale + h * p.c.sh);
        } else {
          const __nv_bfloat16* at = reinterpret_cast<const __nv_bfloat16*>(in) + h * p.c.l.h;
          raw[u][0] = __ldcs(reinterpret_cast<const uint4*>(at + sl.first));
          raw[u][kE4m3 ? 0 : 1] = __ldcs(reinterpret_cast<const uint4*>(at + sl.second));
        }
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int h = h0 + u * step;
      if (h >= H) break;
      __nv_bfloat16* const at = out + h * out_head;
      if constexpr (kE4m3) {
        float x[16];
        const uint32_t e[4] = {raw[u][0].x, raw[u][0].y, raw[u][0].z, raw[u][0].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) from_e4m3x4(e[i], x + 4 * i);
#pragma unroll
        for (int j = 0; j < 16; ++j) x[j] *= scale[u];
        *reinterpret_cast<uint4*>(at + sl.first) = pack8(x);
        *reinterpret_cast<uint4*>(at + sl.second) = pack8(x + 8);
      } else {
        *reinterpret_cast<uint4*>(at + sl.first) = raw[u][0];
        *reinterpret_cast<uint4*>(at + sl.second) = raw[u][kE4m3 ? 0 : 1];
      }
    }
  }
}

cudaError_t fill(const CacheCall& a, RwParams* p) {
  p->c = a.c;
  p->start = a.start;
  p->len = a.len;
  p->in[0] = a.k;
  p->in[1] = a.v;
  p->out[0] = a.ko;
  p->out[1] = a.vo;
  p->l[0] = a.lk;
  p->l[1] = a.lv;
  p->r = a.rope;
  p->T = a.T;
  const long long tokens = (long long)a.B * a.T;
  if (tokens > 0x7fffffffll - kMaxTokens) return cudaErrorInvalidConfiguration;
  p->tokens = (int)tokens;
  p->status = a.status;
  return cudaSuccess;
}

template <bool kWrite, auto kKernel>
cudaError_t go(RwParams& p, cudaStream_t s) {
  p.split = row_split(kThreads, p.c.d / 16, 2 * p.c.heads, p.tokens, device_sm_count(), kMaxTokens);
  size_t smem = 0;
  if (kWrite) {
    const cudaError_t e = allow_smem_once<kKernel>(kMaxTokens * 64 * sizeof(float2) + WriteRing::bytes(kDepth));
    if (e != cudaSuccess) return e;
    smem = WriteRing::bytes((2 * p.c.heads + p.split.lanes - 1) / p.split.lanes);
    if (p.r.freq) smem += sizeof(float2) * p.split.tokens * (p.r.dim / 2);
  }
  return launch_pdl(kKernel, dim3(tiles_of(p.tokens, p.split.tokens)), dim3(kThreads), smem, s, p);
}

}  // namespace

cudaError_t launch_cache_write(const CacheCall& a, cudaStream_t s) {
  RwParams p{};
  cudaError_t e = fill(a, &p);
  if (e != cudaSuccess) return e;
  if (a.c.ks)
    return a.c.d == 64 ? go<true, cache_write_kernel<true, 64>>(p, s)
                       : go<true, cache_write_kernel<true, 128>>(p, s);
  return a.c.d == 64 ? go<true, cache_write_kernel<false, 64>>(p, s)
                     : go<true, cache_write_kernel<false, 128>>(p, s);
}

cudaError_t launch_cache_read(const CacheCall& a, cudaStream_t s) {
  RwParams p{};
  cudaError_t e = fill(a, &p);
  if (e != cudaSuccess) return e;
  if (a.c.ks)
    return a.c.d == 64 ? go<false, cache_read_kernel<true, 64, 4>>(p, s)
                       : go<false, cache_read_kernel<true, 128, 4>>(p, s);
  return a.c.d == 64 ? go<false, cache_read_kernel<false, 64, 2>>(p, s)
                     : go<false, cache_read_kernel<false, 128, 2>>(p, s);
}

}  // namespace fa
