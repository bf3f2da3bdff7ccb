// Attention over the key/value cache: TMA descriptors, workspace and dispatch.
#include "fa_cache_fwd.cuh"

namespace fa {

size_t cache_fwd_workspace(int B, int Hq, int Hkv, int T, int d) {
  // two partial results per run: its first and its last unit (256 rows: two CTAs to a run)
  const int rows = cache_fwd_rows(T * (Hq / Hkv));
  const int runs = rows == 256 ? kCacheMaxCtas / 2 : kCacheMaxCtas;
  return (size_t)2 * runs * rows * (d + 2) * sizeof(float);
}

cudaError_t launch_cache_fwd(const CacheFwdArgs& a, cudaStream_t s) {
  const CacheView& c = a.c;
  CacheFwdParams p{};
  p.q = static_cast<const __nv_bfloat16*>(a.q);
  p.o = static_cast<__nv_bfloat16*>(a.o);
  p.lse = a.lse;
  p.lq = a.lq;
  p.lo = a.lo;
  p.c = c;
  p.start = a.start;
  p.q_len = a.q_len;
  p.mask = a.mask;
  p.ws = a.ws;
  p.B = a.B;
  p.Hq = a.Hq;
  p.T = a.T;
  p.W = (a.T + 31) / 32;
  p.group = a.Hq / c.heads;
  p.group_inv = (uint32_t)(((1ull << 32) + p.group - 1) / p.group);  // unused when group is 1
  p.box_rows = c.table && c.page_size < 128 ? c.page_size : 128;
  p.scale_log2 = a.scale * kLog2e;
  p.status = a.status;
  CacheMaps m{};
  const int esize = c.ks ? 1 : 2;
  if (!encode_cache_map(&m.k, c.k, c.l, c, esize, p.box_rows) ||
      !encode_cache_map(&m.v, c.v, c.l, c, esize, p.box_rows))
    return cudaErrorInvalidValue;
  // e4m3 units of 17 to 32 rows: P costs the keys kernel three terms per element (of two it
  // was), the rows kernel one f16 (16 sequences of 16 K keys, 32 rows: 163, with two terms,
  // and 133 us at d = 128, 157 and 104 at d = 64; of 16 rows: 91 and 98 at d = 64, 64
  // sequences of up to 8 K keys at d = 128: 160 and 204); bf16's cost the keys kernel less
  // than its loads
  const bool keys = p.T * p.group <= (c.ks ? 16 : 32);
  p.slack = keys && !c.ks ? 4.f : 5.5f;
  if (!c.ks) return keys ? launch_cache_keys_bf16(m, p, s) : launch_cache_rows_bf16(m, p, s);
  return keys ? launch_cache_keys_e4m3(m, p, s) : launch_cache_rows_e4m3(m, p, s);
}

}  // namespace fa
