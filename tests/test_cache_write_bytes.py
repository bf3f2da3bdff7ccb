"""What cache_write stores, byte for byte: scale = (largest finite magnitude) / 448 and value =
x / scale in fp32, rounded to e4m3 (nearest, ties to even), as the C header says."""
import math

import pytest
import torch

import _cache_ref as ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("spread", [2.0 ** -60, 2.0 ** -20, 1.0, 300.0, 2.0 ** 90])
def test_written_bytes(fa, d, spread):
    B, H, T = 3, 4, 1500
    g = torch.Generator().manual_seed(70)
    # rows of every size and shape: normal, a few large elements, few significant bits
    x = torch.randn(2, B, H, T, d, generator=g) * spread
    x[:, :, :, ::3] *= torch.exp2(4 * torch.randn(2, B, H, 500, d, generator=g))
    x[:, :, :, 1::3] = x[:, :, :, 1::3].to(ref.F8).float() if spread == 1.0 else x[:, :, :, 1::3]
    x = x.to(torch.bfloat16)
    x[0, 0, 0, 0], x[0, 0, 0, 1, 3], x[1, 1, 1, 1, 4] = 0.0, math.inf, -math.inf
    table = torch.arange(B * 24, dtype=torch.int32, device="cuda").view(B, 24)
    cache = fa.KVCache.empty(B * 24, 64, H, d, ref.F8, table)
    k, v = x.cuda()
    fa.cache_write(cache, k, v, torch.zeros(B, dtype=torch.int32, device="cuda"))
    for side, (t, s) in enumerate(((cache.k, cache.k_scale), (cache.v, cache.v_scale))):
        got = t.view(torch.uint8).view(B, 24, H, 64, d).transpose(2, 3).reshape(B, -1, H, d)
        got = got[:, :T].transpose(1, 2).cpu().view(ref.F8).float()
        sc = s.view(B, 24, H, 64).transpose(2, 3).reshape(B, -1, H)[:, :T].transpose(1, 2).cpu()
        y = x[side].float()
        fin = torch.where(y.isfinite(), y, 0.0)
        want = (fin.abs().amax(-1) / 448.0).clamp_min(2.0 ** -64)
        assert torch.equal(sc, want)
        q = (y / want[..., None]).clamp(-448.0, 448.0).to(ref.F8).float()
        assert torch.equal(got, q), int((got != q).sum())
