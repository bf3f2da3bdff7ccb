"""The README's decoding example, run as it stands."""
import os
import re

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_decoding_example(fa):
    text = open(os.path.join(ROOT, "README.md")).read()
    block = next(b for b in re.findall(r"```python\n(.*?)```", text, re.S) if "decode_step" in b)
    code = "\n".join(line.strip() for line in block.splitlines())
    B, Hkv, Hq, d, T = 3, 2, 4, 64, 70
    g = torch.Generator().manual_seed(80)
    rnd = lambda h, t: torch.randn(B, h, t, d, generator=g).to(torch.bfloat16).cuda()
    k, v, q1, k1, v1 = rnd(Hkv, T), rnd(Hkv, T), rnd(Hq, 1), rnd(Hkv, 1), rnd(Hkv, 1)
    start = torch.zeros(B, dtype=torch.int32, device="cuda")
    q_len = torch.tensor([70, 33, 1], dtype=torch.int32, device="cuda")
    rope = fa.Rope(fa.rope_frequencies(d)[0])
    names = dict(torch=torch, fa=fa, B=B, Hkv=Hkv, d=d, k=k, v=v, q1=q1, k1=k1, v1=v1, start=start,
                 q_len=q_len, rope=rope, n=T + 1, pos=q_len[:, None])
    exec(code, names)
    o = names["o"]
    for b in range(B):                       # the new token sees its whole prompt and itself
        n = int(q_len[b])
        at = torch.arange(n + 1, dtype=torch.int32, device="cuda")
        keys = torch.cat([k[b:b + 1, :, :n], k1[b:b + 1]], 2)
        vals = torch.cat([v[b, :, :n], v1[b]], 1).float()
        keys = fa.rope(keys, None, rope, at)[0][0].float()
        qq = fa.rope(q1[b:b + 1], None, rope, at[n:])[0][0].float()
        for h in range(Hq):
            s = (keys[h // 2] @ qq[h, 0]) * d ** -0.5
            want = s.softmax(0) @ vals[h // 2]
            # e4m3 keys and values: 2^-4 of each element; scores move by 2^-4 sum |q k| scale at
            # most, in the mean far less: an eighth of the values' size tells the two answers apart
            assert (o[b, h, 0].float() - want).abs().mean() <= 0.125 * vals.abs().mean()
