"""Attention over an e4m3 cache where its roundings show: weights far below the largest,
queries of uneven channels, value scales far apart.  Bounds are derived at each test; p are
the weights (they sum to 1), v the values, sv the values' scales.  Every output is rounded
(2^-8 of it), and so is every weight (2^-8)."""
import math

import pytest
import torch

import _cache_ref as ref

pytestmark = pytest.mark.gpu
F64 = torch.float64


def _table(B, pages):
    """Every sequence reads the same pages."""
    return torch.arange(pages, dtype=torch.int32, device="cuda").expand(B, pages).contiguous()


def _attend64(c, q, k, v, kv_scales, sees=None):
    """(o, p @ |v|, max(p sv) per row) in 64 bits of rows q [R, d] over k, v [n, d] (bytes) with
    scales (ks, vs) [n]; sees: bool [R, n]."""
    k, v = (x.float().cpu().to(F64) for x in (k, v))
    ks, vs = (x.cpu().to(F64) for x in kv_scales)
    s = (q.float().cpu().to(F64) @ k.T) * ks * c
    if sees is not None:
        s = s.masked_fill(~sees, -math.inf)
    p = s.softmax(-1)
    pv = p * vs
    return pv @ v, pv @ v.abs(), pv.amax(-1)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G", [1, 8, 13, 16, 24])
@pytest.mark.parametrize("n,w,spread", [(1 << 13, 14, 0.0), (28000, 16, 0.0), (28000, 16, 1.0),
                                        (1 << 16, 17, 0.5), (1 << 17, 18, 0.0), (1 << 17, 20, 0.0)])
def test_a_dominant_key_and_a_long_tail(fa, d, G, n, w, spread):
    """One key at 0 and n keys of 2^-w of its weight and less; as many sequences as SMs, so that
    none is cut and one CTA walks all keys.  Beside its rounding a weight may be off by 2^-29 of
    the row's largest (weight times value scale): n of them."""
    B, page = 152, 256
    rows = -(-(n + 1) // page) * page
    g = torch.Generator().manual_seed(60)
    k = torch.zeros(rows, d)
    k[1:n + 1, 0] = -1.0
    v = (1.0 + 0.25 * torch.randn(rows, d, generator=g)) * 100
    v[0] = 30 * torch.randn(d, generator=g)
    ks = torch.full((rows,), float(w)) + spread * torch.rand(rows, generator=g)
    vs = torch.full((rows,), 0.01)
    lay = lambda x: x.view(rows // page, 1, page, *x.shape[1:])
    k, v = (x.clamp(-448, 448).to(ref.F8).cuda() for x in (k, v))
    ks, vs = ks.cuda(), vs.cuda()
    cache = fa.KVCache(lay(k), lay(v), lay(ks), lay(vs), _table(B, rows // page))
    q = torch.zeros(B, G, 1, d, dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 1.0
    scale = math.log(2.0)
    start = torch.full((B,), n, dtype=torch.int32, device="cuda")
    o, lse = fa.cache_forward(q, cache, start, scale=scale)
    want, mag, top = _attend64(scale, q[0, :1, 0], k[:n + 1], v[:n + 1], (ks[:n + 1], vs[:n + 1]))
    # the scores: the product's fp32 rounding, of 2^6 at most
    tol = (2.0 ** -8 * want.abs() + (2.0 ** -8 + 2.0 ** -16) * mag
           + n * 2.0 ** -29 * top[:, None] * v[:n + 1].float().abs().max().cpu())
    err = (o[:, :, 0].cpu().to(F64) - want).abs()
    assert (err <= tol).all(), (float(err.max()), float((err / want.abs()).max()), float((err / tol).max()))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T,G", [(1, 8), (1, 16), (1, 32), (5, 8), (20, 4), (16, 16)])
@pytest.mark.parametrize("ratio", [2.0 ** 10, 2.0 ** 13])
def test_queries_of_uneven_channels(fa, d, T, G, ratio):
    """One channel of q is `ratio` times the others, and its entry is the same in every key, so
    that the softmax does not see it; the others need all of bf16's bits and their errors would
    add up.  q is exact down to 2^-13 of its row's largest element and at most 2^-21 of that off;
    products are summed in fp32 (2^-21 d^(1/2) of sum |q k|, as in _cache_ref)."""
    n = 600
    c = ref.Cache(fa, 1, n + T, 1, d, 32, "e4m3", seed=62)
    c.ks.fill_(2.0 ** -10)
    c.vs.fill_(1.0 / 60)
    g = torch.Generator().manual_seed(61)
    sign = torch.where(torch.rand(c.k.shape[:3], generator=g) < 0.9, 1.0, -1.0)[..., None]
    c.k.copy_((sign * 256).expand(*c.k.shape).to(ref.F8))
    c.k[..., 5] = 2.0
    q = torch.full((1, G, T, d), 0.50390625 * ratio / 1024)
    q[..., 5] = ratio * torch.where(torch.rand(1, G, T, generator=g) < 0.5, 1.0, -1.0)
    q = q.to(torch.bfloat16).cuda()
    start = torch.tensor([n], dtype=torch.int32)
    scale = 2.0 * 1024 / ratio / d
    o, lse = fa.cache_forward(q, c.fa, start.cuda(), scale=scale)
    raw = c.raw()
    k, _ = c.rows(raw, 0, 0, 0, n + T)
    v, _ = c.rows(raw, 1, 0, 0, n + T)
    k, v = k[0], v[0]
    for t in range(T):
        kk, vv, qq = k[:n + t + 1], v[:n + t + 1], q[0, :, t].cpu().to(F64)
        s = qq @ kk.T * scale
        p = s.softmax(-1)
        want, mag = p @ vv, p @ vv.abs()
        ds = scale * (2.0 ** -21 * ratio * kk.abs().sum(-1).max()
                      + 2.0 ** -21 * d ** 0.5 * (qq.abs() @ kk.abs().T).amax(-1))
        el = (lse[0, :, t].cpu().to(F64) - s.logsumexp(-1)).abs()
        assert (el <= ds + 2.0 ** -18).all(), (float(el.max()), float(ds.max()))
        tol = 2.0 ** -8 * want.abs() + (2.0 ** -8 + 2 * ds[:, None] + 2.0 ** -18) * mag + 2.0 ** -16 * mag
        err = (o[0, :, t].cpu().to(F64) - want).abs()
        assert (err <= tol).all(), (float((err / mag).max()), float((err / tol).max()))


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("d,T,G", [(128, 6, 2), (128, 6, 4), (64, 12, 4), (128, 30, 3), (64, 60, 4)])
@pytest.mark.parametrize("start", [0, 300, 384])
def test_large_hidden_values_stay_hidden(fa, fmt, d, T, G, start):
    """A drafted row whose value scale (bf16: values) is far above the others' changes nothing
    for the tokens that do not see it, bit for bit."""
    c = ref.Cache(fa, 1, 400 + T, 1, d, 32, fmt, seed=63)
    g = torch.Generator().manual_seed(64)
    q = torch.randn(1, G, T, d, generator=g).to(torch.bfloat16).cuda()
    u = T // 2
    sees = torch.ones(T, T).tril().bool()
    sees[:, u] = torch.arange(T) % 3 == u % 3
    sees[u, u] = True
    bits = torch.zeros(1, T, -(-T // 32) * 32, dtype=torch.int64)
    bits[0, :, :T] = sees
    words = (bits.view(1, T, -1, 32) << torch.arange(32)).sum(-1)
    mask = torch.where(words >= 1 << 31, words - (1 << 32), words).int().cuda()
    st = torch.tensor([start], dtype=torch.int32)
    call = lambda: [x.clone() for x in fa.cache_forward(q, c.fa, st.cuda(), tree_mask=mask)]
    o0, l0 = call()
    p, i = c.where(0, start + u)
    blind = ~sees[:, u]
    for shift in (4, 20, 32, 40, 60):
        old = (c.v[p, 0, i].clone(), None if c.vs is None else c.vs[p, 0, i].clone())
        if fmt == "e4m3":
            c.vs[p, 0, i] *= 2.0 ** shift
        else:
            c.v[p, 0, i] *= 2.0 ** shift
        o1, l1 = call()
        assert torch.equal(l1[0][:, blind], l0[0][:, blind]), shift
        assert torch.equal(o1[0][:, blind], o0[0][:, blind]), shift
        ro, rl, to, tl = ref.attend(c, q, st, None, mask, d ** -0.5)
        assert ((o1.cpu().to(F64) - ro).abs() <= to).all()
        c.v[p, 0, i] = old[0]
        if fmt == "e4m3":
            c.vs[p, 0, i] = old[1]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T,G", [(1, 8), (1, 24), (1, 60), (1, 128), (2, 100)])
@pytest.mark.parametrize("shift", [5, 7, 16, 36])
def test_a_large_value_scale_of_a_weak_key(fa, d, T, G, shift):
    """A key of the first tile whose weight is next to nothing has a value scale 2^shift above the
    others: the keys of the other tiles keep their values.  A weight may be 2^-24 of the row's
    largest (weight times value scale) off, beside its rounding; a value 2^-10 of itself."""
    n = 700
    c = ref.Cache(fa, 1, n + T, 1, d, 64, "e4m3", seed=65)
    c.vs.fill_(1.0 / 64)
    c.ks.fill_(1.0 / 60)
    p0, i0 = c.where(0, 17)
    c.k[..., 3] = 0.0
    c.k[p0, 0, i0] = 0.0
    c.k[p0, 0, i0, 3] = -448.0
    c.vs[p0, 0, i0] *= 2.0 ** shift
    g = torch.Generator().manual_seed(66)
    q = torch.randn(1, G, T, d, generator=g)
    q[..., 3] = 10.0 * (d / 64) ** 0.5       # that key's score: -9.3, in 60ths of 448
    q = q.to(torch.bfloat16).cuda()
    if shift > 20:
        c.ks[p0, 0, i0] *= 6.0               # -56: 2^-81 of the others' weight
    o, lse = fa.cache_forward(q, c.fa, torch.tensor([n], dtype=torch.int32).cuda())
    raw = c.raw()
    k, _ = c.rows(raw, 0, 0, 0, n + T)
    v, sv = c.rows(raw, 1, 0, 0, n + T)
    k, v, sv = k[0], v[0], sv[0]
    for t in range(T):
        m = n + t + 1
        kk, vv, qq = k[:m], v[:m], q[0, :, t].cpu().to(F64)
        p = (qq @ kk.T * d ** -0.5).softmax(-1)
        want, mag = p @ vv, p @ vv.abs()
        ds = 2.0 ** -21 * (qq.abs() @ kk.abs().T).amax(-1)
        top = (p * sv[:m]).amax(-1)
        tol = (2.0 ** -8 * want.abs() + (2.0 ** -8 + 2.0 ** -10 + 2 * ds[:, None] + 2.0 ** -18) * mag
               + 2.0 ** -24 * top[:, None] * (vv.abs() / sv[:m, None]).sum(0))
        err = (o[0, :, t].cpu().to(F64) - want).abs()
        assert (err <= tol).all(), (float(err.max()), float((err / tol).max()))


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("G", [1, 12])
def test_scores_far_below_zero(fa, fmt, G):
    """Scores of -2e30 and lower are scores like any other: equal ones share the weight."""
    c = ref.Cache(fa, 1, 400, 1, 64, 32, fmt, seed=67)
    c.k.zero_()
    c.k[..., 0] = -448.0
    if fmt == "e4m3":
        c.ks.fill_(1.0)
        c.vs.fill_(0.01)
    q = torch.zeros(1, G, 1, 64, dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 2.0 ** 100
    n = 300
    for scale in (0.125, 2.0 ** 10):           # -7.1e31, -5.8e35
        o, lse = fa.cache_forward(q, c.fa, torch.tensor([n - 1], dtype=torch.int32).cuda(), scale=scale)
        v, _ = c.rows(c.raw(), 1, 0, 0, n)
        want, mag = v[0].mean(0), v[0].abs().mean(0)
        assert ((o[0, :, 0].cpu().to(F64) - want).abs() <= 2.0 ** -8 * want.abs() + (2.0 ** -8 + 2.0 ** -16) * mag).all()
        s = -448.0 * 2.0 ** 100 * scale
        assert ((lse.cpu().to(F64) - s).abs() <= 2.0 ** -21 * abs(s)).all()
