"""A Rope and a KVCache keep pointers to their tensors: their attributes cannot be exchanged for
others, which the checks would see and the kernels would not.  Needs no GPU."""
import pytest
import torch


@pytest.fixture(scope="module")
def fa():
    import __graft_entry__
    __graft_entry__.build()
    import exact_attention_88_gb300 as m
    return m


def _cache(fa, e4m3):
    k = torch.zeros(4, 2, 16, 64, dtype=torch.float8_e4m3fn if e4m3 else torch.bfloat16)
    s = (torch.ones(4, 2, 16), torch.ones(4, 2, 16)) if e4m3 else (None, None)
    return fa.KVCache(k, k.clone(), *s, torch.zeros(2, 2, dtype=torch.int32))


@pytest.mark.parametrize("e4m3", [False, True])
def test_cache_attributes_are_fixed(fa, e4m3):
    c = _cache(fa, e4m3)
    for name in ("k", "v", "k_scale", "v_scale", "block_table", "struct", "heads", "d", "format",
                 "sequences", "capacity", "device"):
        old = getattr(c, name)
        with pytest.raises(AttributeError):
            setattr(c, name, old)
        with pytest.raises(AttributeError):
            delattr(c, name)
        assert getattr(c, name) is old
    c.block_table.fill_(3)                     # contents may change
    assert c.struct.block_table == c.block_table.data_ptr()


def test_rope_attributes_are_fixed(fa):
    r = fa.Rope(torch.ones(16, dtype=torch.float64))
    for name in ("freq", "dim", "interleaved", "factor"):
        with pytest.raises(AttributeError):
            setattr(r, name, getattr(r, name))
        with pytest.raises(AttributeError):
            delattr(r, name)
    assert (r.dim, r.interleaved, r.factor) == (32, False, 1.0)


def test_workspace_of_paired_ctas(fa):
    # 129 to 256 rows: two CTAs share a run, so there are as many partial rows as at 128
    f = fa.fa_cache_fwd_workspace_size
    for d in (64, 128):
        assert f(1, 8, 1, 1024, d) == f(3, 2, 1, 70, d) == f(1, 8, 1, 16, d) == 2 * f(1, 8, 1, 8, d)


def test_bands_without_a_ramp_are_refused(fa):
    # (equal ends would make 0 / 0 of a pair that turns just as often)
    for slow, fast in ((8.0, 8.0), (9.0, 8.0), (float("nan"), 8.0)):
        with pytest.raises(ValueError):
            fa.rope_frequencies(64, scaling="bands", factor=4.0, slow_turns=slow, fast_turns=fast, device="cpu")
