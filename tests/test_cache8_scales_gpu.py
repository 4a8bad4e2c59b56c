"""Attention over the paged 8-bit cache where a prefix's value scales lie far apart: blocks of zeros
(scale 2^-110), a saturated infinity (2^120), scales of any size, against the 64-bit form dimension by
dimension, so that a large value in one dimension excuses nothing in another.

Error of an output, up to 4 queries per key head.  A score is off by at most 2^-20 of
B = scale |q| |k| (test_operators_gpu), so a weight by 2^-19 B of itself; the two sums round by at most
2^-20 of their size; weights enter in 22 bits, below 2^-29 of the largest of their 16 keys to 2^-51
of it.  So |error| <= (2 * 2^-19 B + 2^-19) sum p |v| + 2^-50 sum |v| + half a step of the output.

More queries.  Weights enter at 22 bits (fp32) or 11 (bf16, each off by 2^-11 of itself at most), and
weight times value scale below 2^-20 of the query's largest to 2^-42 (2^-31) of that, times a byte
of at most 448: keys * 448 * 2^-42 (2^-31) * max(p s) more.
"""
import math

import pytest

from tests.test_operators_gpu import _gen, _settle, _values, sd  # noqa: F401

pytestmark = pytest.mark.gpu

LEAST = 2.0 ** -110                         # the scale of a block of zeros


def _cache(sd, k, v, page):  # noqa: F811
    """A cache of one row that holds k, v fp32 [keys][kv][dh], by appending."""
    import torch
    keys, kv, dh = k.shape
    n_pages = -(-keys // page)
    pages = torch.full((n_pages, 2, kv, page, dh), 0x7f, dtype=torch.uint8, device="cuda")
    scales = torch.ones(n_pages, 2, kv, device="cuda")
    table = torch.randperm(n_pages, generator=_gen(1), device="cuda").int()[None].contiguous()
    cache = sd.Cache8(pages, scales, table, torch.zeros(1, dtype=torch.int32, device="cuda"))
    cache.append(k[None].contiguous(), v[None].contiguous(), torch.zeros(1, dtype=torch.int32, device="cuda"))
    return cache


def _check(sd, cache, q, keys, scale):  # noqa: F811
    """q [n][heads][dh] at the prefix's end."""
    import torch
    n, heads, dh = q.shape
    share = heads // cache.kv_heads
    out = torch.full_like(q, 7.0)[None]
    cache.attend(q[None].contiguous(), torch.tensor([keys], dtype=torch.int32, device="cuda"), out, scale=scale)
    torch.cuda.synchronize()
    assert int(cache.status) == 0
    blocks = cache.table[0, : -(-keys // cache.page)].long()
    x = _values(cache.pages, cache.scales)[blocks].permute(1, 2, 0, 3, 4).flatten(2, 3)[:, :, :keys]
    x = x.repeat_interleave(share, 1)                                   # [2][heads][keys][dh]
    s = torch.einsum("nhd,hkd->hnk", q.double(), x[0]) * scale
    at = torch.arange(keys - n, keys, device="cuda")
    s = s.masked_fill(torch.arange(keys, device="cuda")[None] > at[:, None], -math.inf)
    p = torch.softmax(s, -1)
    want = torch.einsum("hnk,hkd->nhd", p, x[1])
    size = torch.einsum("hnk,hkd->nhd", p, x[1].abs())
    big = abs(scale) * q.double().norm(dim=-1).max() * x[0].norm(dim=-1).max()
    tol = (2.0 ** -18 * big + 2.0 ** -19) * size + 2.0 ** -50 * x[1].abs().sum(1)[None] + 2.0 ** -148
    if n * share > 4:
        vs = cache.scales[blocks, 1].double().repeat_interleave(cache.page, 0)[:keys].T.repeat_interleave(share, 0)
        top = (p * vs[:, None]).amax(-1).T[..., None]                   # [n][heads][1]
        one = q.dtype == torch.bfloat16
        tol = tol + keys * 448 * 2.0 ** (-31 if one else -42) * top + (2.0 ** -11 * size if one else 0.0)
    err = (out[0].double() - want).abs()
    half = 2.0 ** -8 if q.dtype == torch.bfloat16 else 2.0 ** -24
    ok = err <= tol + half * want.abs()                                 # (NaN is not)
    assert bool(ok.all()), (float(err.nan_to_num(math.inf).max()), (~ok).nonzero()[:4].tolist(),
                            out[0][~ok][:4].tolist(), want[~ok][:4].tolist())
    return want


FORMS = [(1, 1, "fp32"), (4, 1, "bf16"), (1, 8, "fp32"), (1, 8, "bf16"), (3, 16, "bf16"), (2, 16, "fp32")]


def _type(t):
    import torch
    return torch.float32 if t == "fp32" else torch.bfloat16


@pytest.mark.parametrize("n,share,t", FORMS)
@pytest.mark.parametrize("keys,bits", [(65536, 17.0), (2049, 12.0), (300, 30.0)])
def test_blocks_of_zeros_weigh_as_much_as_others(sd, n, share, t, keys, bits):  # noqa: F811
    """One key `bits` binary places above all others, whose values are zero: its value times its
    weight, no more."""
    import torch
    k, v = torch.zeros(2, keys, 1, 64, device="cuda")
    k[1, 0, 0], v[1, 0] = 1.0, 384.0
    q = torch.zeros(n, share, 64, device="cuda", dtype=_type(t))
    q[..., 0] = 1.0
    cache = _cache(sd, k, v, 16)
    assert float(cache.scales[:, 1].min()) == LEAST
    want = _check(sd, cache, q, keys, bits * math.log(2.0))
    there = 2.0 ** bits / (2.0 ** bits + keys - n)              # (of the first query)
    assert abs(float(want[0, 0, 0]) / 384.0 - there) < 1e-9


@pytest.mark.parametrize("n,share,t", FORMS)
@pytest.mark.parametrize("dh,page,keys", [(64, 16, 4096), (128, 64, 5000)])
def test_padded_blocks_beside_ordinary_values(sd, n, share, t, dh, page, keys):  # noqa: F811
    """Ordinary values in the first half, zeros in most of the other; a few keys peak."""
    import torch
    k = torch.randn(keys, 2, dh, generator=_gen(1), device="cuda")
    v = torch.randn(keys, 2, dh, generator=_gen(2), device="cuda")
    v[keys // 2:keys - page - 3] = 0.0
    q = torch.randn(n, 2 * share, dh, generator=_gen(3), device="cuda").to(_type(t))
    k[5] = 2.0 * q[0, ::share].float()          # about 12 sqrt(dh) above the rest
    cache = _cache(sd, k, v, page)
    assert float(cache.scales[:, 1].min()) == LEAST
    _check(sd, cache, q, keys, dh ** -0.5)
    _check(sd, cache, torch.zeros_like(q), keys, dh ** -0.5)


@pytest.mark.parametrize("n,share,t", FORMS)
def test_values_that_are_all_zero(sd, n, share, t):  # noqa: F811
    import torch
    k = torch.randn(9000, 1, 64, generator=_gen(1), device="cuda")
    q = 3 * torch.randn(n, share, 64, generator=_gen(3), device="cuda").to(_type(t))
    cache = _cache(sd, k, torch.zeros_like(k), 32)
    out = torch.full_like(q, 7.0)[None]
    cache.attend(q[None].contiguous(), torch.tensor([9000], dtype=torch.int32, device="cuda"), out)
    torch.cuda.synchronize()
    assert not bool(out.any())                  # (NaN counts)


@pytest.mark.parametrize("n,share,t", FORMS)
@pytest.mark.parametrize("lo,hi", [(-110, 90), (-149, -100), (80, 112), (-20, 0)])
@pytest.mark.parametrize("page", [16, 128])
def test_scales_of_any_size(sd, n, share, t, lo, hi, page):  # noqa: F811
    import torch
    keys = 3000
    k = torch.randn(keys, 2, 64, generator=_gen(1), device="cuda")
    v = torch.randn(keys, 2, 64, generator=_gen(2), device="cuda")
    cache = _cache(sd, k, v, page)
    e = torch.randint(lo, hi, cache.scales[:, 1].shape, generator=_gen(4), device="cuda")
    cache.scales[:, 1] = torch.ldexp(torch.full(e.shape, 1.375, dtype=torch.float64, device="cuda"), e).float()
    cache.scales.clamp_(min=2.0 ** -149)
    q = torch.randn(n, 2 * share, 64, generator=_gen(3), device="cuda").to(_type(t))
    _check(sd, cache, q, keys, 0.25)


@pytest.mark.parametrize("n,share,t", [(1, 1, "fp32"), (4, 1, "bf16"), (2, 2, "fp32")])
@pytest.mark.parametrize("at", [0, 700, 1999])
def test_an_infinite_value_leaves_the_other_dimensions(sd, n, share, t, at):  # noqa: F811
    """Appended, it is 448 scales of 2^120; the other dimensions of the output keep their mean."""
    import torch
    k = torch.randn(2000, 1, 64, generator=_gen(1), device="cuda")
    v = torch.randn(2000, 1, 64, generator=_gen(2), device="cuda")
    v[at, 0, 9] = math.inf
    cache = _cache(sd, k, v, 32)
    assert float(cache.scales[:, 1].max()) == 2.0 ** 120
    q = torch.randn(n, share, 64, generator=_gen(3), device="cuda").to(_type(t))
    want = _check(sd, cache, q, 2000, 0.125)
    assert bool((want[..., 9].abs() > 2.0 ** 100)[-1].all()) and float(want[..., :9].abs().max()) < 1.0
