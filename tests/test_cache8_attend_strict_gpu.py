"""Attention over the paged 8-bit cache with a comparison that a NaN cannot pass: the cases of
test_operators_gpu again, blocks as long as prompt pieces, and wide tables of short rows.

Tolerances are those of test_operators_gpu: the 64-bit form's bound of an fp32 computation, for bf16
types and more than 4 queries to a key head 2^-11 of the largest value more, and half a step of the
output's type."""
import math

import pytest

from tests.test_operators_gpu import (ATTEND, ATTEND_BLOCKS, _attend64, _gen, _new_cache, _rope, _settle,  # noqa: F401
                                      _values, sd)

pytestmark = pytest.mark.gpu


def _check(cache, q, out, lens, scale, rope):
    import torch
    want, tol = _attend64(cache, q, lens, scale, rope)
    t = tol[:, None, None, None]
    if q.dtype == torch.bfloat16 and q.shape[1] * q.shape[2] // cache.kv_heads > 4:
        t = t + 2.0 ** -11 * float(_values(cache.pages, cache.scales).abs().max())
    half = 2.0 ** -8 if out.dtype == torch.bfloat16 else 2.0 ** -24
    ok = (out.double() - want).abs() <= t + half * want.abs()
    assert bool(torch.isfinite(want).all()) and bool(ok.all()), (~ok).nonzero()[:4].tolist()


CASES = ATTEND + [c + (False, 0) for c in ATTEND_BLOCKS] + [
    # blocks as long as prompt pieces: lens, n, heads, kv, dh, page, type, rot, interleaved, origin
    ([300, 64, 40], 64, 4, 2, 64, 32, "bf16", 64, False, 0),        # of row 2's queries 24 see nothing
    ([300, 64, 40], 64, 4, 2, 64, 32, "fp32", 0, False, 0),
    ([2500], 200, 3, 1, 128, 64, "bf16", 128, False, 1),
    ([2500], 200, 3, 1, 128, 64, "fp32", 128, True, 1),
    ([700, 701], 577, 2, 2, 64, 16, "bf16", 0, False, 0),
    ([5], 33, 2, 1, 128, 128, "fp32", 0, False, 0),
]


@pytest.mark.parametrize("case", CASES, ids=[str(i) for i in range(len(CASES))])
def test_attend(sd, case):  # noqa: F811
    import torch
    lens, n, heads, kv, dh, page, t, rot, inter, origin = case
    rows = len(lens)
    cache = _new_cache(sd, rows, max(max(lens), 1), page, kv, dh, seed=sum(lens) + 3 * n)
    dt = torch.float32 if t == "fp32" else torch.bfloat16
    q = (2 * torch.randn(rows, n, heads + 1, dh, generator=_gen(7), device="cuda")).to(dt)[:, :, :heads]
    out = torch.full((rows, n, heads, dh), math.nan, device="cuda", dtype=dt)
    rope = _rope(sd, rot, max(max(lens) + origin, 0) + 1, inter, origin)
    cache.attend(q, torch.tensor(lens, dtype=torch.int32, device="cuda"), out, rope=rope)
    torch.cuda.synchronize()
    assert int(cache.status) == 0
    _check(cache, q, out, lens, dh ** -0.5, rope)
    for b, L in enumerate(lens):
        assert not out[b, : max(0, n - L)].any()


@pytest.mark.parametrize("dh,t,n,share", [(128, "bf16", 1, 8), (64, "fp32", 2, 4), (128, "bf16", 1, 1), (128, "fp32", 1, 4),
                                          (64, "bf16", 1, 2)])
def test_short_rows_of_a_wide_table(sd, dh, t, n, share):  # noqa: F811
    """Tables sized for 32768 and 131072 positions, rows of a few hundred (and one that fills half): the same
    bits as in a table that fits them, and right."""
    import torch
    dt = torch.float32 if t == "fp32" else torch.bfloat16
    lens = [500, 1, 17, 499, 333, 16, 130, 257, 450]
    tight = _new_cache(sd, 9, 512, 64, 4, dh, seed=4)
    q = torch.randn(9, n, 4 * share, dh, generator=_gen(6), device="cuda").to(dt)
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
    want = torch.full_like(q, math.nan)
    tight.attend(q, ln, want)
    torch.cuda.synchronize()
    _check(tight, q, want, lens, dh ** -0.5, None)
    for cap in (32768, 131072):
        table = torch.full((9, cap // 64), 2 ** 30, dtype=torch.int32, device="cuda")
        table[:, :8] = tight.table
        wide = sd.Cache8(tight.pages, tight.scales, table, tight.status)
        out = torch.full_like(q, math.nan)
        wide.attend(q, ln, out)
        torch.cuda.synchronize()
        assert int(wide.status) == 0 and torch.equal(out, want), cap


@pytest.mark.parametrize("t", ["bf16", "fp32"])
def test_a_batch_of_clusters_of_16(sd, t):  # noqa: F811
    """Unequal long rows with clusters as large as they get, many queries and few."""
    import torch
    dt = torch.float32 if t == "fp32" else torch.bfloat16
    lens = [33000, 100, 20000, 32768, 4097]
    cache = _new_cache(sd, 5, 33000, 128, 2, 64, seed=5)
    for share in (8, 1):
        q = torch.randn(5, 1, 2 * share, 64, generator=_gen(share), device="cuda").to(dt)
        out = torch.full_like(q, math.nan)
        cache.attend(q, torch.tensor(lens, dtype=torch.int32, device="cuda"), out)
        torch.cuda.synchronize()
        assert int(cache.status) == 0
        _check(cache, q, out, lens, 0.125, None)
