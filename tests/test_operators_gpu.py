"""The paged 8-bit cache (append, attend) and beam search's selection and reordering against
plain 64-bit forms, at the sizes, masks and layouts where they can go wrong.

Half steps: e4m3 2^-4 of a normal value and 2^-10 of a scale below 2^-6 scales; bf16 2^-8;
fp32 2^-24.
"""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

E4M3 = "float8_e4m3fn"


@pytest.fixture(scope="module")
def sd():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from tests.conftest import build_library
    build_library()
    import stateful_decoding_b200 as sd
    return sd


@pytest.fixture(autouse=True)
def _settle(request):
    yield
    import torch
    if torch.cuda.is_available():
        torch.cuda.synchronize()


def _gen(seed):
    import torch
    return torch.Generator(device="cuda").manual_seed(seed)


def _values(pages, scales):
    import torch
    return pages.view(torch.float8_e4m3fn).double() * scales.double()[..., None, None]


def _new_cache(sd, rows, cap, page, kv, dh, seed=0, spare=2, fill=True):
    """A cache of rows x cap tokens, pages shuffled, bytes random finite, scales powers of two."""
    import torch
    g = _gen(seed)
    row_pages = -(-cap // page)
    n_pages = rows * row_pages + spare
    x = torch.randn(n_pages, 2, kv, page, dh, generator=g, device="cuda") * 64
    pages = x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    if not fill:
        pages.fill_(0x7f)                               # NaN everywhere
    scales = torch.exp2(torch.randint(-8, -4, (n_pages, 2, kv), generator=g, device="cuda").float())
    table = torch.randperm(n_pages, generator=g, device="cuda")[: rows * row_pages].int()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    return sd.Cache8(pages, scales, table.view(rows, row_pages).contiguous(), status)


def _rope(sd, rot, positions, interleaved=False, origin=0):
    import torch
    if not rot:
        return None
    at = torch.arange(positions, dtype=torch.float64, device="cuda")[:, None]
    ang = at * 10000.0 ** (-2 * torch.arange(rot // 2, dtype=torch.float64, device="cuda") / rot)
    return sd.Rope(ang.cos().float(), ang.sin().float(), interleaved, origin)


def _turn(x, rope, at):
    """fp64 rotation of x [..., heads, dh] at token indexes `at`; and a bound on an fp32
    rotation's error."""
    import torch
    x = x.double()
    if rope is None:
        return x, torch.zeros_like(x)
    cos, sin = rope.buffers
    rot = 2 * cos.shape[1]
    c, s = (t.double()[at + rope.struct.origin][..., None, :] for t in (cos, sin))
    y, err = x.clone(), torch.zeros_like(x)
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if rope.struct.interleaved else \
        (slice(0, rot // 2), slice(rot // 2, rot))
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    # two products and a sum, each off by 2^-24 of its size
    err[..., a] = err[..., b] = 3 * 2.0 ** -24 * (x[..., a].abs() + x[..., b].abs())
    return y, err


# ------------------------------------------------------------------------------ append
def _check_append(cache, before, bscales, k, v, start, counts, rope):
    """Every byte of the cache after an append of k, v [rows][n][kv][dh]."""
    import torch
    page, cap = cache.page, cache.row_pages * cache.page
    was, now = _values(before, bscales), _values(cache.pages, cache.scales)
    touched = torch.zeros_like(now, dtype=torch.bool)
    seen = set()
    for b in range(cache.rows):
        s, c = int(start[b]), int(counts[b])
        if not c:
            continue
        at = torch.arange(s, s + c, device="cuda")
        kk, ke = _turn(k[b, :c], rope, at)
        vv = v[b, :c].double()
        x = torch.stack((kk, vv), 1).permute(1, 2, 0, 3)            # [2][kv][c][dh]
        err = torch.stack((ke, torch.zeros_like(vv)), 1).permute(1, 2, 0, 3)
        for block in range(s // page, (s + c - 1) // page + 1):
            p = int(cache.table[b, block])
            assert p not in seen
            seen.add(p)
            lo, hi = max(s, block * page), min(s + c, (block + 1) * page)
            a, z = lo - block * page, hi - block * page
            new, e = x[:, :, lo - s:hi - s], err[:, :, lo - s:hi - s]
            scale = cache.scales[p].double()
            # the smallest power of two that holds the largest magnitude (or the old, larger one)
            need = torch.exp2((new.abs().amax((-1, -2)) / 448).log2().sub(1e-9).ceil().clamp(-110, 120))
            want = torch.maximum(need, bscales[p].double()) if a else need
            near = (new.abs().amax((-1, -2)) / 448 / need).log2()
            sure = (near < -1e-6) & (near > -1 + 1e-6)             # away from a power's border
            if rope is None:
                sure = torch.ones_like(sure)
            assert torch.equal(scale[sure], want[sure]), (b, block)
            got = now[p, :, :, a:z]
            tol = new.abs() * 2.0 ** -4 + scale[..., None, None] * 2.0 ** -10 + e * 1.0625
            assert bool(((got - new).abs() <= tol).all()), (b, block, float((got - new).abs().max()))
            if a:
                old = was[p, :, :, :a]
                grown = (scale > bscales[p].double())[..., None, None]
                tol = torch.where(grown, scale[..., None, None] * 2.0 ** -10, torch.zeros_like(old))
                assert bool(((now[p, :, :, :a] - old).abs() <= tol).all())
            touched[p, :, :, :z] = True
    assert torch.equal(cache.pages[~touched], before[~touched])   # nothing else was written
    rest = [p for p in range(len(before)) if p not in seen]
    assert torch.equal(cache.scales[rest], bscales[rest])
    assert int(cache.status) == 0


APPEND = [
    # rows, n, kv, dh, page, type, rot, interleaved, origin, starts, counts
    (3, 1, 2, 64, 16, "bf16", 64, False, 0, [0, 15, 16], None),
    (3, 1, 1, 128, 64, "fp32", 64, True, 1, [63, 64, 127], None),
    (4, 5, 3, 64, 16, "fp32", 0, False, 0, [0, 13, 14, 30], [5, 0, 5, 1]),
    (2, 2, 1, 128, 16, "bf16", 128, False, 0, [15, 31], None),
    (2, 16, 2, 128, 16, "bf16", 64, False, 3, [0, 7], None),
    (2, 33, 1, 64, 32, "fp32", 8, True, 0, [31, 1], [33, 2]),
    (2, 130, 2, 128, 128, "fp32", 128, True, 0, [0, 127], [130, 129]),
    (1, 300, 2, 128, 64, "bf16", 128, False, 0, [1], None),
    (2, 200, 1, 64, 128, "bf16", 64, False, 0, [3, 0], [200, 77]),
]


@pytest.mark.parametrize("case", APPEND, ids=[str(i) for i in range(len(APPEND))])
def test_append(sd, case):
    import torch
    rows, n, kv, dh, page, t, rot, inter, origin, starts, counts = case
    cache = _new_cache(sd, rows, max(starts) + n, page, kv, dh, seed=len(starts) + n)
    dt = torch.float32 if t == "fp32" else torch.bfloat16
    g = _gen(n)
    fused = torch.randn(rows, n, 3, kv, dh, generator=g, device="cuda").to(dt)
    fused[:, :, 1] *= torch.rand(rows, n, 1, 1, generator=g, device="cuda").to(dt) * 8
    k, v = fused[:, :, 1], fused[:, :, 2]                # strided, as a fused projection leaves them
    rope = _rope(sd, rot, max(starts) + n + origin, inter, origin)
    before, bscales = cache.pages.clone(), cache.scales.clone()
    start = torch.tensor(starts, dtype=torch.int32, device="cuda")
    cnt = None if counts is None else torch.tensor(counts, dtype=torch.int32, device="cuda")
    cache.append(k, v, start, counts=cnt, rope=rope)
    torch.cuda.synchronize()
    _check_append(cache, before, bscales, k, v, starts, counts or [n] * rows, rope)


def test_append_token_by_token_equals_at_once(sd):
    """Powers of two: a page filled in steps differs from one filled at once only where a byte
    falls into the subnormal range of a scale that grew (half a step: 2^-10 scales, twice)."""
    import torch
    g = _gen(5)
    k = torch.randn(2, 70, 2, 64, generator=g, device="cuda")
    k *= torch.linspace(0.01, 20, 70, device="cuda")[:, None, None]      # scales keep growing
    v = k.flip(1).contiguous()                                           # and never grow
    a, b = (_new_cache(sd, 2, 80, 32, 2, 64, seed=3) for _ in range(2))
    zero = torch.zeros(2, dtype=torch.int32, device="cuda")
    a.append(k, v, zero)
    for i in range(0, 70, 7):
        b.append(k[:, i:i + 7], v[:, i:i + 7], zero + i)
    torch.cuda.synchronize()
    used = a.table[:, :3].flatten().long()
    assert torch.equal(a.scales[used], b.scales[used])
    for j in range(3):
        z = min(32, 70 - 32 * j)
        p = a.table[:, j].long()
        x, y = (_values(c.pages, c.scales)[p][:, :, :, :z] for c in (a, b))
        assert bool(((x - y).abs() <= 2 * 2.0 ** -10 * a.scales[p].double()[..., None, None]).all())
        if j == 0:      # values fell: their scale was set by the first token, nothing was rounded twice
            assert torch.equal(a.pages[p][:, 1, :, :z], b.pages[p][:, 1, :, :z])


def test_append_special_values(sd):
    import torch
    cache = _new_cache(sd, 1, 16, 16, 1, 64)
    k = torch.zeros(1, 3, 1, 64, device="cuda")
    v = k.clone()
    k[0, 0, 0, :6] = torch.tensor([float("nan"), 448.0, -448.0, 1e-30, 432.0, 17.0], device="cuda")
    v[0, 1, 0, 0] = float("inf")
    v[0, 2, 0, 1] = -float("inf")
    cache.append(k, v, torch.zeros(1, dtype=torch.int32, device="cuda"))
    p = int(cache.table[0, 0])
    x = cache.pages[p].view(torch.float8_e4m3fn).float()
    assert float(cache.scales[p, 0, 0]) == 1.0               # 448 fits exactly
    assert torch.isnan(x[0, 0, 0, 0]) and not torch.isnan(x[0, 0, 0, 1:]).any()
    assert x[0, 0, 0, 1:6].tolist() == [448.0, -448.0, 0.0, 448.0, 16.0]    # ties to even
    # an infinity counts as the largest finite value and comes back as that, saturated
    assert float(cache.scales[p, 1, 0]) == 2.0 ** 120
    assert float(x[1, 0, 1, 0]) == 448.0 and float(x[1, 0, 2, 1]) == -448.0
    # all zeros: the smallest scale
    cache.append(torch.zeros_like(k), torch.zeros_like(v), torch.zeros(1, dtype=torch.int32, device="cuda"))
    assert float(cache.scales[p, 0, 0]) == 2.0 ** -110 and not cache.pages[p, :, :, :3].any()


def test_append_bad_lengths_and_pages_are_stepped_around(sd):
    import torch
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    for starts, counts, spoil, code in (
            ([30, 0], None, None, sd.RLT_E_CAPACITY),         # row 0 passes its two pages
            ([-1, 0], None, None, sd.RLT_E_CAPACITY),
            ([32, 0], None, None, sd.RLT_E_CAPACITY),
            ([2 ** 31 - 1, 0], None, None, sd.RLT_E_CAPACITY),
            ([0, 0], [5, 4], None, sd.RLT_E_CAPACITY),        # more than n
            ([0, 0], [-2 ** 31, 4], None, sd.RLT_E_CAPACITY),
            ([14, 0], None, (0, 1, 99), sd.RLT_E_ARG),        # its second page does not exist
            ([14, 0], None, (0, 1, -1), sd.RLT_E_ARG)):
        cache = _new_cache(sd, 2, 32, 16, 1, 64)
        if spoil:
            cache.table[spoil[0], spoil[1]] = spoil[2]
        k = torch.randn(2, 4, 1, 64, generator=_gen(1), device="cuda")
        before, bscales = cache.pages.clone(), cache.scales.clone()
        cache.append(k, k, i32(*starts), counts=None if counts is None else i32(*counts))
        torch.cuda.synchronize()
        assert int(cache.status) == code, (starts, counts, spoil)
        # row 1 is written, of row 0 only what fits a sane row
        p1 = int(cache.table[1, 0])
        own = torch.zeros_like(cache.pages, dtype=torch.bool)
        own[p1, :, :, :4] = True
        assert bool((_values(cache.pages, cache.scales)[p1, 0, 0, :4] - k[1, :, 0].double()).abs().max() < 0.3)
        if starts[0] in (14, 30):
            p0 = int(cache.table[0, starts[0] // 16])
            own[p0, :, :, :16] = True
            slot = starts[0] % 16
            assert bool((_values(cache.pages, cache.scales)[p0, 0, 0, slot:] - k[0, :2, 0].double()).abs().max() < 0.3)
        assert torch.equal(cache.pages[~own], before[~own]), (starts, counts, spoil)


def test_append_rotation_table_too_short(sd):
    import torch
    cache = _new_cache(sd, 1, 16, 16, 1, 64)
    before = cache.pages.clone()
    k = torch.randn(1, 8, 1, 64, generator=_gen(1), device="cuda")
    cache.append(k, k, torch.zeros(1, dtype=torch.int32, device="cuda"), rope=_rope(sd, 64, 5))
    torch.cuda.synchronize()
    p = int(cache.table[0, 0])
    assert int(cache.status) == sd.RLT_E_CAPACITY
    assert torch.equal(cache.pages[p, :, :, 5:], before[p, :, :, 5:])
    assert bool((_values(cache.pages, cache.scales)[p, 1, 0, :5] - k[0, :5, 0].double()).abs().max() < 0.3)


# ------------------------------------------------------------------------------ attend
def _attend64(cache, q, lens, scale, rope):
    """fp64 attention; and the bound of an fp32 computation's error, per row.

    Scores: q and k enter in 22 and 4 bits, products are summed in fp32 over dh <= 128 terms, so a
    score is off by at most 2^-20 of scale |q| |k| (Cauchy-Schwarz; rotation and rounding of q,
    2^-22, included).  A weight then moves by twice that, and the sums of weights and of weighted
    values round by at most 2^-20 of their size."""
    import torch
    rows, n, heads, dh = q.shape
    share = heads // cache.kv_heads
    out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    tol = torch.zeros(rows, dtype=torch.float64, device="cuda")
    allv = _values(cache.pages, cache.scales)
    for b in range(rows):
        L = int(lens[b])
        if L == 0:
            continue
        blocks = cache.table[b, : -(-L // cache.page)].long()
        x = allv[blocks].permute(1, 2, 0, 3, 4).flatten(2, 3)[:, :, :L].repeat_interleave(share, 1)
        at = torch.arange(L - n, L, device="cuda")
        qq, _ = _turn(q[b], rope, at.clamp_min(0)) if rope is not None else (q[b].double(), None)
        s = torch.einsum("nhd,hkd->hnk", qq, x[0]) * scale
        hide = torch.arange(L, device="cuda")[None] > at[:, None]
        s = s.masked_fill(hide[None], -math.inf)
        p = torch.nan_to_num(torch.softmax(s, -1), nan=0.0)          # a query that sees nothing
        out[b] = torch.einsum("hnk,hkd->nhd", p, x[1])
        big = abs(scale) * qq.norm(dim=-1).max() * x[0].norm(dim=-1).max()
        tol[b] = (2 * 2.0 ** -20 * big + 2.0 ** -20) * x[1].abs().max()
    return out, tol


def _check_attend(cache, q, out, lens, scale, rope, rounded_p):
    import torch
    want, tol = _attend64(cache, q, lens, scale, rope)
    vmax = float(_values(cache.pages, cache.scales).nan_to_num().abs().max())
    t = tol[:, None, None, None] + (2.0 ** -11 * vmax if rounded_p else 0.0)
    half = 2.0 ** -8 if out.dtype == torch.bfloat16 else 2.0 ** -24
    bad = (out.double() - want).abs() > t + half * want.abs()
    assert not bool(bad.any()), (float((out.double() - want).abs().max()), bad.nonzero()[:4].tolist())


ATTEND = [
    # lens, n, heads, kv, dh, page, type, rot, interleaved, origin
    ([1, 15, 16, 17, 0], 1, 2, 2, 64, 16, "fp32", 0, False, 0),
    ([1, 15, 16, 17, 0], 1, 2, 2, 128, 16, "bf16", 128, False, 0),
    ([63, 64, 65, 300], 1, 4, 2, 64, 32, "bf16", 64, True, 1),
    ([63, 64, 65, 300], 1, 3, 1, 128, 64, "fp32", 64, False, 1),
    ([1023, 1024, 1025, 2], 1, 2, 2, 64, 128, "fp32", 64, False, 0),
    ([5000, 4097], 1, 8, 1, 128, 64, "bf16", 0, False, 0),
    ([40001, 9], 1, 2, 1, 64, 16, "fp32", 64, False, 0),
    ([3, 4, 20, 0, 1], 4, 2, 2, 64, 16, "fp32", 64, False, 0),     # some queries see nothing
    ([3, 4, 20, 0, 1], 4, 4, 2, 128, 32, "bf16", 0, False, 0),
    ([2000, 77], 5, 6, 2, 128, 32, "bf16", 128, True, 2),           # 15 queries: 16 rows
    ([2000, 77], 5, 6, 2, 64, 32, "fp32", 64, True, 2),             # two tiles of 8
    ([3333, 17, 16], 16, 8, 1, 64, 64, "bf16", 64, False, 0),       # 128 queries: 8 tiles
    ([1100, 16], 16, 2, 2, 128, 128, "bf16", 32, False, 0),
]


@pytest.mark.parametrize("case", ATTEND, ids=[str(i) for i in range(len(ATTEND))])
def test_attend(sd, case):
    import torch
    lens, n, heads, kv, dh, page, t, rot, inter, origin = case
    rows = len(lens)
    cache = _new_cache(sd, rows, max(max(lens), 1), page, kv, dh, seed=sum(lens) + n)
    dt = torch.float32 if t == "fp32" else torch.bfloat16
    q = (2 * torch.randn(rows, n, heads + 1, dh, generator=_gen(7), device="cuda")).to(dt)[:, :, :heads]
    room = torch.full((rows, n, heads + 2, dh), 5.0, device="cuda", dtype=dt)
    out = room[:, :, :heads]
    rope = _rope(sd, rot, max(lens) + origin + 1, inter, origin)
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
    scale = 1.0 / math.sqrt(dh)
    cache.attend(q, ln, out, rope=rope)
    torch.cuda.synchronize()
    assert int(cache.status) == 0
    assert bool((room[:, :, heads:] == 5.0).all())
    # bf16 types and more than 4 queries to a key head: the weights w_j enter the product as fp16,
    # each off by 2^-11 of itself at most, so sum w_j v_j / sum w_j moves by at most 2^-11 max |v|
    _check_attend(cache, q, out, lens, scale, rope, t == "bf16" and n * heads // kv > 4)
    for b, L in enumerate(lens):
        for i in range(n):
            if L - n + i + 1 <= 0:
                assert not out[b, i].any()


ATTEND_BLOCKS = [
    # many queries to a key head over many tiles and CTAs: lens, n, heads, kv, dh, page, type, rot
    ([1000, 130], 4, 16, 2, 64, 32, "fp32", 0),         # 32 queries of two parts
    ([1000, 130], 4, 16, 2, 64, 32, "bf16", 64),
    ([2500, 3], 8, 16, 2, 64, 16, "bf16", 0),           # 64 queries
    ([5000, 1], 2, 8, 1, 128, 64, "fp32", 128),
    ([4096, 2048, 2049], 3, 8, 2, 128, 128, "fp32", 0),
    ([9000, 513, 128, 127, 129], 2, 32, 1, 128, 16, "bf16", 0),
    ([33000, 70], 1, 8, 1, 64, 128, "fp32", 64),        # 16 CTAs
    ([12001], 16, 4, 1, 64, 64, "fp32", 0),             # 64 queries of two parts: two tiles
    ([3000, 17], 16, 16, 2, 128, 64, "bf16", 128),      # 128 queries: two tiles
]


@pytest.mark.parametrize("case", ATTEND_BLOCKS, ids=[str(i) for i in range(len(ATTEND_BLOCKS))])
def test_attend_blocks(sd, case):
    import torch
    lens, n, heads, kv, dh, page, t, rot = case
    rope = _rope(sd, rot, max(lens) + 4)
    cache = _new_cache(sd, len(lens), max(lens), page, kv, dh, seed=len(lens) + heads)
    q = 2 * torch.randn(len(lens), n, heads, dh, generator=_gen(9), device="cuda")
    q = q.float() if t == "fp32" else q.bfloat16()
    out, again = torch.full_like(q, 7.0), torch.full_like(q, 7.0)
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
    cache.attend(q, ln, out, rope=rope)
    cache.attend(q, ln, again, rope=rope)
    torch.cuda.synchronize()
    assert int(cache.status) == 0
    _check_attend(cache, q, out, lens, dh ** -0.5, rope, t == "bf16")
    assert torch.equal(out, again)


@pytest.mark.parametrize("t", ["fp32", "bf16"])
def test_attend_blocks_captured_and_on_two_streams(sd, t):
    """Many queries to a key head: captured once and replayed with new lengths and queries, and
    two calls at once."""
    import torch
    cache = _new_cache(sd, 3, 3000, 32, 2, 64, seed=8)
    q = torch.randn(3, 5, 6, 64, generator=_gen(4), device="cuda")
    q = q if t == "fp32" else q.bfloat16()
    out, other, want = (torch.zeros_like(q) for _ in range(3))
    lens = torch.tensor([3000, 5, 1200], dtype=torch.int32, device="cuda")
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    cache.attend(q, lens, out, stream=one)
    cache.attend(q, lens, other, stream=two)
    torch.cuda.synchronize()
    cache.attend(q, lens, want)
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(other, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=one):
        cache.attend(q, lens, out, stream=torch.cuda.current_stream())
    for seed, new in ((1, [7, 2999, 0]), (2, [2048, 2049, 64])):
        lens.copy_(torch.tensor(new, dtype=torch.int32))
        q.normal_(generator=_gen(seed))
        graph.replay()
        torch.cuda.synchronize()
        _check_attend(cache, q, out, new, 64 ** -0.5, None, t == "bf16")
    assert int(cache.status) == 0


@pytest.mark.parametrize("dh,t,n,share", [(64, "fp32", 1, 1), (128, "bf16", 1, 2), (64, "bf16", 4, 3),
                                                (128, "fp32", 3, 3), (64, "bf16", 9, 2)])
def test_attend_rows_do_not_depend_on_batch_capacity_or_run(sd, dh, t, n, share):
    """The same row alone, in a batch, in a table of another capacity, and twice: the same bits."""
    import torch
    lens = [700, 2500, 33, 1024]
    dt = torch.float32 if t == "fp32" else torch.bfloat16
    cache = _new_cache(sd, 4, 2600, 32, 2, dh, seed=1)
    q = torch.randn(4, n, 2 * share, dh, generator=_gen(3), device="cuda").to(dt)
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
    out, again = torch.empty_like(q), torch.empty_like(q)
    cache.attend(q, ln, out)
    cache.attend(q, ln, again)
    assert torch.equal(out, again)
    for b, L in enumerate(lens):
        for blocks in (-(-L // 32), cache.row_pages):
            wide = torch.zeros(1, 4 * blocks if blocks < cache.row_pages else blocks, dtype=torch.int32,
                               device="cuda")
            wide[0, :blocks] = cache.table[b, :blocks]
            alone = sd.Cache8(cache.pages, cache.scales, wide)
            one = torch.empty_like(q[b:b + 1])
            alone.attend(q[b:b + 1].contiguous(), ln[b:b + 1].contiguous(), one)
            assert torch.equal(one[0], out[b]), (b, blocks)


@pytest.mark.parametrize("dh,t,share,rows,long", [(128, "bf16", 1, 40, 9000), (64, "fp32", 2, 70, 5000),
                                                  (128, "bf16", 4, 24, 20000), (128, "fp32", 8, 12, 5000)])
def test_attend_long_rows_do_not_depend_on_the_batch(sd, dh, t, share, rows, long):
    """A batch that fills the machine gives a row few warps, a row alone gets many: the same bits."""
    import torch
    dt = torch.float32 if t == "fp32" else torch.bfloat16
    lens = [long - 321 * b % long if b % 3 else 17 * b for b in range(rows)]
    cache = _new_cache(sd, rows, long, 64, 4, dh, seed=2)
    q = torch.randn(rows, 1, 4 * share, dh, generator=_gen(5), device="cuda").to(dt)
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
    out = torch.empty_like(q)
    cache.attend(q, ln, out)
    for b in (0, 1, 2, rows - 1):
        alone = sd.Cache8(cache.pages, cache.scales, cache.table[b:b + 1].contiguous())
        one = torch.empty_like(q[:1])
        alone.attend(q[b:b + 1].contiguous(), ln[b:b + 1].contiguous(), one)
        assert torch.equal(one[0], out[b]), (b, lens[b])


def test_attend_ignores_what_lies_behind_the_prefix(sd):
    """NaN bytes in every slot, page and scale past the prefix, and wild table entries past it."""
    import torch
    for dh, n, heads in ((64, 1, 1), (128, 4, 6)):
        cache = _new_cache(sd, 3, 96, 16, 1, dh, seed=2)
        lens = [5, 33, 96]
        clean = torch.randn(3, n, heads, dh, generator=_gen(4), device="cuda").bfloat16()
        ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
        want = torch.empty_like(clean)
        cache.attend(clean, ln, want)
        used = torch.zeros(len(cache.pages), 16, dtype=torch.bool, device="cuda")
        for b, L in enumerate(lens):
            for j in range(-(-L // 16)):
                used[int(cache.table[b, j]), : min(16, L - 16 * j)] = True
            cache.table[b, -(-L // 16):] = 2 ** 30
        cache.pages.permute(0, 3, 1, 2, 4)[~used] = 0xff
        cache.scales[~used.any(1)] = float("nan")
        got = torch.empty_like(clean)
        cache.attend(clean, ln, got)
        torch.cuda.synchronize()
        assert torch.equal(got, want) and int(cache.status) == 0


def test_attend_nan_reaches_those_that_see_it_only(sd):
    import torch
    for t in (torch.float32, torch.bfloat16):
        cache = _new_cache(sd, 1, 64, 16, 1, 64, seed=6)
        q = torch.randn(1, 4, 3, 64, generator=_gen(4), device="cuda").to(t)   # bf16: 12 queries, 16 rows
        ln = torch.tensor([40], dtype=torch.int32, device="cuda")
        want, got = torch.empty_like(q), torch.empty_like(q)
        cache.attend(q, ln, want)
        cache.pages[int(cache.table[0, 2]), 1, 0, 6, 9] = 0x7f      # value of token 38, dim 9
        cache.attend(q, ln, got)
        assert torch.equal(got[0, :2], want[0, :2])                 # tokens 36 and 37 do not see it
        assert bool(torch.isnan(got[0, 2:, :, 9]).all())
        cache.pages[int(cache.table[0, 2]), 1, 0, 6, 9] = 0
        cache.pages[int(cache.table[0, 0]), 0, 0, 0, 0] = 0xff      # key of token 0
        cache.attend(q, ln, got)
        assert bool(torch.isnan(got).all())
        cache.attend(torch.full_like(q, float("inf")), ln, got)
        torch.cuda.synchronize()


def test_attend_wide_scores_and_scales(sd):
    """Scores far apart, scales 2^-60 to 2^20 apart, values of one page dwarfing the others."""
    import torch
    cache = _new_cache(sd, 2, 200, 16, 2, 64, seed=8)
    cache.scales[:, 0] = torch.exp2(torch.randint(-9, -2, cache.scales[:, 0].shape, generator=_gen(1), device="cuda").float())
    cache.scales[:, 1] = torch.exp2(torch.randint(-60, 20, cache.scales[:, 1].shape, generator=_gen(2), device="cuda").float())
    cache.scales[:, 1] *= 1.375                                     # and no powers of two
    q = 30 * torch.randn(2, 1, 2, 64, generator=_gen(3), device="cuda")
    ln = torch.tensor([200, 131], dtype=torch.int32, device="cuda")
    out = torch.empty_like(q)
    cache.attend(q, ln, out, scale=-0.2)
    torch.cuda.synchronize()
    _check_attend(cache, q, out, [200, 131], -0.2, None, False)
    assert bool(torch.isfinite(out).all())
    zero = torch.zeros_like(q)                                      # all scores equal: the mean
    cache.attend(zero, ln, out)
    _check_attend(cache, zero, out, [200, 131], 0.125, None, False)


def test_attend_bad_lengths_pages_and_positions(sd):
    import torch
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    cache = _new_cache(sd, 2, 64, 16, 1, 64, seed=9)
    q = torch.randn(2, 1, 1, 64, generator=_gen(3), device="cuda")
    out, full = torch.empty_like(q), torch.empty_like(q)
    cache.attend(q, i32(64, 64), full)
    for lens in ((65, 64), (2 ** 31 - 1, 64)):                      # cut to the capacity
        cache.status.zero_()
        cache.attend(q, i32(*lens), out)
        assert int(cache.status) == sd.RLT_E_CAPACITY and torch.equal(out, full)
    cache.status.zero_()
    cache.attend(q, i32(-5, 64), out)
    assert int(cache.status) == sd.RLT_E_CAPACITY
    assert not out[0].any() and torch.equal(out[1], full[1])
    # a page that does not exist: its keys are not seen
    cache.status.zero_()
    table = cache.table.clone()
    cache.table[0, 3] = len(cache.pages)
    cache.attend(q, i32(64, 64), out)
    assert int(cache.status) == sd.RLT_E_ARG
    cut = torch.empty_like(q)
    cache.table.copy_(table)
    cache.attend(q, i32(48, 64), cut)
    assert float((out - cut).abs().max()) < 1e-5
    # a position without a rotation: zeros for that query, the others as they are
    q4 = torch.randn(2, 4, 1, 64, generator=_gen(3), device="cuda")
    a, b = torch.empty_like(q4), torch.empty_like(q4)
    cache.status.zero_()
    cache.attend(q4, i32(64, 30), a, rope=_rope(sd, 64, 64))
    assert int(cache.status) == 0
    cache.attend(q4, i32(64, 30), b, rope=_rope(sd, 64, 62))
    torch.cuda.synchronize()
    assert int(cache.status) == sd.RLT_E_CAPACITY
    assert torch.equal(a[1], b[1]) and torch.equal(a[0, :2], b[0, :2]) and not b[0, 2:].any()


def test_long_cache_offsets_pass_32_bits(sd):
    """Pages beyond 4 GiB, read and written at the far end."""
    import torch
    n_pages, page, dh = 17_000, 128, 128
    pages = torch.zeros(n_pages, 2, 8, page, dh, dtype=torch.uint8, device="cuda")      # 4.4 GB
    scales = torch.ones(n_pages, 2, 8, device="cuda")
    table = torch.tensor([[n_pages - 1, 3], [n_pages - 2, 5]], dtype=torch.int32, device="cuda")
    cache = sd.Cache8(pages, scales, table)
    k = torch.randn(2, 130, 8, dh, generator=_gen(2), device="cuda").bfloat16()
    cache.append(k, k, torch.zeros(2, dtype=torch.int32, device="cuda"))
    x = pages[n_pages - 1].view(torch.float8_e4m3fn).float() * scales[n_pages - 1][..., None, None]
    ref = k[0, :128].float().permute(1, 0, 2)
    assert bool(((x[0] - ref).abs() <= ref.abs() * 2.0 ** -4 + 2.0 ** -10 * scales[n_pages - 1, 0][:, None, None]).all())
    q = torch.randn(2, 1, 8, dh, generator=_gen(3), device="cuda")
    out = torch.empty_like(q)
    ln = torch.tensor([130, 129], dtype=torch.int32, device="cuda")
    cache.attend(q, ln, out)
    small = sd.Cache8(pages[[n_pages - 1, 3, n_pages - 2, 5]].contiguous(),
                      scales[[n_pages - 1, 3, n_pages - 2, 5]].contiguous(),
                      torch.tensor([[0, 1], [2, 3]], dtype=torch.int32, device="cuda"))
    same = torch.empty_like(q)
    small.attend(q, ln, same)
    torch.cuda.synchronize()
    assert torch.equal(out, same) and bool(out.any())


# ------------------------------------------------------------------------------ selection
def _select64(logits, scores, finished, eos, temperature, k):
    """(parents, tokens, scores in fp64) by the definition, and every candidate's value."""
    import torch
    G, K, V = logits.shape
    x = logits.double()
    x = torch.where(torch.isnan(x), -math.inf, x) / temperature
    c = scores.double()[..., None] + torch.log_softmax(x, -1)
    if finished is not None:
        only = torch.full_like(c, -math.inf)
        only[..., eos] = scores.double()
        c = torch.where(finished.bool()[..., None], only, c)
    c = torch.where(torch.isnan(c) | ~torch.isfinite(scores)[..., None], -math.inf, c).flatten(1)
    top, at = c.sort(dim=1, descending=True, stable=True)
    top, at = top[:, :k], at[:, :k]
    none = top == -math.inf
    return torch.where(none, 0, at // V), torch.where(none, 0, at % V), top, c


def _run_select(sd, logits, scores, k, finished=None, eos=-1, temperature=1.0, stream=None):
    import torch
    G = logits.shape[0]
    out = [torch.full((G, k), -7, dtype=torch.int32, device="cuda") for _ in range(2)]
    new = torch.full((G, k), 3.0, device="cuda")
    fin = torch.full((G, k), 9, dtype=torch.uint8, device="cuda")
    sd.beam_select(logits, scores, out[0], out[1], new, finished=finished, new_finished=fin, eos=eos,
                   temperature=temperature, stream=stream)
    return out[0], out[1], new, fin


def _check_select(sd, logits, scores, k, finished=None, eos=-1, temperature=1.0):
    import torch
    p, t, new, fin = _run_select(sd, logits, scores, k, finished, eos, temperature)
    wp, wt, wc, every = _select64(logits, scores, finished, eos, float(np.float32(temperature)), k)
    torch.cuda.synchronize()
    V = logits.shape[2]
    finite = wc > -math.inf
    # Values: the log-sum's error (2^-21: single exponentials are off by about 2^-22, the fp64 sums
    # by nothing) and one fp32 rounding.
    tol = 2.0 ** -21 + 2.0 ** -24 * wc.abs()
    assert torch.equal(torch.isinf(new), ~finite)
    assert bool(((new.double() - wc).abs() <= tol)[finite].all()), float((new.double() - wc)[finite].abs().max())
    # Choices: the same, unless two candidates of different beams lie within that error
    same = (p == wp) & (t == wt)
    mine = every.gather(1, (p.long() * V + t))
    gap = (mine - wc).abs()
    other_beam = p != wp
    assert bool((same | (finite & other_beam & (gap < 2 * 2.0 ** -21))).all())
    assert bool(((p == 0) & (t == 0))[~finite].all())
    was = torch.zeros_like(p, dtype=torch.bool) if finished is None else finished.bool().gather(1, p.long())
    assert torch.equal(fin.bool(), finite & (was | (t == eos)))
    flat = p.long() * V + t
    for g in range(len(p)):                                         # no candidate twice
        f = flat[g][finite[g]]
        assert len(set(f.tolist())) == len(f)


@pytest.mark.parametrize("groups,beams,vocab,k,t", [
    (1, 1, 1, 1, "fp32"), (2, 1, 7, 7, "bf16"), (3, 2, 32, 4, "fp32"), (1, 4, 32000, 4, "fp32"),
    (5, 3, 4097, 6, "bf16"), (2, 8, 5003, 16, "fp32"), (1, 1, 131071, 64, "bf16"),
    (2, 9, 1000, 9, "bf16"), (1, 64, 513, 64, "fp32"), (3, 17, 2049, 33, "fp32"), (40, 5, 12, 5, "bf16")])
def test_select(sd, groups, beams, vocab, k, t):
    import torch
    g = _gen(groups + vocab)
    dt = torch.float32 if t == "fp32" else torch.bfloat16
    logits = (3 * torch.randn(groups, beams, vocab, generator=g, device="cuda")).to(dt)
    scores = -5 * torch.rand(groups, beams, generator=g, device="cuda")
    _check_select(sd, logits, scores, k)
    fin = (torch.rand(groups, beams, generator=g, device="cuda") < 0.3).to(torch.uint8)
    scores[0, beams // 2:] = -math.inf
    _check_select(sd, logits, scores, k, finished=fin, eos=vocab // 2, temperature=0.6)


def test_select_ties_take_the_lowest_index(sd):
    """Equal logits and equal beams: ascending (beam, token), past the candidate buffer too."""
    import torch
    for V in (16, 1000, 20000):
        for t in (torch.float32, torch.bfloat16):
            logits = torch.zeros(2, 3, V, device="cuda", dtype=t)
            scores = torch.zeros(2, 3, device="cuda")
            p, tok, new, _ = _run_select(sd, logits, scores, 6)
            assert p.tolist() == [[0] * 6] * 2 and tok.tolist() == [[0, 1, 2, 3, 4, 5]] * 2
            # two values, the larger one at scattered places, more of them than any buffer
            logits[:, :, 3::2] = 1.0
            scores[:, 0] = -1.0
            p, tok, new, _ = _run_select(sd, logits, scores, 5)
            assert p.tolist() == [[1] * 5] * 2 and tok.tolist() == [[3, 5, 7, 9, 11]] * 2
    logits = torch.arange(5000, device="cuda").float().repeat(1, 2, 1)
    p, tok, _, _ = _run_select(sd, logits, torch.zeros(1, 2, device="cuda"), 4)
    assert p.tolist() == [[0, 1, 0, 1]] and tok.tolist() == [[4999, 4999, 4998, 4998]]


def test_select_masked_and_unusual_logits(sd):
    import torch
    g = _gen(4)
    V = 9001
    low = torch.finfo(torch.float32).min
    x = 4 * torch.randn(6, 2, V, generator=g, device="cuda")
    x[0, :, 5:] = -math.inf                     # few tokens left
    x[1, 0] = -math.inf                         # a beam with none
    x[2, :, ::2] = low                          # masks of the type's lowest value
    x[3, 0, 17] = math.inf                      # no candidate of this beam
    x[4, :, 100:200] = math.nan
    x[5] = -math.inf
    x[5, 1, 8] = -3.0                           # one candidate in all
    s = -torch.rand(6, 2, generator=g, device="cuda")
    want = x.clone()
    want[3, 0] = -math.inf
    p, t, new, fin = _run_select(sd, x, s, 12)
    wp, wt, wc, _ = _select64(want, s, None, -1, 1.0, 12)
    torch.cuda.synchronize()
    ok = wc > -math.inf
    assert torch.equal(p, wp.int()) and torch.equal(t, wt.int())
    assert torch.equal(ok, torch.isfinite(new))
    assert float((new.double() - wc)[ok].abs().max()) < 2.0 ** -21 + 2.0 ** -24 * 60
    assert int(ok[0].sum()) == 10 and int(ok[5].sum()) == 1 and not fin.any()
    # all masked by the lowest value, and huge spreads
    x = torch.full((1, 2, 50), low, device="cuda")
    _check_select(sd, x, torch.zeros(1, 2, device="cuda"), 3)
    x[0, 0, 7] = -low
    _check_select(sd, x, torch.zeros(1, 2, device="cuda"), 2)


def test_select_groups_do_not_depend_on_the_batch(sd):
    import torch
    g = _gen(9)
    x = torch.randn(7, 3, 9999, generator=g, device="cuda")          # rows off every 16-byte boundary
    s = torch.randn(7, 3, generator=g, device="cuda")
    p, t, new, _ = _run_select(sd, x, s, 3)
    for i in range(7):
        a = _run_select(sd, x[i:i + 1].clone(), s[i:i + 1].clone(), 3)
        assert torch.equal(a[0][0], p[i]) and torch.equal(a[1][0], t[i]) and torch.equal(a[2][0], new[i])


# ------------------------------------------------------------------------------ reordering
@pytest.mark.parametrize("groups,beams,planes,cap,width,dtype,start,stop", [
    (1, 2, 1, 1, 512, "float32", 0, 1), (3, 4, 5, 9, 64, "bfloat16", 2, 7), (2, 8, 2, 33, 128, "bfloat16", 0, 33),
    (2, 16, 3, 5, 64, "uint8", 1, 5), (2, 17, 3, 5, 24, "uint8", 0, 4), (1, 32, 2, 7, 16, "float32", 3, 4),
    (1, 64, 2, 5, 8, "float32", 0, 5), (3, 5, 2, 7, 3, "uint8", 1, 6), (2, 3, 4, 5, 3, "float32", 2, 5),
    (2, 33, 1, 3, 5, "bfloat16", 0, 2), (4, 1, 2, 3, 8, "float32", 0, 3), (2, 4, 2, 3, 8, "float32", 2, 2),
    (2, 6, 1, 700, 1000, "uint8", 1, 699)])
def test_reorder(sd, groups, beams, planes, cap, width, dtype, start, stop):
    import torch
    dt = getattr(torch, dtype)
    g = _gen(groups * beams)
    rows = torch.randint(0, 200, (groups * beams, planes, cap, width), generator=g, device="cuda").to(dt)
    for kind in ("random", "cycle", "same", "out of range"):
        if kind == "random":
            parents = torch.randint(0, beams, (groups, beams), generator=g, device="cuda")
        elif kind == "cycle":
            parents = torch.stack([torch.randperm(beams, generator=g, device="cuda") for _ in range(groups)])
        elif kind == "same":
            parents = torch.arange(beams, device="cuda").repeat(groups, 1)
        else:
            parents = torch.randint(0, beams, (groups, beams), generator=g, device="cuda")
            parents[:, 0] = -1
            parents[:, beams // 2] = beams
        src = torch.where((parents < 0) | (parents >= beams), torch.arange(beams, device="cuda"), parents)
        src = (src + beams * torch.arange(groups, device="cuda")[:, None]).flatten()
        want = rows.clone()
        want[:, :, start:stop] = rows[src, :, start:stop]
        got = rows.clone()
        sd.rows_reorder(got, parents.int().contiguous(), start=start, stop=stop)
        torch.cuda.synchronize()
        assert torch.equal(got, want), kind


def test_reorder_strided_layouts(sd):
    """Rows inside planes (plane-major), rows with a gap behind them, a base off the alignment."""
    import torch
    g = _gen(1)
    parents = torch.tensor([[1, 2, 0], [2, 2, 1]], dtype=torch.int32, device="cuda")
    src = torch.tensor([1, 2, 0, 5, 5, 4], device="cuda")
    store = torch.randn(4, 6, 5, 16, generator=g, device="cuda")           # [planes][rows][cap][width]
    want = store[:, src].clone()
    sd.rows_reorder(store.transpose(0, 1), parents)
    assert torch.equal(store, want)
    store = torch.randn(6, 7, 5, 16, generator=g, device="cuda")           # three of seven planes
    want = store.clone()
    want[:, 2:5] = store[src, 2:5]
    sd.rows_reorder(store[:, 2:5], parents)
    assert torch.equal(store, want)
    flat = torch.randn(6 * 40 + 1, generator=g, device="cuda")
    view = flat[1:].view(6, 2, 5, 4)                                       # 4-byte aligned only
    want = view[src].clone()
    keep = flat[0].clone()
    sd.rows_reorder(view, parents)
    torch.cuda.synchronize()
    assert torch.equal(view, want) and torch.equal(flat[0], keep)
    with pytest.raises(ValueError):
        sd.rows_reorder(view.transpose(2, 3), parents)
    with pytest.raises(sd.RLTError):
        sd.rows_reorder(view[:1].expand(6, 2, 5, 4), parents)              # one row six times


# ------------------------------------------------------------------------------ refusals
def test_owners_refuse(sd):
    import torch
    cache = _new_cache(sd, 2, 32, 16, 2, 64)
    i32 = torch.zeros(2, dtype=torch.int32, device="cuda")
    k = torch.zeros(2, 1, 2, 64, device="cuda")
    for bad in (k.half(), k.double(), k.cpu()):
        with pytest.raises(TypeError):
            cache.append(bad, bad, i32)
        with pytest.raises(TypeError):
            cache.attend(bad, i32, bad)
    with pytest.raises(TypeError):
        cache.append(k, k.bfloat16(), i32)
    with pytest.raises(TypeError):
        cache.append(k, k, i32.long())
    with pytest.raises(ValueError):
        cache.append(k[:1], k[:1], i32)
    with pytest.raises(ValueError):
        cache.append(k, k, i32[:1])
    with pytest.raises(ValueError):
        cache.append(k.transpose(2, 3).contiguous().transpose(2, 3), k, i32)
    with pytest.raises(sd.RLTError):                               # a pitch off 16 bytes
        odd = torch.zeros(2, 131, device="cuda")[:, :128].view(2, 1, 2, 64)
        cache.append(odd, odd, i32)
    with pytest.raises(sd.RLTError):                               # heads no multiple of kv_heads
        cache.attend(torch.zeros(2, 1, 3, 64, device="cuda"), i32, torch.zeros(2, 1, 3, 64, device="cuda"))
    with pytest.raises(sd.RLTError):
        cache.attend(k, i32, torch.empty_like(k), scale=float("nan"))
    with pytest.raises(sd.RLTError):
        cache.append(k, k, i32, rope=_rope(sd, 12, 32))            # not a multiple of 8
    with pytest.raises(sd.RLTError):
        cache.append(k, k, i32, rope=_rope(sd, 128, 32))           # wider than the head
    assert cache.append(k[:, :0], k[:, :0], i32) == sd.RLT_OK      # nothing to do
    assert cache.attend(k[:, :0], i32, k[:, :0]) == sd.RLT_OK


# ------------------------------------------------------------------------------ together
def test_streams_and_graphs(sd):
    """On another stream, and captured once and replayed with new lengths, tables and logits."""
    import torch
    st = torch.cuda.Stream()
    cache = _new_cache(sd, 2, 128, 16, 2, 64, seed=1)
    k = torch.randn(2, 1, 2, 64, generator=_gen(1), device="cuda")
    q, out = torch.randn(2, 1, 4, 64, generator=_gen(2), device="cuda"), torch.zeros(2, 1, 4, 64, device="cuda")
    start = torch.tensor([30, 99], dtype=torch.int32, device="cuda")
    lens = start + 1
    x = torch.randn(1, 2, 5000, generator=_gen(3), device="cuda")
    sc = torch.zeros(1, 2, device="cuda")
    par, tok = (torch.zeros(1, 2, dtype=torch.int32, device="cuda") for _ in range(2))
    new = torch.zeros(1, 2, device="cuda")
    rows = torch.randn(2, 1, 4, 16, generator=_gen(4), device="cuda")

    def step(stream):
        cache.append(k, k, start, stream=stream)
        cache.attend(q, lens, out, stream=stream)
        sd.beam_select(x, sc, par, tok, new, stream=stream)
        sd.rows_reorder(rows, par, stream=stream)

    torch.cuda.synchronize()
    step(st)                                                       # also before any capture
    st.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        step(torch.cuda.current_stream())
    for seed in (5, 6):
        k.normal_(generator=_gen(seed))
        q.normal_(generator=_gen(seed + 10))
        x.normal_(generator=_gen(seed + 20))
        start.copy_(torch.tensor([seed, 100 + seed], dtype=torch.int32))
        lens.copy_(start + 1)
        twin = sd.Cache8(cache.pages.clone(), cache.scales.clone(), cache.table.clone())
        twin_out, twin_rows = torch.zeros_like(out), rows.clone()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        twin.append(k, k, start)
        twin.attend(q, lens, twin_out)
        p, t, n, _ = _run_select(sd, x, sc, 2)
        sd.rows_reorder(twin_rows, p)
        torch.cuda.synchronize()
        assert torch.equal(cache.pages, twin.pages) and torch.equal(cache.scales, twin.scales)
        assert torch.equal(out, twin_out) and torch.equal(par, p) and torch.equal(tok, t)
        assert torch.equal(new, n) and torch.equal(rows, twin_rows)
    assert torch.cuda.current_device() == 0


def test_a_decoding_step_of_all_four(sd):
    """Three steps of a beam search over a cache of pages whose rows are moved as they fork:
    append, attend, a readout by a fixed matrix, select, reorder; against the plain forms."""
    import torch
    g = _gen(11)
    G, K, H, D, page, V = 2, 3, 2, 64, 16, 101
    B = G * K
    cache = _new_cache(sd, B, 32, page, H, D, seed=4, spare=0)
    order = torch.arange(len(cache.pages), dtype=torch.int32, device="cuda")
    cache.table.copy_(order.view(B, -1))                           # page j of row b at b * row_pages + j
    emb = torch.randn(V, H * D, generator=g, device="cuda")
    rope = _rope(sd, D, 64)
    start = torch.full((B,), 13, dtype=torch.int32, device="cuda")
    tok = torch.randint(0, V, (B,), generator=g, device="cuda").int()
    scores = torch.zeros(G, K, device="cuda")
    scores[:, 1:] = -math.inf
    hist = cache.pages.clone(), cache.scales.clone()
    for step in range(3):
        x = emb[tok.long()].view(B, 1, H, D)
        before, bs = cache.pages.clone(), cache.scales.clone()
        cache.append(x, x * 0.5, start, rope=rope)
        _check_append(cache, before, bs, x, x * 0.5, start.tolist(), [1] * B, rope)
        out = torch.empty_like(x)
        cache.attend(x, start + 1, out, rope=rope)
        _check_attend(cache, x, out, (start + 1).tolist(), D ** -0.5, rope, False)
        logits = (out.view(B, -1) @ emb.T).view(G, K, V).contiguous()
        par, t, new, _ = _run_select(sd, logits, scores, K)
        wp, wt, wc, _ = _select64(logits, scores, None, -1, 1.0, K)
        assert torch.equal(par, wp.int()) and torch.equal(t, wt.int())
        want_p, want_s = (z.view(B, -1)[(par.long() + K * torch.arange(G, device="cuda")[:, None]).flatten()]
                          for z in (cache.pages.clone(), cache.scales.clone()))
        sd.rows_reorder(cache.pages.view(B, cache.row_pages, 1, -1), par)
        sd.rows_reorder(cache.scales.view(B, 1, 1, -1), par)
        torch.cuda.synchronize()
        assert torch.equal(cache.pages.view(B, -1), want_p) and torch.equal(cache.scales.view(B, -1), want_s)
        tok, scores, start = t.flatten(), new, start + 1
    assert int(cache.status) == 0
