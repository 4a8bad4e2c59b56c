"""Appended keys, byte by byte: rotated by products and sums that round to fp32 one by one, divided by a power
of two, rounded to nearest even.  What separate elementary operations give, millions of values long: a fused
multiply-add differs in about one byte of a million, where a sum lies at a rounding border."""
import pytest

from tests.test_operators_gpu import _gen, _rope, _settle, sd  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dh,rot,interleaved,t", [
    (64, 64, False, "fp32"), (128, 128, False, "fp32"), (128, 64, True, "fp32"), (64, 24, False, "fp32"), (64, 40, True, "fp32"),
    (128, 128, True, "bf16"), (64, 32, False, "bf16")])
@pytest.mark.parametrize("n", [1, 5, 1024])
def test_keys_are_rotated_with_every_rounding(sd, dh, rot, interleaved, t, n):  # noqa: F811
    import torch
    page, kv, rows = 64, 8, 16384 // max(n, 64)
    row_pages = -(-n // page)
    cache = sd.Cache8(torch.zeros(rows * row_pages, 2, kv, page, dh, dtype=torch.uint8, device="cuda"),
                      torch.ones(rows * row_pages, 2, kv, device="cuda"),
                      torch.arange(rows * row_pages, dtype=torch.int32, device="cuda").view(rows, row_pages))
    rope = _rope(sd, rot, n + 3000, interleaved, 2999)
    for seed in range(2 if n > 64 else 12):
        k = torch.randn(rows, n, kv, dh, generator=_gen(seed), device="cuda")
        k = k if t == "fp32" else k.bfloat16()
        cache.append(k, k, torch.zeros(rows, dtype=torch.int32, device="cuda"), rope=rope)
        torch.cuda.synchronize()
        cos, sin = (x[2999:2999 + n, None] for x in rope.buffers)
        x = k.float()
        a, b = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
        ac, bs, bc, as_ = x[..., a] * cos, x[..., b] * sin, x[..., b] * cos, x[..., a] * sin     # rounded,
        y = x.clone()
        y[..., a], y[..., b] = ac - bs, bc + as_                                                 # and again
        pages = cache.pages.view(rows, row_pages, 2, kv, page, dh).permute(0, 1, 4, 2, 3, 5).reshape(rows, -1, 2, kv, dh)
        scales = cache.scales.view(rows, row_pages, 1, 2, kv).expand(-1, -1, page, -1, -1).reshape(rows, -1, 2, kv)
        for w, z in ((0, y), (1, x)):
            want = (z / scales[:, :n, w, :, None]).to(torch.float8_e4m3fn).view(torch.uint8)
            assert int((pages[:, :n, w] != want).sum()) == 0
