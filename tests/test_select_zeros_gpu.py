"""Beam selection's ties between zeros of either sign: they are equal, so the lower index goes first."""
import pytest

from tests.test_operators_gpu import _gen, _run_select, _select64, _settle, sd  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("t", ["fp32", "bf16"])
@pytest.mark.parametrize("vocab,zeros", [(50, 12), (50, 50), (3001, 40), (40000, 300), (40000, 40000)])
def test_zeros_of_either_sign_are_equal(sd, t, vocab, zeros):  # noqa: F811
    import torch
    dt = torch.float32 if t == "fp32" else torch.bfloat16
    g = _gen(vocab + zeros)
    for beams, k in ((1, 7), (3, 5)):
        x = -1.0 - torch.rand(4, beams, vocab, generator=g, device="cuda")
        at = torch.rand(4, beams, vocab, generator=g, device="cuda").argsort(-1)[..., :zeros]
        sign = torch.where(torch.rand(at.shape, generator=g, device="cuda") < 0.5, -0.0, 0.0)
        x = x.scatter(-1, at, sign).to(dt)
        x[1, :, 3] = 2.0                            # the zeros are not the best, but among them
        x[2] = torch.where(x[2] == 0, -0.0, x[2])   # all negative, but the last
        x[2, :, at[2, :, 0].max()] = 0.0
        scores = torch.zeros(4, beams, device="cuda")
        scores[:, 1:] = -3.0
        p, tok, new, _ = _run_select(sd, x, scores, k)
        wp, wt, wc, _ = _select64(x, scores, None, -1, 1.0, k)
        torch.cuda.synchronize()
        assert torch.equal(p, wp.int()) and torch.equal(tok, wt.int())
        # the log-sum is off by 2^-21 at most, the score rounds once
        assert bool(((new.double() - wc).abs() <= 2.0 ** -21 + 2.0 ** -24 * wc.abs()).all())


@pytest.mark.parametrize("t", ["fp32", "bf16"])
def test_the_first_zero_wins(sd, t):  # noqa: F811
    import torch
    dt = torch.float32 if t == "fp32" else torch.bfloat16
    x = torch.full((1, 1, 1000), -2.0, device="cuda")
    x[0, 0, 10], x[0, 0, 500:600], x[0, 0, 700] = -0.0, 0.0, -0.0
    p, tok, _, _ = _run_select(sd, x.to(dt), torch.zeros(1, 1, device="cuda"), 3)
    assert tok.tolist() == [[10, 500, 501]]
