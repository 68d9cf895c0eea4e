"""Layer norm's backward where |mean| rstd leaves fp32 while every gradient is
an ordinary number: constant rows of a large value and a small eps."""
import pytest
import torch

import transformer_xl_relative_rel_gb300 as txl
from tests.train_helpers import BF, F32, H, U

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from transformer_xl_relative_rel_gb300 import _build
    _build.build()


@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("form", ["x", "residual", "dsum"])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d", [1, 8, 33, 200, 256, 384, 410, 500, 512, 520, 771, 1000, 1024, 1500])
def test_constant_rows_far_from_zero(d, dtype, form, shift):
    """x = 2^80 in each of the columns, whose sums and mean are exact: xh is 0,
    rstd 1 / sqrt(eps) = 2^50, and dx = rstd (g - mean_d(g)) + dsum."""
    g = torch.Generator(device="cuda").manual_seed(d)
    n = lambda *s: torch.randn(*s, device="cuda", generator=g)

    def place(t):      # `shift` elements behind a 16-byte boundary
        flat = torch.empty(t.numel() + 8, dtype=t.dtype, device="cuda")
        y = flat[shift:shift + t.numel()].view(t.shape)
        y.copy_(t)
        return y

    rows = 20
    x, dy, dsum = place(torch.full((rows, d), 2.0 ** 80, device="cuda").to(dtype)), place(n(rows, d).to(dtype)), None
    residual = x.clone() if form == "residual" else None
    if form == "dsum":
        dsum = place((2.0 ** 50 * n(rows, d)).to(dtype))
    gamma = 1 + 0.3 * n(d)
    y, mean, rstd = txl.layer_norm_fwd(x, gamma, residual=residual, eps=2.0 ** -100)
    assert (mean == (2.0 ** 81 if form == "residual" else 2.0 ** 80)).all() and not y.any()
    got = txl.layer_norm_bwd(dy, x, mean, rstd, gamma=gamma, residual=residual, dsum=dsum)
    txl.check()
    t = dy.double() * gamma.double()
    m = t.mean(1, keepdim=True)
    add = 0 * t if dsum is None else dsum.double()
    want = 2.0 ** 50 * (t - m) + add
    # the sum over a row in at most 64 additions, a product, a mean, a difference, a product with rstd
    # (which is 2^-19 off at most), a sum, a rounding
    err = 2.0 ** 50 * (64 * H * t.abs().mean(1, keepdim=True) + (8 * H + 2.0 ** -19) * (t.abs() + m.abs())) + \
        2 * H * (add.abs() + want.abs())
    lim = err + U[dtype] * (want.abs() + err)
    assert torch.isfinite(got["dx"]).all()
    assert float(((got["dx"].double() - want).abs() - lim).max()) <= 0
    assert not got["dgamma"].any()
    b = dy.double().sum(0)
    assert float(((got["dbeta"].double() - b).abs() - 84 * H * dy.double().abs().sum(0)).max()) <= 0
