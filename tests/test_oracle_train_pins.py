"""The oracle's embedding, layer norm and optimiser step, pinned independently:
gradients by differences, values by hand and against torch in float64, the
8-bit moments by the e4m3 type's own values."""
import numpy as np
import pytest
import torch

import oracle


def _rng(seed):
    return np.random.Generator(np.random.PCG64(seed))


def test_embed_by_hand():
    table = np.array([[1.0, 2.0], [3.0, 4.0], [5.0, 6.0]])
    dout = np.array([[1.0, 0.0], [0.0, 1.0], [7.0, 7.0], [2.0, 2.0], [9.0, 9.0]])
    out, grad = oracle.embed([2, 0, -1, 2, 3], table, 2.0, dout)
    assert out.tolist() == [[10, 12], [2, 4], [0, 0], [10, 12], [0, 0]]
    assert grad.tolist() == [[0, 2], [0, 0], [6, 4]]


def test_embed_gradient_by_differences():
    r = _rng(1)
    table, tok, dout = r.standard_normal((6, 3)), np.array([1, 5, 1, -3, 0, 6]), r.standard_normal((6, 3))
    _, grad = oracle.embed(tok, table, 1.7, dout)
    for t in range(6):
        for c in range(3):
            e = np.zeros_like(table)
            e[t, c] = 1e-3
            num = ((oracle.embed(tok, table + e, 1.7) - oracle.embed(tok, table - e, 1.7)) * dout).sum() / 2e-3
            assert abs(num - grad[t, c]) < 1e-9


@pytest.mark.parametrize("d", [1, 2, 7])
def test_layer_norm_by_differences(d):
    r = _rng(2)
    s, dy, ds = (r.standard_normal((4, d)) for _ in range(3))
    gamma, beta = r.standard_normal(d), r.standard_normal(d)
    y, mean, rstd, g = oracle.layer_norm(s, gamma, beta, 1e-2, dy, ds)
    want = torch.nn.functional.layer_norm(torch.from_numpy(s), (d,), torch.from_numpy(gamma), torch.from_numpy(beta), 1e-2)
    assert np.allclose(y, want.numpy(), atol=1e-12)
    value = lambda s, gamma, beta: float((oracle.layer_norm(s, gamma, beta, 1e-2)[0] * dy).sum() + (ds * s).sum())
    for name, x in (("dx", s), ("dgamma", gamma), ("dbeta", beta)):
        for at in np.ndindex(x.shape):
            e = np.zeros_like(x)
            e[at] = 1e-5
            args = {"dx": lambda k: (s + k * e, gamma, beta), "dgamma": lambda k: (s, gamma + k * e, beta),
                    "dbeta": lambda k: (s, gamma, beta + k * e)}[name]
            num = (value(*args(1)) - value(*args(-1))) / 2e-5
            assert abs(num - g[name][at]) < 1e-6 * (1 + abs(num)), (name, at)


def test_adamw_against_torch():
    r = _rng(3)
    p0 = r.standard_normal(50)
    p = torch.nn.Parameter(torch.from_numpy(p0.copy()))
    opt = torch.optim.AdamW([p], lr=3e-2, betas=(0.8, 0.95), eps=1e-4, weight_decay=0.1, foreach=False)
    x, m, v = p0, np.zeros(50), np.zeros(50)
    for t in range(1, 6):
        g = r.standard_normal(50)
        p.grad = torch.from_numpy(g.copy())
        opt.step()
        x, m, v = oracle.adamw(x, g * 4, m, v, 3e-2, t, 0.8, 0.95, 1e-4, 0.1, grad_scale=0.25)
        # torch multiplies by 1 - lr wd first: the same to rounding
        assert np.allclose(x, p.detach().numpy(), atol=1e-13)


def test_grad_norm():
    g = [np.full(9, 2.0), np.full((4, 4), -2.0)]
    assert oracle.grad_norm(g, 100.0) == (10.0, 1.0)
    assert oracle.grad_norm(g, 2.5) == (10.0, 0.25)


def _e4m3_values():
    return torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double()


def test_moment_codes_are_e4m3_values():
    """Every code is a value of the type, one of the two next to what is
    stored, and the average over the random fractions is what is stored."""
    values = _e4m3_values()
    values = np.unique(values[values.isfinite()].numpy())
    r = _rng(4)
    x = r.standard_normal(700) * 10.0 ** r.uniform(-6, 0, 700)
    x[300:310] = 0.0
    u = (np.arange(700) * 37 % 65536) / 65536.0
    c, scale, _ = oracle.moment_codes(x, u, False)
    assert np.isin(c, values).all()
    y = x / np.repeat(scale, 256)[:700]
    at = np.searchsorted(values, y, side="right") - 1
    low, high = values[np.maximum(at, 0)], values[np.minimum(at + 1, len(values) - 1)]
    near = (c == low) | (c == high)
    assert near.all()
    assert abs(np.abs(c).max() - 448.0) < 1e-12 and len(scale) == 3
    total = np.zeros(256)
    for k in range(256):
        total += oracle.moment_codes(x[:256], np.full(256, k / 256.0 + 1 / 512), False)[0]
    one = np.abs(y[:256]) < 447
    # the mean of 256 equidistant fractions is within half a step of 1/256 of the code's step
    assert (np.abs(total / 256 - y[:256]) <= np.maximum(np.abs(y[:256]) / 8, 2.0 ** -9) / 256 + 1e-12)[one].all()


def test_moment_codes_keep_denominators():
    x = np.full(300, 1e-12)
    x[0] = x[299] = 1.0
    x[7] = 0.0
    c, _, _ = oracle.moment_codes(x, np.zeros(300), True)
    assert (c[x > 0] > 0).all() and c[7] == 0 and c[0] == c[299] == 448 and c[5] == 2.0 ** -9
    assert not oracle.moment_codes(np.full(5, 1e-31), np.zeros(5), True)[0].any()


def test_moment_bits():
    """Uniform, independent between the halves, tensors and steps."""
    a, b = oracle.moment_bits(7, 0, 1, 20000)
    assert a.min() >= 0 and a.max() < 1 and (a * 65536 % 1 == 0).all()
    other = [oracle.moment_bits(7, 0, 2, 20000)[0], oracle.moment_bits(7, 1, 1, 20000)[0],
             oracle.moment_bits(8, 0, 1, 20000)[0], oracle.moment_bits(7 + (1 << 32), 0, 1, 20000)[0],
             oracle.moment_bits(7, 0, 1, 20000, first=1 << 32)[0]]
    for x in (a, b):
        # 10 bins of 2000: five standard deviations are 212
        assert np.abs(np.histogram(x, 10, (0, 1))[0] - 2000).max() < 213
    for x in [b] + other:
        # a correlation over 20000 pairs has a standard deviation of 0.0071
        assert abs(np.corrcoef(a, x)[0, 1]) < 0.036
