"""Layer norm of a residual sum and its gradients on the GPU against float64
(tests/train_helpers.py has the formulas and bounds)."""
import pytest
import torch

from tests.loss_helpers import check
from tests.train_helpers import BF, F32, norm_reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from transformer_xl_relative_rel_gb300 import _build
    _build.build()


def _shifted(x, by):
    flat = torch.empty(x.numel() + 8, dtype=x.dtype, device=x.device)
    y = flat[by:by + x.numel()].view(x.shape)
    y.copy_(x)
    return y


def _inputs(rows, d, dtype, seed, shift=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda *s: torch.randn(*s, device="cuda", generator=g)
    p = dict(x=(n(rows, d) + 3 * n(rows, 1)).to(dtype), residual=(0.5 * n(rows, d)).to(dtype), gamma=1 + 0.3 * n(d),
             beta=0.2 * n(d), dy=n(rows, d).to(dtype), dsum=n(rows, d).to(dtype))
    return {k: _shifted(v, shift) for k, v in p.items()} if shift else p


def _run(p, residual=True, keep=False, affine=True, dsum=False, eps=1e-5, **kw):
    import transformer_xl_relative_rel_gb300 as txl
    x, res = p["x"], p["residual"] if residual else None
    gamma, beta = (p["gamma"], p["beta"]) if affine else (None, None)
    total = torch.full_like(x, 7.0) if keep else None
    y, mean, rstd = txl.layer_norm_fwd(x, gamma, beta, residual=res, eps=eps, sum=total)
    a, b = (total, None) if keep else (x, res)
    g = txl.layer_norm_bwd(p["dy"], a, mean, rstd, gamma=gamma, residual=b, dsum=p["dsum"] if dsum else None, **kw)
    out = dict(y=y, mean=mean, rstd=rstd, **g)
    return dict(out, sum=total) if keep else out


def _check(p, residual=True, keep=False, affine=True, dsum=False, eps=1e-5, got=None):
    import transformer_xl_relative_rel_gb300 as txl
    got = _run(p, residual, keep, affine, dsum, eps) if got is None else got
    check(got, *norm_reference(p["x"], p["gamma"] if affine else None, p["beta"] if affine else None, eps,
                               p["residual"] if residual else None, keep, p["dy"], p["dsum"] if dsum else None))
    txl.check()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,d", [
    (1, 1), (1, 512), (2, 2), (7, 8), (8, 31), (9, 33), (300, 64), (33, 255), (40, 256), (41, 257), (1111, 410),
    (100, 511), (64, 512), (65, 520), (200, 1000), (2433, 1024), (50, 1025), (37, 1032), (20, 2047), (21, 2048), (5, 4095),
    (400, 4096), (9, 4097), (3, 5000), (170, 8191), (305, 8192), (20000, 72)])
def test_sizes(rows, d, dtype):
    p = _inputs(rows, d, dtype, rows + d)
    _check(p)
    _check(p, residual=False, affine=False, eps=0.1)
    _check(p, keep=True, dsum=True)


@pytest.mark.parametrize("flags", range(16))
@pytest.mark.parametrize("dtype,d", [(BF, 512), (F32, 90), (BF, 41), (F32, 1500)])
def test_every_form(dtype, d, flags):
    p = _inputs(60, d, dtype, 3)
    _check(p, *(bool(flags >> k & 1) for k in range(4)))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,d", [(3000, 1024), (77, 1022), (500, 768), (40, 1000), (30, 700), (900, 4096)])
def test_every_tensor_of_wide_rows(dtype, rows, d):
    """dy, x, the residual and dsum together take the most shared memory."""
    p = _inputs(rows, d, dtype, 30)
    _check(p, residual=True, dsum=True)
    _check(p, residual=True, keep=True, dsum=True)


@pytest.mark.parametrize("shift", [1, 2, 4])
@pytest.mark.parametrize("dtype,d", [(BF, 512), (F32, 256), (BF, 3000), (BF, 8192), (F32, 8192), (BF, 410)])
def test_unaligned(dtype, d, shift):
    p = _inputs(45, d, dtype, 4, shift)
    _check(p)
    _check(p, keep=True, dsum=True)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,d,shift", [(1, 513, 0), (7, 769, 0), (3000, 771, 0), (1300, 1023, 0), (2500, 411, 0),
                                          (1, 514, 1), (9, 770, 1), (5000, 1000, 1), (5000, 1024, 1), (3000, 256, 1)])
def test_rows_read_by_single_elements(dtype, rows, d, shift):
    """Odd widths, and even ones that start at an odd element; more rows than
    the backward has groups of warps, and fewer."""
    p = _inputs(rows, d, dtype, rows + d, shift)
    _check(p)
    _check(p, residual=False, affine=False, dsum=True)


def test_one_pointer_unaligned():
    p = _inputs(45, 512, BF, 5)
    for name in p:
        _check(dict(p, **{name: _shifted(p[name], 1)}), dsum=True)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_rows_far_from_zero_and_constant(dtype):
    """A mean a thousand times the deviation costs the bits it has to, no more;
    a constant row is beta."""
    p = _inputs(64, 512, dtype, 6)
    p["x"] = (p["x"].float() + 1000.0 * torch.sign(p["x"].float()[:, :1])).to(dtype)
    _check(p)
    p["x"] = torch.full_like(p["x"], 3.0)
    p["residual"].zero_()
    got = _run(p)
    assert (got["mean"] == 3).all()
    # (512 threes sum exactly)
    assert torch.equal(got["y"], p["beta"].to(dtype).expand_as(got["y"]))
    _check(p)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_large_and_small_values(dtype):
    for scale in (1e-12, 1e12):
        p = _inputs(30, 300, dtype, 7)
        for n in ("x", "residual"):
            p[n] = (p[n].float() * scale).to(dtype)
        _check(p, eps=1e-30 if scale < 1 else 1e-5)


def test_rows_that_are_not_finite_stay_alone():
    p = _inputs(100, 512, BF, 8)
    clean = _run(p)
    p["x"][7, 5], p["x"][50, 3] = float("nan"), float("inf")
    got = _run(p)
    bad = torch.zeros(100, dtype=torch.bool, device="cuda")
    bad[7] = bad[50] = True
    for n in ("y", "dx", "mean", "rstd"):
        assert torch.equal(got[n][~bad], clean[n][~bad]), n
        if n != "mean":
            assert got[n][bad].isnan().all(), n
    assert torch.equal(got["dbeta"], clean["dbeta"])


@pytest.mark.parametrize("dtype,rows,d", [(BF, 20000, 512), (F32, 900, 1024), (BF, 700, 4096)])
def test_the_same_call_gives_the_same_bits(dtype, rows, d):
    import transformer_xl_relative_rel_gb300 as txl
    p = _inputs(rows, d, dtype, 9)
    want = _run(p)
    size = txl.layer_norm_bwd_workspace_bytes(rows, d, txl.TXL_BF16 if dtype == BF else txl.TXL_F32)
    for k in range(4):
        got = _run(p, workspace=torch.full((size // 4,), float("nan"), device="cuda"))
        for n in want:
            assert torch.equal(got[n], want[n]), n


def test_gradients_asked_for_alone():
    import ctypes
    from transformer_xl_relative_rel_gb300 import abi
    p = _inputs(300, 256, BF, 10)
    want = _run(p)
    got = _run(p, weight_grads=False)
    assert got["dgamma"] is None and got["dbeta"] is None and torch.equal(got["dx"], want["dx"])
    lib = abi.load_library()
    ws = torch.empty(abi.layer_norm_bwd_workspace_bytes(300, 256, 1), dtype=torch.uint8, device="cuda")
    for which in range(2):
        out = torch.full((256,), 7.0, device="cuda")
        dx = torch.empty_like(p["x"])
        st = lib.txl_layer_norm_bwd(p["dy"].data_ptr(), p["x"].data_ptr(), p["residual"].data_ptr(), None,
                                    p["gamma"].data_ptr(), want["mean"].data_ptr(), want["rstd"].data_ptr(), 300, 256, 1,
                                    dx.data_ptr(), out.data_ptr() if which == 0 else None,
                                    out.data_ptr() if which else None, ws.data_ptr(), ctypes.c_size_t(ws.numel()),
                                    torch.cuda.current_stream().cuda_stream)
        assert st == 0
        torch.cuda.synchronize()
        assert torch.equal(out, want["dbeta" if which else "dgamma"]) and torch.equal(dx, want["dx"])


def test_statistics_not_asked_for():
    from transformer_xl_relative_rel_gb300 import abi
    p = _inputs(70, 256, BF, 11)
    want = _run(p)
    y = torch.empty_like(p["x"])
    st = abi.load_library().txl_layer_norm_fwd(p["x"].data_ptr(), p["residual"].data_ptr(), p["gamma"].data_ptr(),
                                               p["beta"].data_ptr(), 1e-5, 70, 256, 1, y.data_ptr(), None, None, None,
                                               torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert st == 0 and torch.equal(y, want["y"])


def test_no_rows():
    import transformer_xl_relative_rel_gb300 as txl
    p = _inputs(0, 64, BF, 12)
    y, mean, rstd = txl.layer_norm_fwd(p["x"], p["gamma"], p["beta"])
    assert y.shape == (0, 64) and mean.shape == rstd.shape == (0,)
    grads = dict(dgamma=torch.full((64,), 7.0, device="cuda"), dbeta=torch.full((64,), 7.0, device="cuda"))
    g = txl.layer_norm_bwd(p["dy"], p["x"], mean, rstd, gamma=p["gamma"], grads=grads)
    assert g["dgamma"] is grads["dgamma"] and not g["dgamma"].any() and not g["dbeta"].any() and g["dx"].shape == (0, 64)
    txl.check()


def test_shapes_of_more_dimensions():
    import transformer_xl_relative_rel_gb300 as txl
    p = _inputs(24, 48, F32, 13)
    want = _run(p)
    v = {n: p[n].view(2, 3, 4, 48) for n in ("x", "residual", "dy")}
    y, mean, rstd = txl.layer_norm_fwd(v["x"], p["gamma"], p["beta"], residual=v["residual"])
    assert mean.shape == rstd.shape == (2, 3, 4)
    g = txl.layer_norm_bwd(v["dy"], v["x"], mean, rstd, gamma=p["gamma"], residual=v["residual"])
    assert g["dx"].shape == y.shape == (2, 3, 4, 48)
    assert torch.equal(y.view(24, 48), want["y"]) and torch.equal(g["dx"].view(24, 48), want["dx"])
    one = txl.layer_norm_fwd(p["x"][5], p["gamma"], p["beta"], residual=p["residual"][5])
    assert one[1].shape == () and torch.equal(one[0], want["y"][5])


def test_offsets_past_32_bits():
    import transformer_xl_relative_rel_gb300 as txl
    rows, d = 2 ** 31 // 1024 + 1000, 1024
    x = torch.zeros(rows, d, dtype=BF, device="cuda")
    p = _inputs(999, d, BF, 14)
    x[-999:] = p["x"]
    dy = torch.zeros_like(x)
    dy[-999:] = p["dy"]
    y, mean, rstd = txl.layer_norm_fwd(x, p["gamma"], p["beta"])
    g = txl.layer_norm_bwd(dy, x, mean, rstd, gamma=p["gamma"])
    want, tol = norm_reference(p["x"], p["gamma"], p["beta"], 1e-5, dy=p["dy"])
    got = dict(y=y[-999:], mean=mean[-999:], rstd=rstd[-999:], dx=g["dx"][-999:], dgamma=g["dgamma"], dbeta=g["dbeta"])
    check(got, want, tol)
    assert torch.equal(y[12345], p["beta"].to(BF)) and not g["dx"][:-999].any()


def test_captured_and_replayed():
    import transformer_xl_relative_rel_gb300 as txl
    ps = [_inputs(500, 512, BF, 15), _inputs(77, 90, F32, 16)]
    ws = [torch.empty(txl.layer_norm_bwd_workspace_bytes(*p["x"].shape, c), dtype=torch.uint8, device="cuda")
          for p, c in zip(ps, (txl.TXL_BF16, txl.TXL_F32))]
    torch.cuda.synchronize()
    outs, graphs = [], []
    for p, w in zip(ps, ws):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(_run(p, keep=True, dsum=True, workspace=w))
        graphs.append(g)
    for seed in (17, 18):
        for p in ps:
            q = _inputs(*p["x"].shape, p["x"].dtype, seed)
            for n in p:
                p[n].copy_(q[n])
        for g in graphs + graphs:
            g.replay()
        torch.cuda.synchronize()
        for p, out in zip(ps, outs):
            _check(p, keep=True, dsum=True, got=out)


def test_streams_and_host_threads_at_once():
    import threading
    ps = [_inputs(3000, 512, BF, 20), _inputs(500, 90, F32, 21), _inputs(900, 2048, BF, 22)]
    want = [_run(p) for p in ps]
    torch.cuda.synchronize()
    wrong = []

    def work(x):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(20):
                got = _run(ps[x])
            s.synchronize()
        wrong.extend((x, n) for n in got if not torch.equal(got[n], want[x][n]))

    threads = [threading.Thread(target=work, args=(x,)) for x in range(len(ps))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong, wrong


def test_calls_back_to_back_in_one_workspace():
    import transformer_xl_relative_rel_gb300 as txl
    ps = [_inputs(r, d, BF, r) for r, d in [(5, 72), (5000, 512), (33, 4000), (900, 1024), (700, 41)]]
    size = max(txl.layer_norm_bwd_workspace_bytes(*p["x"].shape, txl.TXL_BF16) for p in ps)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    want = [_run(p) for p in ps]
    torch.cuda.synchronize()
    order = [0, 1, 2, 3, 4, 3, 1, 4, 0, 2] * 3
    got = [_run(ps[k], workspace=ws) for k in order]
    torch.cuda.synchronize()
    for k, x in zip(order, got):
        for n in x:
            assert torch.equal(x[n], want[k][n]), n


def test_gradients_match_differences_of_the_forward():
    """fp32: (L(x + e) - L(x - e)) / 2e along random directions."""
    import transformer_xl_relative_rel_gb300 as txl
    p = _inputs(50, 40, F32, 23)
    grads = _run(p)
    g = torch.Generator(device="cuda").manual_seed(2)

    def value(q):
        y, _, _ = txl.layer_norm_fwd(q["x"], q["gamma"], q["beta"], residual=q["residual"])
        return float((y.double() * q["dy"].double()).sum())

    for name, grad in (("x", "dx"), ("residual", "dx"), ("gamma", "dgamma"), ("beta", "dbeta")):
        e = torch.randn(p[name].shape, device="cuda", generator=g)
        e /= e.norm()
        eps = 1e-2
        up, down = dict(p), dict(p)
        up[name], down[name] = p[name] + eps * e, p[name] - eps * e
        num = (value(up) - value(down)) / (2 * eps)
        ana = float((grads[grad].double() * e.double()).sum())
        # values of 2000 terms of a few units, each 2^-19 off, over eps; eps^2 times a third derivative of a few units
        assert abs(num - ana) <= 2000 ** 0.5 * 8 * 2.0 ** -19 / eps + 50 * eps ** 2, (name, num, ana)


def test_oracle():
    import numpy as np
    import oracle
    p = _inputs(40, 30, F32, 24)
    got = _run(p, dsum=True)
    f = lambda n: p[n].double().cpu().numpy()
    y, mean, rstd, g = oracle.layer_norm(f("x") + f("residual"), f("gamma"), f("beta"), 1e-5, f("dy"), f("dsum"))
    for n, want in dict(y=y, mean=mean, rstd=rstd, **g).items():
        assert np.abs(got[n].cpu().numpy() - want).max() <= 1e-4 * (1 + np.abs(want).max()), n
