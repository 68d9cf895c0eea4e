"""What the embedding, layer norm and optimiser step refuse, on the host: the C
entry points reject bad arguments before anything is launched, and the binding
rejects wrong shapes, types and devices.  No compute call is made."""
import ctypes
import itertools
import random

import pytest
import torch

import transformer_xl_relative_rel_gb300 as txl
from transformer_xl_relative_rel_gb300 import abi

OK, INVALID, UNSUPPORTED, CUDA = 0, 1, 2, 3
FAKE = 1 << 24     # 256-byte aligned, never dereferenced
FAR = 2 ** 32 + 5
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def lib():
    from transformer_xl_relative_rel_gb300 import _build
    _build.build()
    return abi.load_library()


def _no_gpu():
    return not torch.cuda.is_available()


# ------------------------------------------------------------------ embedding

def _embed(backward, **kw):
    a = dict(tokens=FAKE, x=FAKE * 2, scale=1.0, rows=10, d=16, vocab=100, dt=1, acc=0, out=FAKE * 3, ws=FAKE * 4,
             nws=1 << 20)
    a.update(kw)
    f = abi.load_library()
    head = (a["tokens"], a["x"], a["scale"], a["rows"], a["d"], a["vocab"], a["dt"])
    if backward:
        return f.txl_embed_bwd(*head, a["acc"], a["out"], a["ws"], a["nws"], None)
    return f.txl_embed_fwd(*head, a["out"], None)


@pytest.mark.parametrize("backward", [False, True])
def test_embed_bad_arguments(backward):
    c = lambda **kw: _embed(backward, **kw)
    assert c(dt=7) == UNSUPPORTED
    for bad in (dict(rows=-1), dict(d=0), dict(vocab=0), dict(vocab=-3)):
        assert c(**bad) == INVALID
    assert c(rows=(1 << 30) + 1) == UNSUPPORTED
    assert c(vocab=(1 << 30) + 1) == UNSUPPORTED
    assert c(d=(1 << 24) + 1) == UNSUPPORTED
    assert c(d=1 << 20, vocab=(1 << 20) + 1) == UNSUPPORTED
    assert c(d=1 << 20, rows=(1 << 20) + 1) == UNSUPPORTED
    for name in ("tokens", "x", "out"):
        assert c(**{name: None}) == INVALID, name
    assert c(tokens=FAKE + 4) == INVALID
    assert c(x=FAKE * 2 + 1) == INVALID
    assert c(x=FAKE * 2 + 2, dt=0) == INVALID
    assert c(out=FAKE * 3 + 1) == INVALID
    assert c(out=FAKE) == INVALID                   # overlaps the tokens
    assert c(out=FAKE * 2 + 32) == INVALID          # overlaps the other input
    if backward:
        assert c(ws=None) == INVALID
        assert c(nws=256) == INVALID
        assert c(ws=FAKE * 4 + 64) == INVALID
        assert c(ws=FAKE * 3 + 256) == INVALID      # overlaps dtable
        assert c(ws=FAKE * 2 - 256) == INVALID      # runs into dout


def test_embed_nothing_to_do():
    assert _embed(False, rows=0, tokens=None, x=None, out=None) == OK
    assert _embed(True, rows=0, tokens=None, x=None, ws=None, nws=0, acc=1, out=None) == OK
    assert _embed(True, rows=0, tokens=None, x=None, ws=None, nws=0, acc=0, out=None) == INVALID   # dtable is set to 0
    if _no_gpu():
        assert _embed(False) == CUDA and _embed(True) == CUDA and _embed(True, acc=1) == CUDA
        assert _embed(True, rows=0, tokens=None, x=None, ws=None, nws=0) == CUDA


def test_embed_workspace_queries():
    rng = random.Random(3)
    edge = [1, 2, 31, 32, 33, 255, 256, 257, 511, 512, 1023, 1024, 1025, 1 << 18, 1 << 20, 1 << 30]
    for dt, rows in itertools.product((0, 1), (0, 1, 5)):
        assert txl.embed_bwd_workspace_bytes(rows, 8, 9, dt) > 0
    for _ in range(1000):
        pick = lambda most: min(most, rng.choice(edge) if rng.random() < 0.4 else int(2 ** rng.uniform(0, 30)))
        d = pick(1 << 14)
        rows, vocab = pick((1 << 40) // d), pick((1 << 40) // d)
        # the sorted rows and tokens, and partial sums of every 16 rows
        assert txl.embed_bwd_workspace_bytes(rows, d, vocab, rng.choice((0, 1))) >= 8 * rows + rows // 16 * 8 * d
    f = abi.load_library()
    n = ctypes.c_size_t(0)
    assert f.txl_embed_bwd_workspace(10, 8, 9, 1, None) == INVALID
    assert f.txl_embed_bwd_workspace(-1, 8, 9, 1, ctypes.byref(n)) == INVALID
    assert f.txl_embed_bwd_workspace(10, 8, 9, 5, ctypes.byref(n)) == UNSUPPORTED
    with pytest.raises(txl.TxlError, match="unsupported"):
        txl.embed_bwd_workspace_bytes(FAR, 8, 9, 1)


def test_embed_binding_checks():
    tok, table, dout = torch.zeros(6, dtype=torch.int64), torch.zeros(9, 16, dtype=BF), torch.zeros(6, 16, dtype=BF)
    with pytest.raises(ValueError, match="contiguous CUDA tensors"):
        txl.embed_fwd(tok, table)
    with pytest.raises(ValueError, match="contiguous CUDA tensors"):
        txl.embed_bwd(tok, dout, vocab=9)
    with pytest.raises(TypeError, match="tokens must be"):
        txl.embed_fwd(tok.int(), table)
    with pytest.raises(TypeError, match="unsupported dtype"):
        txl.embed_fwd(tok, table.half())
    with pytest.raises(ValueError, match="table must be"):
        txl.embed_fwd(tok, table[0])
    with pytest.raises(ValueError, match="out must be"):
        txl.embed_fwd(tok, table, out=dout[:5])
    with pytest.raises(TypeError, match="out must be"):
        txl.embed_fwd(tok, table, out=dout.float())
    with pytest.raises(ValueError, match="tokens must be"):
        txl.embed_bwd(tok[:5], dout, vocab=9)
    with pytest.raises(ValueError, match="vocab is required"):
        txl.embed_bwd(tok, dout)
    with pytest.raises(ValueError, match="vocab is required"):
        txl.embed_bwd(tok, dout, vocab=9, accumulate=True)
    with pytest.raises(ValueError, match="dtable must be"):
        txl.embed_bwd(tok, dout, table[:, :8])
    with pytest.raises(ValueError, match="dtable must be"):
        txl.embed_bwd(tok, dout, table, vocab=8)
    with pytest.raises(TypeError, match="dtable must be"):
        txl.embed_bwd(tok, dout, table.float())
    with pytest.raises(ValueError, match="dout must be"):
        txl.embed_bwd(tok[0], dout[0, 0], vocab=9)
    meta = dict(device="meta")
    for rows, vocab, d in ((FAR, 8, 8), (8, FAR, 8), (8, 8, FAR)):
        t, w = torch.empty(rows, dtype=torch.int64, **meta), torch.empty(vocab, d, dtype=BF, **meta)
        with pytest.raises(txl.TxlError, match="unsupported"):
            txl.embed_fwd(t, w)
        with pytest.raises(txl.TxlError, match="unsupported"):
            txl.embed_bwd(t, torch.empty(rows, d, dtype=BF, **meta), w)


# ------------------------------------------------------------------ layer norm

def _norm(backward, **kw):
    a = dict(dy=FAKE, x=FAKE * 2, residual=FAKE * 3, dsum=FAKE * 4, gamma=FAKE * 5, beta=FAKE * 6, eps=1e-5, rows=10,
             d=16, dt=1, out=FAKE * 7, sum=FAKE * 8, mean=FAKE * 9, rstd=FAKE * 10, dgamma=FAKE * 11, dbeta=FAKE * 12,
             ws=FAKE * 13, nws=1 << 20)
    a.update(kw)
    f = abi.load_library()
    if backward:
        return f.txl_layer_norm_bwd(a["dy"], a["x"], a["residual"], a["dsum"], a["gamma"], a["mean"], a["rstd"], a["rows"],
                                    a["d"], a["dt"], a["out"], a["dgamma"], a["dbeta"], a["ws"], a["nws"], None)
    return f.txl_layer_norm_fwd(a["x"], a["residual"], a["gamma"], a["beta"], a["eps"], a["rows"], a["d"], a["dt"],
                                a["out"], a["sum"], a["mean"], a["rstd"], None)


@pytest.mark.parametrize("backward", [False, True])
def test_norm_bad_arguments(backward):
    c = lambda **kw: _norm(backward, **kw)
    assert c(dt=7) == UNSUPPORTED
    assert c(rows=-1) == INVALID
    assert c(d=0) == INVALID
    assert c(rows=(1 << 30) + 1) == UNSUPPORTED
    assert c(d=8193) == UNSUPPORTED
    for name in ("x", "out") + (("dy", "mean", "rstd") if backward else ()):
        assert c(**{name: None}) == INVALID, name
    assert c(x=FAKE * 2 + 1) == INVALID
    assert c(residual=FAKE * 3 + 2, dt=0) == INVALID
    assert c(gamma=FAKE * 5 + 2) == INVALID
    assert c(mean=FAKE * 9 + 2) == INVALID
    assert c(out=FAKE * 2) == INVALID                   # overlaps x
    assert c(out=FAKE * 3 + 64) == INVALID              # overlaps the residual
    if backward:
        assert c(dgamma=FAKE * 12 + 32) == INVALID      # overlaps dbeta
        assert c(dbeta=FAKE * 5) == INVALID             # overlaps gamma
        assert c(out=FAKE * 4) == INVALID               # overlaps dsum
        assert c(ws=None) == INVALID
        assert c(nws=16) == INVALID
        assert c(ws=FAKE * 13 + 4) == INVALID
        assert c(ws=FAKE * 11 - 256) == INVALID         # runs into dgamma
    else:
        for eps in (0.0, -1.0, float("nan"), float("inf"), 1e-60):
            assert c(eps=eps) == INVALID
        assert c(rstd=None) == INVALID and c(mean=None) == INVALID      # both or neither
        assert c(sum=FAKE * 7 + 32) == INVALID          # overlaps y
        assert c(sum=FAKE * 2) == INVALID               # overlaps x
        assert c(mean=FAKE * 10 + 8) == INVALID         # overlaps rstd


def test_norm_nothing_to_do():
    none = dict(rows=0, x=None, residual=None, out=None, mean=None, rstd=None)
    assert _norm(False, sum=None, gamma=None, beta=None, **none) == OK
    assert _norm(True, dy=None, dsum=None, ws=None, nws=0, dgamma=None, dbeta=None, **none) == OK
    if _no_gpu():
        assert _norm(False) == CUDA and _norm(True) == CUDA
        assert _norm(False, residual=None, gamma=None, beta=None, sum=None, mean=None, rstd=None) == CUDA
        assert _norm(True, ws=None, nws=0, dgamma=None, dbeta=None) == CUDA          # no workspace without them
        assert _norm(True, dy=None, dsum=None, ws=None, nws=0, **none) == CUDA       # dgamma and dbeta are set to 0


def test_norm_workspace_queries():
    for rows, d, dt in itertools.product((0, 1, 7, 3000, 1 << 30), (1, 410, 1024, 8192), (0, 1)):
        assert 0 < txl.layer_norm_bwd_workspace_bytes(rows, d, dt) <= 32 << 20
    with pytest.raises(txl.TxlError, match="unsupported"):
        txl.layer_norm_bwd_workspace_bytes(5, 8193, 1)
    with pytest.raises(txl.TxlError, match="unsupported"):
        txl.layer_norm_bwd_workspace_bytes(FAR, 8, 1)
    with pytest.raises(txl.TxlError, match="invalid"):
        txl.layer_norm_bwd_workspace_bytes(-1, 8, 1)
    assert abi.load_library().txl_layer_norm_bwd_workspace(1, 8, 1, None) == INVALID


def test_norm_binding_checks():
    x, f, g = torch.zeros(6, 16, dtype=BF), torch.zeros(6), torch.zeros(16)
    with pytest.raises(ValueError, match="contiguous CUDA tensors"):
        txl.layer_norm_fwd(x, g, g)
    with pytest.raises(ValueError, match="contiguous CUDA tensors"):
        txl.layer_norm_bwd(x, x, f, f)
    with pytest.raises(ValueError, match="x must be"):
        txl.layer_norm_fwd(x[0, 0])
    for bad, error in ((dict(residual=x[:5]), "residual"), (dict(gamma=g[:5]), "gamma"), (dict(beta=g[:5]), "beta"),
                       (dict(y=x[:5]), "y"), (dict(sum=x[:5]), "sum"), (dict(mean=f[:5]), "mean"),
                       (dict(rstd=f[:5]), "rstd")):
        with pytest.raises(ValueError, match=error + " must be"):
            txl.layer_norm_fwd(x, **bad)
    with pytest.raises(TypeError, match="gamma must be"):
        txl.layer_norm_fwd(x, g.to(BF))
    with pytest.raises(TypeError, match="residual must be"):
        txl.layer_norm_fwd(x, residual=x.float())
    with pytest.raises(TypeError, match="unsupported dtype"):
        txl.layer_norm_fwd(x.half())
    with pytest.raises(ValueError, match="dy must be"):
        txl.layer_norm_bwd(x[:5], x, f, f)
    with pytest.raises(ValueError, match="dsum must be"):
        txl.layer_norm_bwd(x, x, f, f, dsum=x[:5])
    with pytest.raises(ValueError, match="dgamma must be"):
        txl.layer_norm_bwd(x, x, f, f, grads=dict(dgamma=f))
    for shape in ((FAR, 8), (8, FAR)):
        m = torch.empty(*shape, dtype=BF, device="meta")
        with pytest.raises(txl.TxlError, match="unsupported"):
            txl.layer_norm_fwd(m)
        with pytest.raises(txl.TxlError, match="unsupported"):
            txl.layer_norm_bwd(m, m, m, m)


# ------------------------------------------------------------------ optimiser

def _tensors(n=2, at=None, **kw):
    """n bf16 tensors with masters and 8-bit moments; `at`: the one that kw changes."""
    t = (abi._AdamwTensor * max(n, 1))()
    for k in range(n):
        base = FAKE * (1 + 8 * k)
        a = dict(param=base, master=base + FAKE, grad=base + 2 * FAKE, exp_avg=base + 3 * FAKE, exp_avg_sq=base + 4 * FAKE,
                 exp_avg_scale=base + 5 * FAKE, exp_avg_sq_scale=base + 6 * FAKE, size=1000, weight_decay=0.1, param_dtype=1,
                 grad_dtype=1)
        if k == at or at is None:
            a.update(kw)
        for name, v in a.items():
            setattr(t[k], name, v)
    return t


def _step(t=None, n=2, **kw):
    o = abi._AdamwOptions()
    for name, v in dict(dict(lr=1e-3, eps=1e-8, beta1=0.9, beta2=0.999, step=1), **kw).items():
        setattr(o, name, v)
    return abi.load_library().txl_adamw_step(n, _tensors(n) if t is None else t, ctypes.byref(o), None)


def _grad_norm(t=None, n=2, max_norm=1.0, norm=FAKE * 40, clip=FAKE * 41, ws=FAKE * 42, nws=1 << 20):
    return abi.load_library().txl_grad_norm(n, _tensors(n) if t is None else t, max_norm, norm, clip, ws, nws, None)


def test_adamw_bad_arguments():
    one = lambda **kw: _step(_tensors(at=1, **kw))
    for name in ("param", "grad", "exp_avg", "exp_avg_sq", "exp_avg_scale", "exp_avg_sq_scale"):
        assert one(**{name: None}) == INVALID, name
    base = FAKE * 9
    for bad in (dict(param=base + 1), dict(master=base + FAKE + 2), dict(grad=base + 2 * FAKE + 1),
                dict(exp_avg_scale=base + 5 * FAKE + 2), dict(size=-1), dict(weight_decay=-0.1),
                dict(weight_decay=float("nan")), dict(weight_decay=float("inf")), dict(param_dtype=0),      # a master of fp32
                dict(exp_avg_scale=None, exp_avg_sq_scale=None, exp_avg=base + 3 * FAKE + 2)):
        assert one(**bad) == INVALID, bad
    assert one(param_dtype=3) == UNSUPPORTED and one(grad_dtype=-1) == UNSUPPORTED
    assert one(size=(1 << 40) + 1) == UNSUPPORTED
    assert abi.load_library().txl_adamw_step(1, None, ctypes.byref(abi._AdamwOptions()), None) == INVALID
    assert abi.load_library().txl_adamw_step(1, _tensors(1), None, None) == INVALID
    assert _step(n=-1) == INVALID
    for bad in (dict(beta1=1.0), dict(beta1=-0.1), dict(beta2=1.0), dict(beta2=float("nan")), dict(eps=0.0), dict(eps=-1.0),
                dict(eps=float("inf")), dict(step=0), dict(step=-1), dict(lr=-1.0), dict(lr=float("nan")),
                dict(lr=float("inf")), dict(lr_device=FAKE * 30 + 2), dict(step_device=FAKE * 30 + 4),
                dict(grad_scale=FAKE * 30 + 1)):
        assert _step(**bad) == INVALID, bad


def test_adamw_overlaps():
    names = ("param", "master", "exp_avg", "exp_avg_sq", "exp_avg_scale", "exp_avg_sq_scale")
    for name, other, first in itertools.product(names, names + ("grad",), (False, True)):
        # the last bytes of another buffer, in the same tensor and in the other one
        t = _tensors()
        width = dict(param=2, grad=2, master=4, exp_avg=1, exp_avg_sq=1)
        end = {n: 1000 * width[n] if n in width else 16 for n in names + ("grad",)}
        target = t[0] if first else t[1]
        if first and name == other:
            continue
        setattr(t[0], name, getattr(target, other) + end[other] - 4)
        assert _step(t) == INVALID, (name, other, first)
    t = _tensors()
    t[0].grad = t[1].grad                   # gradients are only read
    if _no_gpu():
        assert _step(t) == CUDA
    assert _step(lr_device=FAKE * 9 + FAKE) == INVALID
    assert _step(grad_scale=FAKE * 9) == INVALID
    assert _step(step_device=FAKE * 1 + 8) == INVALID


def test_adamw_nothing_to_do():
    none = dict(param=None, master=None, grad=None, exp_avg=None, exp_avg_sq=None, exp_avg_scale=None,
                exp_avg_sq_scale=None)
    assert _step(_tensors(2, size=0, **none)) == OK
    assert abi.load_library().txl_adamw_step(0, None, ctypes.byref(abi._AdamwOptions()), None) == INVALID     # betas, eps
    assert _step(n=0) == OK
    if _no_gpu():
        assert _step() == CUDA
        assert _step(_tensors(500), n=500) == CUDA
        assert _step(lr_device=FAKE * 30, step_device=FAKE * 31, grad_scale=FAKE * 32, lr=-1.0, step=0) == CUDA
        assert _step(_tensors(at=1, size=0, **none)) == CUDA


def test_grad_norm_arguments():
    assert _grad_norm(max_norm=0.0) == INVALID and _grad_norm(max_norm=float("nan")) == INVALID
    assert _grad_norm(max_norm=-1.0) == INVALID
    assert _grad_norm(ws=None) == INVALID and _grad_norm(nws=0) == INVALID and _grad_norm(ws=FAKE * 42 + 128) == INVALID
    assert _grad_norm(norm=FAKE * 40 + 2) == INVALID
    assert _grad_norm(clip=FAKE * 40) == INVALID                     # overlaps norm
    assert _grad_norm(norm=FAKE * 3) == INVALID                      # overlaps a gradient
    assert _grad_norm(_tensors(grad=FAKE * 50 + 1)) == INVALID
    assert _grad_norm(_tensors(at=0, grad=None)) == INVALID
    assert _grad_norm(_tensors(at=0, size=-5)) == INVALID
    assert _grad_norm(_tensors(at=0, grad_dtype=9)) == UNSUPPORTED
    assert _grad_norm(norm=None, clip=None) == OK
    assert _grad_norm(n=-1) == INVALID
    n = ctypes.c_size_t(0)
    f = abi.load_library()
    assert f.txl_grad_norm_workspace(2, _tensors(), None) == INVALID
    assert f.txl_grad_norm_workspace(-2, _tensors(), ctypes.byref(n)) == INVALID
    assert f.txl_grad_norm_workspace(0, None, ctypes.byref(n)) == OK and n.value > 0
    assert f.txl_grad_norm_workspace(2, _tensors(), ctypes.byref(n)) == OK and 0 < n.value <= 4096
    # only gradients are looked at
    assert f.txl_grad_norm_workspace(2, _tensors(param=None, exp_avg=None), ctypes.byref(n)) == OK
    if _no_gpu():
        assert _grad_norm() == CUDA and _grad_norm(norm=None) == CUDA and _grad_norm(clip=None) == CUDA
        assert _grad_norm(n=0, t=_tensors(1), ws=None, nws=0) == CUDA          # the norm of nothing is written
        assert _grad_norm(_tensors(param=None, exp_avg=None)) == CUDA


def test_adamw_binding_checks():
    e4m3 = torch.float8_e4m3fn
    p, m = torch.zeros(300, dtype=BF), torch.zeros(300)
    c, s = torch.zeros(300, dtype=e4m3), torch.zeros(2)
    T = txl.AdamwTensors
    with pytest.raises(ValueError, match="contiguous CUDA tensors"):
        T([p], [p], [m], [m])
    with pytest.raises(ValueError, match="entry per param"):
        T([p], [p, p], [m], [m])
    with pytest.raises(ValueError, match="entry per param"):
        T([p], [p], [m], [m], weight_decay=[0.1, 0.2])
    for args in (([p], [p[:5]], [m], [m]), ([p], [p], [m[:5]], [m]), ([p], [p], [m], [m[:5]])):
        with pytest.raises(ValueError, match="must be"):
            T(*args)
    with pytest.raises(ValueError, match="must be"):
        T([p], [p], [m], [m], masters=[m[:5]])
    with pytest.raises(TypeError, match="master"):
        T([m], [p], [m], [m], masters=[m])
    with pytest.raises(TypeError, match="master"):
        T([p], [p], [m], [m], masters=[p])
    with pytest.raises(TypeError, match="moments"):
        T([p], [p], [c], [c])
    with pytest.raises(TypeError, match="moments"):
        T([p], [p], [m], [m], exp_avg_scales=[s], exp_avg_sq_scales=[s])
    with pytest.raises(TypeError, match="moments"):
        T([p], [p], [c], [c], exp_avg_scales=[s])
    with pytest.raises(ValueError, match="scales"):
        T([p], [p], [c], [c], exp_avg_scales=[s], exp_avg_sq_scales=[torch.zeros(1)])
    with pytest.raises(TypeError, match="unsupported dtype"):
        T([p.half()], [p], [m], [m])
    with pytest.raises(TypeError, match="AdamwTensors"):
        txl.adamw_step([p], 1e-3, 1)
    with pytest.raises(TypeError, match="AdamwTensors"):
        txl.grad_norm([p], 1.0)
