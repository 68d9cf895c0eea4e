"""What the output-layer losses refuse, on the host: the C entry points reject
bad arguments before anything is launched, and the binding rejects wrong
shapes, types and devices.  No compute call is made."""
import ctypes

import pytest
import torch

import transformer_xl_relative_rel_gb300 as txl
from transformer_xl_relative_rel_gb300 import abi

OK, INVALID, UNSUPPORTED, CUDA = 0, 1, 2, 3
FAKE = 1 << 24     # 256-byte aligned, never dereferenced


@pytest.fixture(scope="module", autouse=True)
def lib():
    from transformer_xl_relative_rel_gb300 import _build
    _build.build()
    return abi.load_library()


def _ws(rows=10, d=16, vocab=100, k=None, dt=1, backward=0):
    n = ctypes.c_size_t(0)
    f = abi.load_library()
    st = f.txl_softmax_xent_workspace(rows, d, vocab, dt, backward, ctypes.byref(n)) if k is None else \
        f.txl_distill_workspace(rows, d, vocab, k, dt, backward, ctypes.byref(n))
    return st, n.value


def _call(op, backward, **kw):
    a = dict(h=FAKE, w=FAKE * 2, bias=FAKE * 3, idx=FAKE * 4, y=FAKE * 5, ydt=0, t=2.0, lse=FAKE * 6, dloss=FAKE * 7,
             rows=10, d=16, vocab=100, k=4, dt=1, loss=FAKE * 8, lse_out=FAKE * 9, dh=FAKE * 10, dw=FAKE * 11,
             db=FAKE * 12, ws=FAKE * 13, nws=1 << 23)
    a.update(kw)
    f = abi.load_library()
    head = [a["h"], a["w"], a["bias"], a["idx"]]
    mid, size = [], [a["rows"], a["d"], a["vocab"], a["dt"]]
    if op == "distill":
        mid, size = [a["y"], a["ydt"], a["t"]], [a["rows"], a["d"], a["vocab"], a["k"], a["dt"]]
    tail = [a["ws"], a["nws"], None]
    if backward:
        fn = f.txl_distill_bwd if op == "distill" else f.txl_softmax_xent_bwd
        return fn(*head, *mid, a["lse"], a["dloss"], *size, a["dh"], a["dw"], a["db"], *tail)
    fn = f.txl_distill_fwd if op == "distill" else f.txl_softmax_xent_fwd
    return fn(*head, *mid, *size, a["loss"], a["lse_out"], *tail)


BOTH = [(op, b) for op in ("xent", "distill") for b in (False, True)]


@pytest.mark.parametrize("op,backward", BOTH)
def test_bad_arguments(op, backward):
    c = lambda **kw: _call(op, backward, **kw)
    assert c(dt=7) == UNSUPPORTED
    assert c(rows=-1) == INVALID
    assert c(d=0) == INVALID
    assert c(vocab=0) == INVALID
    assert c(vocab=(1 << 30) + 1, nws=1 << 60) == UNSUPPORTED
    assert c(rows=(1 << 30) + 1) == UNSUPPORTED
    assert c(d=2 ** 31 - 1) == UNSUPPORTED
    assert c(d=1 << 20, vocab=(1 << 20) + 1, nws=1 << 60) == UNSUPPORTED
    for name in ("h", "w", "idx", "ws") + (("lse", "dloss") if backward else ("loss", "lse_out")):
        assert c(**{name: None}) == INVALID, name
    assert c(nws=256) == INVALID
    assert c(ws=FAKE * 13 + 64) == INVALID
    assert c(h=FAKE + 1) == INVALID
    assert c(h=FAKE + 2, dt=0) == INVALID
    assert c(bias=FAKE * 3 + 2) == INVALID
    assert c(idx=FAKE * 4 + 4) == INVALID
    assert c(ws=FAKE * 2 - 256) == INVALID                       # the workspace runs into w
    if backward:
        assert c(dh=FAKE * 10 + 1) == INVALID
        assert c(db=FAKE * 12 + 2) == INVALID
        assert c(dh=FAKE) == INVALID                             # dh overlaps h
        assert c(dw=FAKE * 10 + 32) == INVALID                   # dw overlaps dh
        assert c(db=FAKE * 6) == INVALID                         # db overlaps lse
        assert c(dh=None, dw=None, db=None) == OK                # nothing asked for
    else:
        assert c(loss=FAKE * 8 + 2) == INVALID
        assert c(loss=FAKE * 9 + 4) == INVALID                   # loss overlaps lse
        assert c(lse_out=FAKE * 2) == INVALID


@pytest.mark.parametrize("backward", [False, True])
def test_bad_teacher_arguments(backward):
    c = lambda **kw: _call("distill", backward, **kw)
    assert c(k=0) == INVALID
    assert c(k=257) == UNSUPPORTED
    assert c(ydt=5) == UNSUPPORTED
    assert c(y=None) == INVALID
    assert c(y=FAKE * 5 + 2) == INVALID
    for t in (0.0, -1.0, float("nan"), float("inf"), 1e-40):
        assert c(t=t) == INVALID


@pytest.mark.parametrize("op,backward", BOTH)
def test_no_rows_and_no_gpu(op, backward):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present: the call would launch on the fake pointers")
    assert _call(op, backward) == CUDA
    assert _call(op, backward, bias=None) == CUDA
    if backward:
        assert _call(op, backward, rows=0, dw=None, db=None, h=None, ws=None, nws=0) == OK
        assert _call(op, backward, rows=0, h=None, w=None, dh=None) == CUDA     # dw and db are set to zero
    else:
        assert _call(op, backward, rows=0, h=None, w=None, idx=None, y=None, loss=None, lse_out=None, ws=None,
                     nws=0) == OK


def test_workspace_queries():
    for k in (None, 4):
        st, n = _ws(k=k)
        assert st == OK and n > 0
        assert _ws(k=k, backward=1)[1] >= n                      # the backward's serves the forward too
        assert _ws(k=k, dt=7)[0] == UNSUPPORTED
        assert _ws(rows=-1, k=k)[0] == INVALID
        assert _ws(vocab=0, k=k)[0] == INVALID
        assert _ws(rows=0, k=k)[0] == OK
    assert _ws(k=0)[0] == INVALID
    assert _ws(k=257)[0] == UNSUPPORTED
    f = abi.load_library()
    assert f.txl_softmax_xent_workspace(1, 1, 1, 1, 0, None) == INVALID
    # far below the logits: 8192 x 262144 in bf16 would be 4 GB
    assert _ws(rows=8192, d=1024, vocab=262144, backward=1)[1] < 1 << 30
    with pytest.raises(txl.TxlError, match="invalid"):
        txl.softmax_xent_workspace_bytes(-1, 8, 8, txl.TXL_BF16)
    with pytest.raises(txl.TxlError, match="unsupported"):
        txl.distill_workspace_bytes(8, 8, 8, 300, txl.TXL_BF16)


def test_binding_checks():
    n, d, v, k = 6, 16, 40, 3
    h, w = torch.zeros(n, d, dtype=torch.bfloat16), torch.zeros(v, d, dtype=torch.bfloat16)
    y = torch.zeros(n, dtype=torch.int64)
    idx, t = torch.zeros(n, k, dtype=torch.int64), torch.zeros(n, k)
    f = torch.zeros(n)
    with pytest.raises(ValueError, match="w must be"):
        txl.softmax_xent_fwd(h, w[:, :8], y)
    with pytest.raises(ValueError, match="w must be"):
        txl.softmax_xent_fwd(h, w.float(), y)
    with pytest.raises(ValueError, match="target must be"):
        txl.softmax_xent_fwd(h, w, y[:-1])
    with pytest.raises(TypeError, match="target must be"):
        txl.softmax_xent_fwd(h, w, y.int())
    with pytest.raises(ValueError, match="bias must be"):
        txl.softmax_xent_fwd(h, w, y, bias=torch.zeros(v + 1))
    with pytest.raises(TypeError, match="bias must be"):
        txl.softmax_xent_fwd(h, w, y, bias=torch.zeros(v, dtype=torch.bfloat16))
    with pytest.raises(TypeError, match="unsupported dtype"):
        txl.softmax_xent_fwd(h.half(), w.half(), y)
    with pytest.raises(ValueError, match="contiguous CUDA tensors"):
        txl.softmax_xent_fwd(h, w, y)
    with pytest.raises(ValueError, match="dloss must be"):
        txl.softmax_xent_bwd(h, w, y, f, f[:1])
    with pytest.raises(TypeError, match="lse must be"):
        txl.softmax_xent_bwd(h, w, y, f.double(), f)
    with pytest.raises(ValueError, match="teacher_idx must be"):
        txl.distill_fwd(h, w, idx[:-1], t)
    with pytest.raises(ValueError, match="teacher_logits must be"):
        txl.distill_fwd(h, w, idx, t[:, :1])
    with pytest.raises(TypeError, match="teacher_logits must be"):
        txl.distill_fwd(h, w, idx, t.half())
    with pytest.raises(TypeError, match="teacher_idx must be"):
        txl.distill_bwd(h, w, idx.int(), t, f, f)
    with pytest.raises(ValueError, match="contiguous CUDA tensors"):
        txl.distill_bwd(h, w, idx, t, f, f)
