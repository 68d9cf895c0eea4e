"""Layer norm's backward called at once by host threads, and captured, in forms
that share a kernel and take different amounts of shared memory (x alone, with
a residual, with the kept sum's gradient): the kernel's limit is the device's,
not the call's."""
import threading

import pytest
import torch

import transformer_xl_relative_rel_gb300 as txl
from transformer_xl_relative_rel_gb300 import abi
from tests.train_helpers import BF, F32

pytestmark = pytest.mark.gpu

# (residual, dsum)
FORMS = [(False, False), (True, False), (False, True), (True, True)]
WIDTHS = [(BF, 256), (BF, 512), (BF, 1024), (BF, 410), (F32, 256), (F32, 512), (F32, 1024), (F32, 771)]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from transformer_xl_relative_rel_gb300 import _build
    _build.build()


def _inputs(rows, d, dtype):
    g = torch.Generator(device="cuda").manual_seed(d)
    n = lambda *s: torch.randn(*s, device="cuda", generator=g)
    p = dict(x=n(rows, d).to(dtype), residual=n(rows, d).to(dtype), dy=n(rows, d).to(dtype), dsum=n(rows, d).to(dtype),
             gamma=1 + 0.3 * n(d))
    p["stats"] = {r: txl.layer_norm_fwd(p["x"], p["gamma"], residual=p["residual"] if r else None)[1:] for r in (False, True)}
    torch.cuda.synchronize()
    return p


def _backward(p, form, **kw):
    residual, dsum = form
    return txl.layer_norm_bwd(p["dy"], p["x"], *p["stats"][residual], gamma=p["gamma"],
                              residual=p["residual"] if residual else None, dsum=p["dsum"] if dsum else None, **kw)


@pytest.mark.parametrize("dtype,d", WIDTHS)
def test_forms_of_one_width_at_once(dtype, d):
    """The library's entry in tight loops (the interpreter is let go of during
    a call), then the binding's."""
    p = _inputs(40, d, dtype)
    want = {f: _backward(p, f) for f in FORMS}
    entry, code = abi.load_library().txl_layer_norm_bwd, txl.TXL_BF16 if dtype == BF else txl.TXL_F32
    size = txl.layer_norm_bwd_workspace_bytes(40, d, code)
    torch.cuda.synchronize()
    failed, start = [], threading.Barrier(len(FORMS))

    def work(form):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                got = {n: torch.full_like(x, float("nan")) for n, x in want[form].items()}
                ws = torch.empty(size, dtype=torch.uint8, device="cuda")
                s.synchronize()
                args = (p["dy"].data_ptr(), p["x"].data_ptr(), p["residual"].data_ptr() if form[0] else None,
                        p["dsum"].data_ptr() if form[1] else None, p["gamma"].data_ptr(),
                        *(t.data_ptr() for t in p["stats"][form[0]]), 40, d, code, got["dx"].data_ptr(),
                        got["dgamma"].data_ptr(), got["dbeta"].data_ptr(), ws.data_ptr(), size, s.cuda_stream)
                start.wait()
                states = {entry(*args) for _ in range(4000)}
                s.synchronize()
                failed.extend((form, st) for st in states if st != 0)
                got = [got] + [_backward(p, form) for _ in range(100)]
                s.synchronize()
            failed.extend((form, name) for g in got for name in g if not torch.equal(g[name], want[form][name]))
        except Exception as e:      # an error of a thread is the test's
            failed.append((form, repr(e)))

    threads = [threading.Thread(target=work, args=(f,)) for f in FORMS]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed[:5]
    txl.check()


@pytest.mark.parametrize("dtype,d", WIDTHS)
def test_forms_of_one_width_in_a_graph(dtype, d):
    """Instantiated and replayed after each form was the last one to be called."""
    p = _inputs(40, d, dtype)
    want = {f: _backward(p, f) for f in FORMS}
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = {f: _backward(p, f) for f in FORMS + FORMS[::-1]}
    for last in FORMS:
        _backward(p, last)
        for g in got.values():
            for x in g.values():
                x.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        for f in FORMS:
            assert all(torch.equal(got[f][n], want[f][n]) for n in want[f]), (last, f)
    txl.check()
