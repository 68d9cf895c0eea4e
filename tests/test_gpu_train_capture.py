"""Captures of the embedding's, norm's and optimiser's calls among other work:
behind memory sets and copies, and on streams that leave and join the capture."""
import pytest
import torch

import transformer_xl_relative_rel_gb300 as txl
from tests.train_helpers import BF, F32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from transformer_xl_relative_rel_gb300 import _build
    _build.build()


def _inputs():
    g = torch.Generator(device="cuda").manual_seed(3)
    n = lambda *s: torch.randn(*s, device="cuda", generator=g)
    p = dict(tok=torch.randint(-1, 90, (700,), device="cuda", generator=g), table=n(90, 64).to(BF), dout=n(700, 64).to(BF),
             gamma=1 + 0.1 * n(64), w=n(5000), g=n(5000))
    p["none"], p["empty"] = torch.empty(0, dtype=torch.int64, device="cuda"), torch.empty(0, 64, dtype=BF, device="cuda")
    return p


def _weights(p):
    w = [p["w"].clone(), torch.zeros(5000, device="cuda"), torch.zeros(5000, device="cuda")]
    return w, txl.AdamwTensors([w[0]], [p["g"]], [w[1]], [w[2]])


def test_behind_memory_sets_and_copies():
    """A call of no rows sets its outputs by a memory set; the next call's
    kernels, a copy and others follow it."""
    p = _inputs()
    (w, t), (w2, t2) = _weights(p), _weights(p)

    def calls(w, t):
        table = txl.embed_bwd(p["none"], p["empty"], vocab=90)
        table2 = txl.embed_bwd(p["tok"], p["dout"], table.clone(), accumulate=True)
        stat = torch.empty(0, device="cuda")
        first = txl.layer_norm_bwd(p["empty"], p["empty"], stat, stat, gamma=p["gamma"])
        y, mean, rstd = txl.layer_norm_fwd(p["dout"], p["gamma"], first["dbeta"])
        kept = torch.empty_like(y)
        kept.copy_(y)
        g = txl.layer_norm_bwd(kept, p["dout"], mean, rstd, gamma=p["gamma"])
        first = txl.embed_bwd(p["none"], p["empty"], vocab=90)
        txl.adamw_step(t, 1e-2, 1, grad_scale=txl.grad_norm(t, 0.1)[1])
        return [table, table2, y, mean, rstd, g["dx"], g["dgamma"], g["dbeta"], first] + w

    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = calls(w, t)
    graph.replay()
    torch.cuda.synchronize()
    for k, (x, y) in enumerate(zip(got, calls(w2, t2))):
        assert torch.equal(x, y), k
    txl.check()


def test_streams_that_leave_and_join_a_capture():
    p = _inputs()
    (w, t), (w2, t2) = _weights(p), _weights(p)
    side = torch.cuda.Stream()

    def calls(w, t, fork):
        x = txl.embed_fwd(p["tok"], p["table"], 3.0)
        main = torch.cuda.current_stream()
        if fork:
            side.wait_stream(main)
        with torch.cuda.stream(side if fork else main):
            y, mean, rstd = txl.layer_norm_fwd(x, p["gamma"], residual=p["dout"])
            norm, clip = txl.grad_norm(t, 0.1)
        dtable = txl.embed_bwd(p["tok"], x, vocab=90)
        if fork:
            main.wait_stream(side)
        g = txl.layer_norm_bwd(y, x, mean, rstd, gamma=p["gamma"], residual=p["dout"])
        txl.embed_bwd(p["tok"], g["dx"], dtable, accumulate=True)
        txl.adamw_step(t, 1e-2, 1, grad_scale=clip)
        return [x, y, mean, rstd, norm, clip, dtable, g["dx"], g["dgamma"], g["dbeta"]] + w

    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = calls(w, t, True)
    graph.replay()
    torch.cuda.synchronize()
    for k, (x, y) in enumerate(zip(got, calls(w2, t2, False))):
        assert torch.equal(x, y), k
    txl.check()
