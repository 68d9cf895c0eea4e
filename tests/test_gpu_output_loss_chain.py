"""The output-layer losses on the GPU where calls, launches, items and pieces
follow one another: empty batches, calls of different inputs back to back in
one workspace, row blocks that end inside a warp's rows, vocabularies of one
strip and of several pieces, and masks of a type's lowest value.  Bounds as in
tests/loss_helpers.py."""
import os
import subprocess
import sys

import pytest
import torch

from tests.test_gpu_output_loss import (BF, F32, _check_distill, _check_xent, _distill, _inputs,  # noqa: F401
                                        _lib, _xent)

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("vocab", [257, 32768])
def test_no_rows_of_larger_vocabularies(vocab, dtype):
    import transformer_xl_relative_rel_gb300 as txl
    p = _inputs(0, 64, vocab, dtype, 3, k=3)
    for fn in (_xent, lambda q: _distill(q, 2.0)):
        grads = dict(dw=torch.full_like(p["w"], 7.0), db=torch.full_like(p["bias"], 7.0))
        g = fn(p)
        assert g["loss"].shape == g["lse"].shape == (0,) and g["dh"].shape == (0, 64)
        assert not g["dw"].any() and not g["db"].any()
    g = txl.softmax_xent_bwd(p["h"], p["w"], p["target"], p["dloss"], p["dloss"], bias=p["bias"], grads=grads)
    assert g["dw"] is grads["dw"] and not g["dw"].any() and not g["db"].any()
    txl.check()


@pytest.mark.parametrize("t", [0.25, 0.5, 1.0, 2.0])
@pytest.mark.parametrize("t_dtype", [F32, BF])
@pytest.mark.parametrize("dtype,rows,vocab", [(F32, 5, 300), (BF, 40, 300), (BF, 300, 200), (F32, 140, 150)])
def test_teacher_logits_of_the_lowest_value(dtype, rows, vocab, t_dtype, t):
    """A teacher's entries masked by the type's lowest value weigh nothing next
    to others and are alike where there are no others, at any temperature."""
    p = _inputs(rows, 64, vocab, dtype, 11, k=6, t_dtype=t_dtype)
    p["y"][4] = torch.finfo(t_dtype).min          # a whole row
    p["y"][0, 2:] = torch.finfo(t_dtype).min      # some of a row
    got = _distill(p, t)
    torch.cuda.synchronize()
    # p is 1/6 throughout: the float64 reference takes the same logits divided by t
    _check_distill(p, t, got=got)
    one = dict(p, y=p["y"].clone())
    one["y"][4] = 0.0
    want = _distill(one, t)
    for n in got:
        assert torch.equal(got[n], want[n]), n


@pytest.mark.parametrize("dtype,vocab", [(BF, 768), (BF, 740), (F32, 384), (F32, 361)])
def test_row_blocks_that_end_inside_a_warps_rows(dtype, vocab):
    """39 row blocks of 256, 10 rows in the last: of 117 tiles some pairs of
    CTAs take a whole block's and the last one's in turn, whose other warps
    have no rows and leave what is still being stored alone."""
    p = _inputs(38 * 256 + 10, 64, vocab, dtype, 13, k=5)
    for fn, ref in ((_xent, _check_xent), (lambda q: _distill(q, 2.0), lambda q, got: _check_distill(q, 2.0, got=got))):
        got = fn(p)
        ref(p, got=got)
        for _ in range(10):
            again = fn(p)
            for n in got:
                assert torch.equal(again[n], got[n]), n


# rows, d_model, vocabulary, teacher entries, type: a handful of rows (one block, a cluster, many
# blocks), one and several row blocks, lists of one and of many entries, copied weights and biases
BACK_TO_BACK = [(5, 72, 300, 4, F32), (3, 41, 4000, 9, BF), (8, 64, 20000, 1, F32), (40, 72, 1500, 5, BF),
                (300, 64, 3001, 64, BF), (700, 41, 900, 200, BF), (140, 48, 700, 7, F32), (1500, 128, 250, 33, BF)]


def _steps(ps, ws, outs):
    """A training step under each loss for each of ps, all in the workspace ws."""
    import transformer_xl_relative_rel_gb300 as txl
    for p, (a, b) in zip(ps, outs):
        kw = dict(bias=p["bias"], workspace=ws)
        txl.softmax_xent_fwd(p["h"], p["w"], p["target"], loss=a["loss"], lse=a["lse"], **kw)
        txl.distill_fwd(p["h"], p["w"], p["idx"], p["y"], 2.0, loss=b["loss"], lse=b["lse"], **kw)
        txl.softmax_xent_bwd(p["h"], p["w"], p["target"], a["lse"], p["dloss"], grads=a, **kw)
        txl.distill_bwd(p["h"], p["w"], p["idx"], p["y"], b["lse"], p["dloss"], 2.0, grads=b, **kw)


def _unaligned(x):
    """x, one element behind a 16-byte boundary."""
    flat = torch.empty(x.numel() + 8, dtype=x.dtype, device=x.device)
    y = flat[1:1 + x.numel()].view(x.shape)
    y.copy_(x)
    return y


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("shapes", [[s] * 6 for s in BACK_TO_BACK] + [BACK_TO_BACK + BACK_TO_BACK[::-1]])
def test_calls_back_to_back_in_one_workspace(shapes, graph):
    """Calls of different inputs one behind another with nothing in between:
    each gives what it gives alone in a workspace of its own."""
    import transformer_xl_relative_rel_gb300 as txl
    ps, size = [], 0
    for x, (rows, d, vocab, k, dtype) in enumerate(shapes):
        p = _inputs(rows, d, vocab, dtype, 100 + x, k=k)
        p["bias"] = _unaligned(p["bias"])         # a copy of it is made in the workspace
        ps.append(p)
        code = txl.TXL_BF16 if dtype == BF else txl.TXL_F32
        size = max(size, txl.distill_workspace_bytes(rows, d, vocab, k, code, backward=True))
    ws = torch.full((size // 4,), float("nan"), device="cuda")

    def outputs():
        f = lambda n: torch.full((n,), 7.0, device="cuda")
        return [[dict(loss=f(len(p["h"])), lse=f(len(p["h"])), dh=torch.full_like(p["h"], 7.0),
                      dw=torch.full_like(p["w"], 7.0), db=f(len(p["w"]))) for _ in range(2)] for p in ps]

    want = outputs()
    for p, pair in zip(ps, want):
        own = torch.full_like(ws, float("nan"))
        _steps([p], own, [pair])
        torch.cuda.synchronize()
    got = outputs()
    torch.cuda.synchronize()
    if graph:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            _steps(ps, ws, got)
        g.replay()
        torch.cuda.synchronize()
        got_again = outputs()
        for a, b in zip(got, got_again):
            for x, y in zip(a, b):
                for n in x:
                    x[n].copy_(y[n])
        g.replay()
        g.replay()
    else:
        _steps(ps, ws, got)
        _steps(ps, ws, got)
    torch.cuda.synchronize()
    txl.check()
    for x, (a, b) in enumerate(zip(got, want)):
        for one, other in zip(a, b):
            for n in one:
                assert torch.equal(one[n], other[n]), (x, n)


def _xent_forward_bytes(rows, d, vocab, dtype, slots):
    """The forward's workspace for operands copied whole and that many partial
    results per row: bias, h, w, the targets' logits, the partial results."""
    parts, dp = (3 if dtype == F32 else 1), (d + 7) // 8 * 8
    up = lambda n: (n + 255) // 256 * 256
    return up(4 * vocab) + up(rows * dp * parts * 2) + up(vocab * dp * parts * 2) + up(4 * rows) + up(8 * rows * slots)


@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("dtype,rows,d,vocab", [
    (BF, 16896, 64, 256), (BF, 20001, 64, 200), (BF, 40000, 40, 129), (BF, "1", 64, 1000), (BF, "2", 72, 997),
    (BF, 30000, 33, 65), (F32, 20001, 64, 128), (F32, 40000, 40, 100), (F32, "1", 24, 250), (F32, "3", 24, 250)])
def test_vocabularies_of_one_strip(dtype, rows, d, vocab, bias):
    """The cross entropy's product launch joins its two halves of a row itself:
    both with tokens, one tile and several, more row blocks than pairs of CTAs
    (a pair's second item takes over the place where halves are joined).  Rows
    as text: so many row blocks per pair, the last one ragged."""
    import transformer_xl_relative_rel_gb300 as txl
    if isinstance(rows, str):
        rows = int(rows) * (torch.cuda.get_device_properties(0).multi_processor_count // 2) * 256 - 35
    code = txl.TXL_BF16 if dtype == BF else txl.TXL_F32
    # two partial results per row: one strip
    assert txl.softmax_xent_workspace_bytes(rows, d, vocab, code) == _xent_forward_bytes(rows, d, vocab, dtype, 2)
    p = _inputs(rows, d, vocab, dtype, 17, bias=bias)
    p["target"][::7] = -1
    p["dloss"][5::11] = 0.0
    p["target"][3], p["target"][4], p["target"][rows - 1] = 0, vocab - 1, vocab - 1
    p["h"][::7] = 3.0     # (an empty row's lse is still computed)
    got = _xent(p)
    _check_xent(p, got=got)
    for _ in range(4):
        loss, lse = txl.softmax_xent_fwd(p["h"], p["w"], p["target"], bias=p["bias"])
        assert torch.equal(loss, got["loss"]) and torch.equal(lse, got["lse"])


@pytest.mark.parametrize("dtype,rows,d,vocab", [(F32, 20, 1024, 180003), (BF, 150, 1023, 540000), (F32, 300, 520, 380001)])
def test_forward_of_several_vocabulary_pieces(dtype, rows, d, vocab):
    """Weights that are copied, in pieces; targets and entries in each."""
    import transformer_xl_relative_rel_gb300 as txl
    code, parts = (txl.TXL_BF16, 1) if dtype == BF else (txl.TXL_F32, 3)
    assert txl.softmax_xent_workspace_bytes(rows, d, vocab, code) < vocab * d * parts * 2
    p = _inputs(rows, d, vocab, dtype, 19, k=16)
    from tests.loss_helpers import check, distill_reference, xent_reference
    loss, lse = txl.softmax_xent_fwd(p["h"], p["w"], p["target"], bias=p["bias"])
    check(dict(loss=loss, lse=lse), *xent_reference(p["h"], p["w"], p["bias"], p["target"]))
    loss, lse = txl.distill_fwd(p["h"], p["w"], p["idx"], p["y"], 2.0, bias=p["bias"])
    check(dict(loss=loss, lse=lse), *distill_reference(p["h"], p["w"], p["bias"], p["idx"], p["y"], 2.0))
    txl.check()


@pytest.mark.parametrize("dtype,rows,d,vocab", [(BF, 9000, 64, 70001), (BF, 9000, 41, 65000), (F32, 4000, 41, 50003)])
def test_backward_of_several_vocabulary_pieces(dtype, rows, d, vocab):
    """dz in pieces, dh added up over them; targets and entries in each."""
    import transformer_xl_relative_rel_gb300 as txl
    code, parts = (txl.TXL_BF16, 1) if dtype == BF else (txl.TXL_F32, 3)
    assert txl.distill_workspace_bytes(rows, d, vocab, 20, code, backward=True) < rows * vocab * parts * 2
    p = _inputs(rows, d, vocab, dtype, 23, k=20)
    _check_xent(p)
    _check_distill(p, 2.0)


def test_check_costs_what_the_program_uses():
    """txl_check reads the losses' error words only in a program that has
    called them: one that has not pays for three copies, not five (about
    11 us each)."""
    code = """
import time, torch
import transformer_xl_relative_rel_gb300 as txl
def cost():
    best = 1e9
    for _ in range(40):
        t = time.perf_counter()
        for _ in range(50):
            txl.check()
        best = min(best, (time.perf_counter() - t) / 50)
    return best
torch.zeros(1, device="cuda")
cost()
before = cost()
w = torch.zeros(300, 64, device="cuda")
for rows in (3, 200):
    txl.softmax_xent_fwd(torch.zeros(rows, 64, device="cuda"), w, torch.zeros(rows, dtype=torch.int64, device="cuda"))
after = cost()
print("COST", before * 1e6, after * 1e6)
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300, cwd=ROOT)
    assert r.returncode == 0, r.stderr
    before, after = map(float, r.stdout.split("COST")[1].split())
    # 3 / 5 of it, and a synchronisation that both have
    assert before < 0.8 * after, (before, after)


@pytest.mark.parametrize("dtype,rows", [(F32, 5), (BF, 40), (F32, 140), (BF, 300)])
def test_biases_of_the_lowest_value(dtype, rows):
    """They mask as -infinity does, to the bit: some tokens, a target among
    them, and the whole vocabulary."""
    p = _inputs(rows, 64, 130, dtype, 29, k=4)
    for masked in (torch.arange(130, device="cuda") % 3 == 1, torch.ones(130, dtype=torch.bool, device="cuda")):
        both = [dict(p, bias=torch.where(masked, torch.full_like(p["bias"], v), p["bias"]))
                for v in (torch.finfo(F32).min, -float("inf"))]
        a, b = (_xent(q) for q in both)
        for n in a:
            assert torch.equal(a[n], b[n]), n
        counted = (p["target"] >= 0) & (p["target"] < 130)
        lost = counted & masked[p["target"].clamp(0, 129)] & ~masked.all()
        assert (a["loss"][lost] == float("inf")).all() and torch.isfinite(a["loss"][~lost]).all()
        assert ((a["lse"] == -float("inf")) == masked.all()).all()
        if masked.all():
            assert not a["loss"].any() and not any(a[n].any() for n in ("dh", "dw", "db"))


def test_first_calls_of_a_process_captured():
    """No call has to come before a capture: kernels of every kind are first
    launched while a graph is recorded."""
    code = """
import torch
from tests.test_gpu_output_loss import BF, F32, _distill, _inputs, _xent
shapes = [(1, 512, 256, BF), (5, 72, 3000, F32), (40, 72, 1500, BF), (300, 64, 3001, BF), (90, 41, 700, F32),
          (300, 41, 700, F32), (700, 64, 128, BF)]
ps = [_inputs(r, d, v, t, 3 + r, bias=r != 40, k=4) for r, d, v, t in shapes]
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    got = [(_xent(p), _distill(p, 2.0)) for p in ps]
g.replay()
torch.cuda.synchronize()
for p, (a, b) in zip(ps, got):
    for x, y in ((a, _xent(p)), (b, _distill(p, 2.0))):
        for n in x:
            assert x[n] is None and y[n] is None or torch.equal(x[n], y[n]), n
print("FINE")
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300, cwd=ROOT)
    assert r.returncode == 0 and "FINE" in r.stdout, r.stdout + r.stderr
