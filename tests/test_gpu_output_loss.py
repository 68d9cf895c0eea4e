"""The output layer's losses (softmax_xent, distill) on the GPU against the
float64 formulas, within the elementwise bounds of tests/loss_helpers.py:
odd and ragged sizes, one row, one token, empty rows, infinities, unaligned
buffers, several vocabulary pieces, streams, graphs, determinism."""
import math

import numpy as np
import pytest
import torch

import oracle
from tests.loss_helpers import check, distill_reference, xent_reference

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from transformer_xl_relative_rel_gb300 import _build, abi
    _build.build()
    abi.load_library()


def abi_library():
    from transformer_xl_relative_rel_gb300 import abi
    return abi.load_library()


def _inputs(rows, d, vocab, dtype, seed, bias=True, k=None, t_dtype=F32):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, device="cuda", generator=g)
    p = dict(h=r(rows, d).to(dtype), w=(r(vocab, d) * (2 / math.sqrt(d))).to(dtype), bias=r(vocab) if bias else None,
             dloss=r(rows))
    p["target"] = torch.randint(0, vocab, (rows,), device="cuda", generator=g)
    if rows > 3:
        p["target"][1] = -100
        p["target"][rows // 2] = vocab         # just outside
        p["dloss"][2] = 0.0
    if k:
        p["idx"] = torch.randint(0, vocab, (rows, k), device="cuda", generator=g)   # repeats happen
        p["y"] = (r(rows, k) * 2).to(t_dtype)
        if rows > 3:
            p["idx"][1] = -1
            p["idx"][0, k // 2] = vocab + 5
            p["y"][3, k - 1] = -float("inf")
    return p


def _xent(p, weight_grads=True, **kw):
    import transformer_xl_relative_rel_gb300 as txl
    loss, lse = txl.softmax_xent_fwd(p["h"], p["w"], p["target"], bias=p["bias"], **kw)
    g = txl.softmax_xent_bwd(p["h"], p["w"], p["target"], lse, p["dloss"], bias=p["bias"], weight_grads=weight_grads,
                             **kw)
    return dict(loss=loss, lse=lse, **g)


def _distill(p, t, weight_grads=True, **kw):
    import transformer_xl_relative_rel_gb300 as txl
    loss, lse = txl.distill_fwd(p["h"], p["w"], p["idx"], p["y"], t, bias=p["bias"], **kw)
    g = txl.distill_bwd(p["h"], p["w"], p["idx"], p["y"], lse, p["dloss"], t, bias=p["bias"],
                        weight_grads=weight_grads, **kw)
    return dict(loss=loss, lse=lse, **g)


def _check_xent(p, what="", got=None):
    import transformer_xl_relative_rel_gb300 as txl
    got = _xent(p) if got is None else got
    torch.cuda.synchronize()
    txl.check()
    want, tol = xent_reference(p["h"], p["w"], p["bias"], p["target"], p["dloss"])
    # the forward's lse covers empty rows too
    full, ftol = xent_reference(p["h"], p["w"], p["bias"], p["target"])
    want["lse"], tol["lse"] = full["lse"], ftol["lse"]
    check(got, want, tol, what)


def _check_distill(p, t, what="", got=None):
    import transformer_xl_relative_rel_gb300 as txl
    got = _distill(p, t) if got is None else got
    torch.cuda.synchronize()
    txl.check()
    want, tol = distill_reference(p["h"], p["w"], p["bias"], p["idx"], p["y"], t, p["dloss"])
    full, ftol = distill_reference(p["h"], p["w"], p["bias"], p["idx"], p["y"], t)
    want["lse"], tol["lse"] = full["lse"], ftol["lse"]
    check(got, want, tol, what)


SIZES = [(1, 8, 1), (1, 64, 2), (1, 512, 256), (1, 1024, 5003), (2, 1, 7), (3, 41, 63), (5, 16, 64), (31, 7, 65),
         (64, 64, 257), (127, 100, 255), (128, 128, 256), (129, 130, 513), (200, 410, 1000), (257, 256, 5003),
         (300, 520, 300), (1000, 72, 40), (70, 33, 20011)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,d,vocab", SIZES)
def test_xent_sizes(rows, d, vocab, dtype):
    _check_xent(_inputs(rows, d, vocab, dtype, rows * 7 + d, bias=(rows + d) % 2 == 0))


@pytest.mark.parametrize("rows,d,vocab,k,t,dtype,t_dtype", [
    (1, 8, 3, 1, 1.0, BF, F32), (1, 64, 300, 5, 2.0, F32, F32), (4, 41, 63, 2, 0.5, BF, BF),
    (33, 64, 64, 64, 4.0, BF, F32), (130, 128, 500, 33, 1.5, BF, BF), (257, 256, 5003, 16, 2.0, BF, F32),
    (65, 410, 777, 100, 3.0, F32, BF), (128, 512, 1024, 256, 2.0, BF, F32), (300, 72, 40, 8, 1.0, F32, F32)])
def test_distill_sizes(rows, d, vocab, k, t, dtype, t_dtype):
    _check_distill(_inputs(rows, d, vocab, dtype, rows * 5 + d + k, bias=k % 2 == 1, k=k, t_dtype=t_dtype), t)


# few rows: heights 2, 8, 16 and the first past them, rows of every alignment,
# chunks of 16 to 64 tokens, blocks of one and of many chunks, the widest rows
FEW = [(1, 1, 1), (2, 3, 17), (1, 1024, 9001), (2, 410, 20011), (3, 30, 65), (8, 769, 3001), (9, 64, 64),
       (8, 1023, 5001), (15, 2, 40000), (16, 1024, 5003), (16, 410, 2433), (17, 410, 300), (7, 1025, 200), (5, 6, 9729),
       (2, 1024, 512), (8, 100, 513), (16, 128, 512), (8, 256, 500), (1, 8, 129)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,d,vocab", FEW)
def test_few_rows(rows, d, vocab, dtype):
    _check_xent(_inputs(rows, d, vocab, dtype, rows + d, bias=(rows + d) % 2 == 0))
    k = min(256, 3 + vocab // 50)     # listed columns in chunks of both parities
    _check_distill(_inputs(rows, d, vocab, dtype, rows + 2 * d, bias=d % 2 == 1, k=k), 2.0)


@pytest.mark.parametrize("dtype,d", [(BF, 41), (BF, 62), (F32, 41), (F32, 62), (F32, 64)])
def test_few_rows_edges(dtype, d):
    """Empty rows, infinities, absent gradients, untouched neighbours and a
    gradient that is only element-aligned, as for many rows."""
    import transformer_xl_relative_rel_gb300 as txl
    p = _inputs(6, d, 1500, dtype, 5, k=9)
    q = dict(p, h=p["h"].clone(), dloss=p["dloss"].clone(), bias=p["bias"].clone())
    q["h"][1] = float("nan")
    q["dloss"][1] = float("nan")
    for fn in (_xent, lambda x: _distill(x, 2.0)):
        a, b = fn(p), fn(q)
        for n in ("loss", "dh", "dw", "db"):
            assert torch.equal(a[n], b[n]), n
        assert not b["dh"][1].any() and not b["dh"][2].any()      # an empty row, dloss 0
        assert torch.equal(fn(dict(p, bias=None))["lse"], fn(dict(p, bias=torch.zeros_like(p["bias"])))["lse"])
    p["bias"][10:1490] = -float("inf")
    for n in ("target", "idx"):
        p[n] = torch.where((p[n] >= 0) & (p[n] < 1500), p[n] % 10, p[n])
    _check_xent(p)
    _check_distill(p, 2.0)
    whole = _xent(p)
    loss, lse = txl.softmax_xent_fwd(p["h"], p["w"], p["target"], bias=p["bias"])
    for names in (("dh",), ("dw",), ("db",), ("dh", "db")):
        flats = {n: torch.full((whole[n].numel() + 16,), 7.0, dtype=whole[n].dtype, device="cuda") for n in names}
        grads = {n: flats[n][1:1 + whole[n].numel()].view(whole[n].shape) for n in names}
        txl.softmax_xent_bwd(p["h"], p["w"], p["target"], lse, p["dloss"], bias=p["bias"], grads=grads)
        for n in names:
            assert torch.equal(grads[n], whole[n]), (names, n)
            assert flats[n][0] == 7 and (flats[n][1 + whole[n].numel():] == 7).all(), (names, n)
    p["bias"][:] = -float("inf")
    g = _xent(p)
    assert (g["lse"] == -float("inf")).all() and not g["loss"].any()
    assert not g["dh"].any() and not g["dw"].any() and not g["db"].any()
    txl.check()


@pytest.mark.parametrize("dtype,rows,d,vocab", [(BF, 70, 64, 3000), (BF, 300, 72, 5003), (F32, 90, 41, 700)])
def test_each_gradient_alone(dtype, rows, d, vocab):
    import transformer_xl_relative_rel_gb300 as txl
    p = _inputs(rows, d, vocab, dtype, 6, k=7)
    loss, lse = txl.softmax_xent_fwd(p["h"], p["w"], p["target"], bias=p["bias"])
    t_loss, t_lse = txl.distill_fwd(p["h"], p["w"], p["idx"], p["y"], 2.0, bias=p["bias"])
    f = abi_library()
    code = {BF: txl.TXL_BF16, F32: txl.TXL_F32}[dtype]
    ws = torch.empty(txl.distill_workspace_bytes(rows, d, vocab, 7, code, backward=True), dtype=torch.uint8, device="cuda")
    at = lambda x: None if x is None else x.data_ptr()
    for op, whole in (("xent", _xent(p)), ("distill", _distill(p, 2.0))):
        for names in (("dh",), ("dw",), ("db",), ("dw", "db"), ("dh", "db"), ("dh", "dw")):
            g = {n: torch.full_like(whole[n], 7.0) if n in names else None for n in ("dh", "dw", "db")}
            out = [at(g[n]) for n in ("dh", "dw", "db")] + [at(ws), ws.numel(), torch.cuda.current_stream().cuda_stream]
            head = [at(p["h"]), at(p["w"]), at(p["bias"])]
            if op == "xent":
                st = f.txl_softmax_xent_bwd(*head, at(p["target"]), at(lse), at(p["dloss"]), rows, d, vocab, code, *out)
            else:
                st = f.txl_distill_bwd(*head, at(p["idx"]), at(p["y"]), 0, 2.0, at(t_lse), at(p["dloss"]), rows, d, vocab,
                                       7, code, *out)
            assert st == 0
            for n in names:
                assert torch.equal(g[n], whole[n]), (op, names, n)
    txl.check()


def test_few_rows_unaligned_weights():
    for dtype, d in ((BF, 64), (BF, 41), (F32, 64), (F32, 31)):
        p = _inputs(7, d, 900, dtype, 8, k=5)
        flat = torch.empty(p["w"].numel() + 1, dtype=dtype, device="cuda")
        w = flat[1:].view_as(p["w"])
        w.copy_(p["w"])
        _check_xent(dict(p, w=w))
        _check_distill(dict(p, w=w), 2.0)


@pytest.mark.parametrize("dtype,rows,d,vocab", [(BF, 3, 1023, 2100003), (BF, 40, 1024, 2100003), (BF, 200, 1024, 2100003),
                                                (F32, 2, 1024, 1050003), (F32, 20, 1024, 2100003)])
def test_offsets_past_32_bits(dtype, rows, d, vocab):
    """Only the last 500 tokens take part (the others' bias is -infinity): the
    result is that of a vocabulary of 500."""
    import transformer_xl_relative_rel_gb300 as txl
    n = 500
    p = _inputs(rows, d, n, dtype, 9)
    w = torch.empty(vocab, d, dtype=dtype, device="cuda").normal_(std=2 / math.sqrt(d),
                                                                  generator=torch.Generator(device="cuda").manual_seed(1))
    w[-n:] = p["w"]
    bias = torch.full((vocab,), -float("inf"), device="cuda")
    bias[-n:] = p["bias"]
    y = p["target"]
    far = torch.where((y >= 0) & (y < n), y + (vocab - n), y.clamp(max=-1))
    got = _xent(dict(p, w=w, bias=bias, target=far))
    assert not got["db"][:-n].any()
    for x in got["dw"][:-n].split(200000):
        assert not x.any()
    _check_xent(p, got=dict(got, dw=got["dw"][-n:].clone(), db=got["db"][-n:]))
    txl.check()


def test_small_problem_matches_the_oracle():
    p = _inputs(9, 16, 70, F32, 3, k=4)
    n = lambda x: x.double().cpu().numpy()
    loss, lse, g = oracle.softmax_xent(n(p["h"]), n(p["w"]), p["target"].cpu().numpy(), n(p["bias"]), n(p["dloss"]))
    _, tol = xent_reference(p["h"], p["w"], p["bias"], p["target"], p["dloss"])
    want = {k: torch.from_numpy(np.asarray(v)) for k, v in dict(loss=loss, lse=lse, **g).items()}
    check(_xent(p), want, tol)
    loss, lse, g = oracle.distill(n(p["h"]), n(p["w"]), p["idx"].cpu().numpy(), n(p["y"]), 2.0, n(p["bias"]),
                                  n(p["dloss"]))
    _, tol = distill_reference(p["h"], p["w"], p["bias"], p["idx"], p["y"], 2.0, p["dloss"])
    want = {k: torch.from_numpy(np.asarray(v)) for k, v in dict(loss=loss, lse=lse, **g).items()}
    check(_distill(p, 2.0), want, tol)


@pytest.mark.parametrize("dtype,rows,d,vocab", [(BF, 2048, 128, 70001), (BF, 3000, 410, 24000), (F32, 900, 64, 41003)])
def test_several_vocabulary_pieces(dtype, rows, d, vocab):
    _check_xent(_inputs(rows, d, vocab, dtype, 11))
    _check_distill(_inputs(rows, d, vocab, dtype, 12, k=20), 2.0)


def test_small_vocabulary_many_rows():
    _check_xent(_inputs(9000, 512, 204, BF, 21))
    _check_distill(_inputs(5000, 96, 130, BF, 22, k=12), 1.5)


def test_empty_rows_may_hold_anything():
    p = _inputs(140, 64, 300, BF, 31, k=6)
    empty = torch.arange(0, 140, 3, device="cuda")
    p["target"][empty] = -1
    p["target"][7] = 2 ** 40
    p["idx"][empty] = -7
    keep = p["h"].clone()
    for bad in (float("nan"), float("inf")):
        p["h"] = keep.clone()
        p["h"][empty] = bad
        p["dloss"][empty] = bad
        for fn, name in ((_xent, "xent"), (lambda q: _distill(q, 2.0), "distill")):
            got = fn(p)
            clean = dict(p, h=keep, dloss=torch.nan_to_num(p["dloss"], 0.0, 0.0, 0.0))
            want = fn(clean)
            assert not got["loss"][empty].any() and not got["dh"][empty].any(), name
            for n in ("loss", "dh", "dw", "db"):
                assert torch.equal(got[n], want[n]), (name, n)
    # a row of dloss 0 adds nothing either, whatever it holds
    p["h"] = keep.clone()
    p["h"][2] = float("nan")
    g = _xent(p)
    assert not g["dh"][2].any() and torch.isfinite(g["dw"]).all()


def test_all_rows_empty():
    p = _inputs(50, 64, 200, BF, 33, k=3)
    p["target"][:] = -100
    p["idx"][:] = 200
    for g in (_xent(p), _distill(p, 1.0)):
        for n in ("loss", "dh", "dw", "db"):
            assert not g[n].any(), n
        assert torch.isfinite(g["lse"]).all()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_masked_vocabulary(dtype):
    p = _inputs(90, 64, 500, dtype, 41, k=5)
    off = torch.arange(500, device="cuda") % 3 == 0
    off[256:320] = True
    p["bias"][off] = -float("inf")
    allowed = torch.nonzero(~off)[:, 0]
    p["target"] = torch.where(p["target"].clamp(0, 499) == p["target"], allowed[p["target"] % len(allowed)],
                              p["target"])
    p["idx"] = torch.where(p["idx"].clamp(0, 499) == p["idx"], allowed[p["idx"] % len(allowed)], p["idx"])
    _check_xent(p)
    _check_distill(p, 2.0)
    assert not _xent(p)["dw"][off].any()
    # the type's lowest value masks as well (its logit overflows nowhere)
    q = dict(p, bias=torch.where(off, torch.full_like(p["bias"], torch.finfo(F32).min), p["bias"]))
    for n, x in _xent(q).items():
        assert torch.equal(x, _xent(p)[n]), n
    # a target that is masked out: an infinite loss
    p["target"][5] = int(torch.nonzero(off)[0])
    loss = _xent(p)["loss"]
    assert loss[5] == float("inf") and torch.isfinite(loss[6:]).all()


def test_no_finite_logit():
    p = _inputs(40, 64, 130, BF, 42, k=2)
    p["bias"][:] = -float("inf")
    for g in (_xent(p), _distill(p, 2.0)):
        assert (g["lse"] == -float("inf")).all()
        for n in ("loss", "dh", "dw", "db"):
            assert not g[n].any(), n


def test_large_logits_and_nan():
    p = _inputs(60, 64, 300, BF, 43)
    p["h"] = (p["h"].float() * 200).to(BF)         # logits in the hundreds: exp overflows without the maximum
    _check_xent(p)
    p["h"][4] = float("nan")
    p["target"][4] = 3
    got = _xent(p)
    assert torch.isnan(got["loss"][4]) and torch.isnan(got["lse"][4]) and torch.isnan(got["dh"][4]).all()
    ok = torch.arange(60, device="cuda") != 4
    assert torch.isfinite(got["loss"][ok]).all() and torch.isfinite(got["dh"][ok]).all()


def test_unaligned_buffers_and_untouched_neighbours():
    import transformer_xl_relative_rel_gb300 as txl
    for dtype, d in ((BF, 64), (BF, 41), (F32, 64), (F32, 30)):
        p = _inputs(75, d, 210, dtype, 51, k=3)

        def shifted(x, by):
            flat = torch.full((x.numel() + 16,), 7.0, dtype=x.dtype, device="cuda")
            v = flat[by:by + x.numel()].view(x.shape)
            v.copy_(x)
            return flat, v

        q = dict(p)
        for n, by in (("h", 1), ("w", 3), ("bias", 1), ("dloss", 3)):
            q[n] = shifted(p[n], by)[1]
        flats, grads = {}, {}
        for n, like, by in (("dh", p["h"], 5), ("dw", p["w"], 1), ("db", p["bias"], 3)):
            flats[n], grads[n] = shifted(torch.zeros_like(like), by)
        loss, lse = txl.softmax_xent_fwd(q["h"], q["w"], q["target"], bias=q["bias"])
        txl.softmax_xent_bwd(q["h"], q["w"], q["target"], lse, q["dloss"], bias=q["bias"], grads=grads)
        _check_xent(p, got=dict(loss=loss, lse=lse, **grads))
        for n, by in (("dh", 5), ("dw", 1), ("db", 3)):
            rest = torch.cat([flats[n][:by], flats[n][by + grads[n].numel():]])
            assert (rest == 7).all(), n


def test_leading_shape_absent_gradients_and_workspace_contents():
    import transformer_xl_relative_rel_gb300 as txl
    p = _inputs(6 * 11, 64, 333, BF, 61, bias=False, k=4)
    lead = dict(p, h=p["h"].view(6, 11, 64), target=p["target"].view(6, 11), dloss=p["dloss"].view(6, 11),
                idx=p["idx"].view(6, 11, 4), y=p["y"].view(6, 11, 4))
    a, b = _xent(p), _xent(lead)
    assert b["loss"].shape == (6, 11) and b["db"] is None
    for n in ("loss", "lse", "dh", "dw"):
        assert torch.equal(a[n].flatten(), b[n].flatten()), n
    assert torch.equal(_distill(p, 2.0)["dw"], _distill(lead, 2.0)["dw"])
    only = _xent(p, weight_grads=False)
    assert only["dw"] is None and only["db"] is None and torch.equal(only["dh"], a["dh"])
    # a bias gradient without a bias; a workspace full of NaN, larger than asked for
    n = txl.softmax_xent_workspace_bytes(66, 64, 333, txl.TXL_BF16, backward=True)
    ws = torch.full((n // 4 + 100,), float("nan"), device="cuda")
    loss, lse = txl.softmax_xent_fwd(p["h"], p["w"], p["target"], workspace=ws)
    ws.fill_(float("nan"))
    g = txl.softmax_xent_bwd(p["h"], p["w"], p["target"], lse, p["dloss"], workspace=ws,
                             grads=dict(db=torch.empty(333, device="cuda")))
    _check_xent(p, got=dict(loss=loss, lse=lse, **g))
    assert torch.isnan(ws[n // 4 + 1:]).all()


def test_no_rows():
    import transformer_xl_relative_rel_gb300 as txl
    p = _inputs(0, 64, 100, BF, 62, k=3)
    g = _xent(p)
    assert g["loss"].shape == (0,) and not g["dw"].any() and not g["db"].any() and g["dh"].shape == (0, 64)
    g = _distill(p, 2.0)
    assert not g["dw"].any() and not g["db"].any()
    txl.check()


def test_same_bits_again_and_on_other_streams():
    p = [_inputs(700, 128, 3001, BF, 70 + x, k=9) for x in range(2)]
    want = [(_xent(q), _distill(q, 2.0)) for q in p]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for rep in range(3):
        for s, q in zip(streams, p):          # two calls at once, each with buffers of its own
            got.append((_xent(q, stream=s), _distill(q, 2.0, stream=s)))
    torch.cuda.synchronize()
    for x, pair in enumerate(got):
        for a, b in zip(pair, want[x % 2]):
            for n in b:
                assert torch.equal(a[n], b[n]), n


def test_captured_and_replayed():
    import transformer_xl_relative_rel_gb300 as txl
    p = _inputs(260, 64, 1500, BF, 81, k=5)
    outs = [dict(), dict()]
    graphs = []
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for which, fn in enumerate((_xent, lambda q: _distill(q, 2.0))):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            outs[which] = fn(p)
        graphs.append(g)
    eager_first = _xent(p)
    for seed in (82, 83):
        q = _inputs(260, 64, 1500, BF, seed, k=5)
        for n in ("h", "w", "bias", "dloss", "target", "idx", "y"):
            p[n].copy_(q[n])
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        _check_xent(q, got=outs[0])
        _check_distill(q, 2.0, got=outs[1])
    assert torch.isfinite(eager_first["loss"]).all()
    txl.check()


@pytest.mark.parametrize("dtype,rows", [(F32, 5), (BF, 40)])
def test_few_rows_captured_and_replayed(dtype, rows):
    p = _inputs(rows, 72, 1500, dtype, 84, k=5)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        a, b = _xent(p), _distill(p, 2.0)
    for seed in (85, 86):
        q = _inputs(rows, 72, 1500, dtype, seed, k=5)
        for n in ("h", "w", "bias", "dloss", "target", "idx", "y"):
            p[n].copy_(q[n])
        g.replay()
        g.replay()
        torch.cuda.synchronize()
        _check_xent(q, got=a)
        _check_distill(q, 2.0, got=b)


def test_host_threads_at_once():
    import threading
    shapes = [(5, 72, 900, F32), (300, 64, 2000, BF), (20, 128, 700, BF), (90, 40, 300, F32)]
    ps = [_inputs(r, d, v, t, 95 + r, k=6) for r, d, v, t in shapes]
    want = [(_xent(p), _distill(p, 2.0)) for p in ps]
    torch.cuda.synchronize()
    wrong = []

    def work(x):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(15):
                got = _xent(ps[x]), _distill(ps[x], 2.0)
            s.synchronize()
        for a, b in zip(got, want[x]):
            wrong.extend((x, n) for n in b if not torch.equal(a[n], b[n]))

    threads = [threading.Thread(target=work, args=(x,)) for x in range(len(ps))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong, wrong


def test_gradients_match_differences_of_the_forward():
    """fp32: (L(x + e) - L(x - e)) / 2e along random directions."""
    import transformer_xl_relative_rel_gb300 as txl
    p = _inputs(70, 48, 150, F32, 91, k=6)
    p["target"].clamp_(0, 149)
    g = torch.Generator(device="cuda").manual_seed(5)

    def value(q, op):
        f = txl.softmax_xent_fwd(q["h"], q["w"], q["target"], bias=q["bias"]) if op == "xent" else \
            txl.distill_fwd(q["h"], q["w"], q["idx"], q["y"], 2.0, bias=q["bias"])
        return float((f[0].double() * q["dloss"].double()).sum())

    for op, grads in (("xent", _xent(p)), ("distill", _distill(p, 2.0))):
        for name in ("h", "w", "bias"):
            e = torch.randn(p[name].shape, device="cuda", generator=g)
            e /= e.norm()
            eps = 1e-2
            up, down = dict(p), dict(p)
            up[name], down[name] = p[name] + eps * e, p[name] - eps * e
            num = (value(up, op) - value(down, op)) / (2 * eps)
            ana = float((grads["db" if name == "bias" else "d" + name].double() * e.double()).sum())
            # third derivatives of a log-sum-exp along a unit direction are below the
            # cube of the operand's row norm (8 here): eps^2/6 * 512 * sum|dloss| / sqrt(rows);
            # the forward's own error (2^-19 per row) divides by eps
            lim = eps ** 2 / 6 * 8 + 70 * 2.0 ** -19 / eps
            assert abs(num - ana) <= lim, (op, name, num, ana)


def test_training_step_of_a_layer_and_its_output():
    """The attention's backward takes what the losses' backwards give: cross
    entropy and distillation on the same hidden states, their gradients added,
    against float64 autograd through the same layer."""
    import transformer_xl_relative_rel_gb300 as txl
    from tests.helpers import unit_shape
    from transformer_xl_relative_rel_gb300 import inputs
    B, H, D, L, M, V, K = 2, 2, 64, 40, 24, 150, 4
    lay = inputs.unit_layer(unit_shape(B, H, D, L, M), 7)
    dev = {n: torch.from_numpy(lay[n]).cuda().to(BF) for n in ("q", "k", "v", "r")}
    u, b = (torch.from_numpy(lay[n]).cuda() for n in ("u", "w"))
    p = _inputs(L * B, H * D, V, BF, 17, k=K)
    target, idx, y = p["target"].view(L, B), p["idx"].view(L, B, K), p["y"].view(L, B, K)
    dloss = torch.full((L, B), 1.0 / (L * B), device="cuda")
    lse_a = torch.empty(B, H, L, device="cuda")
    out = txl.rel_attn_fwd(dev["q"], dev["k"], dev["v"], dev["r"], u, b, mem_len=M, lse=lse_a)
    hid = out.view(L, B, H * D)
    l1, lse1 = txl.softmax_xent_fwd(hid, p["w"], target, bias=p["bias"])
    l2, lse2 = txl.distill_fwd(hid, p["w"], idx, y, 2.0, bias=p["bias"])
    g1 = txl.softmax_xent_bwd(hid, p["w"], target, lse1, dloss, bias=p["bias"])
    g2 = txl.distill_bwd(hid, p["w"], idx, y, lse2, dloss, 2.0, bias=p["bias"])
    dout = (g1["dh"] + g2["dh"]).view(L, B, H, D)
    ga = txl.rel_attn_bwd(dev["q"], dev["k"], dev["v"], dev["r"], u, b, dout, mem_len=M, out=out, lse=lse_a)
    torch.cuda.synchronize()
    txl.check()
    h2 = hid.reshape(L * B, H * D)
    f = lambda x: x.reshape((L * B,) + x.shape[2:])
    w1, t1 = xent_reference(h2, p["w"], p["bias"], f(target), f(dloss))
    w2, t2 = distill_reference(h2, p["w"], p["bias"], f(idx), f(y), 2.0, f(dloss))
    for n in ("dh", "dw", "db"):
        # the sum of two bf16 gradients is rounded once more
        tol = t1[n] + t2[n] + 2.0 ** -8 * (w1[n] + w2[n]).abs() * (n == "dh")
        check({n: (g1[n] + g2[n]).reshape(w1[n].shape) if n != "dw" else g1[n].double() + g2[n].double()},
              {n: w1[n] + w2[n]}, {n: tol})
    host = {n: dev[n].double().cpu().numpy() for n in dev}
    ref = oracle.rel_attn_bwd(**host, u=u.double().cpu().numpy(), w=b.double().cpu().numpy(),
                              dout=dout.double().cpu().numpy(), mem_len=M)
    for n in ("dq", "dk", "dv", "dr", "du", "dw"):
        e = np.abs(ga[n].double().cpu().numpy() - ref[n]).max() / max(1.0, np.abs(ref[n]).max())
        assert e <= 2e-2, n
