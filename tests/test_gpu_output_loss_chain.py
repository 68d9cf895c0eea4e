"""The output-layer losses on the GPU where calls, launches, items and pieces
follow one another: empty batches, calls of different inputs back to back in
one workspace, row blocks that end inside a warp's rows, vocabularies of one
strip and of several pieces, and masks of a type's lowest value.  Bounds as in
tests/loss_helpers.py."""
import pytest
import torch

from tests.test_gpu_output_loss import (BF, F32, _check_distill, _check_xent, _distill, _inputs,  # noqa: F401
                                        _lib, _xent)

pytestmark = pytest.mark.gpu


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
