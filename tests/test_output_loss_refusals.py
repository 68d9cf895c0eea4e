"""Calls of the output-layer losses that no kernel could answer rightly are
refused on the host.  No compute call is made."""
import pytest
import torch

import transformer_xl_relative_rel_gb300 as txl
from tests.test_output_loss_host import CUDA, INVALID, UNSUPPORTED, _call, lib  # noqa: F401 (lib: a fixture)


@pytest.mark.parametrize("backward", [False, True])
def test_temperatures_whose_square_is_no_float(backward):
    """t^2 scales the loss: 2^64 and more would make it infinite or NaN, below
    2^-63 it would lose bits and vanish."""
    for t in (2.0 ** 64, 1e38, 2.0 ** -64, 1e-30):
        assert _call("distill", backward, t=t) == INVALID, t
    if not torch.cuda.is_available():           # accepted: only the launch fails
        for t in (2.0 ** 63, 2.0 ** -63, 1.0):
            assert _call("distill", backward, t=t) == CUDA, t


def test_sizes_past_a_c_int():
    """2^32 + 5 rows are not 5 rows: sizes that ctypes would cut to 32 bits are
    refused, in queries and calls."""
    far = 2 ** 32 + 5
    bf, f32, i64 = (dict(dtype=x, device="meta") for x in (torch.bfloat16, torch.float32, torch.int64))
    for sizes in ((far, 8, 16), (8, far, 16), (8, 8, far)):
        for backward in (False, True):
            with pytest.raises(txl.TxlError, match="unsupported"):
                txl.softmax_xent_workspace_bytes(*sizes, txl.TXL_BF16, backward=backward)
            with pytest.raises(txl.TxlError, match="unsupported"):
                txl.distill_workspace_bytes(*sizes, 4, txl.TXL_BF16, backward=backward)
        rows, d, vocab = sizes
        h, w = torch.empty(rows, d, **bf), torch.empty(vocab, d, **bf)
        y, f = torch.empty(rows, **i64), torch.empty(rows, **f32)
        idx, t = torch.empty(rows, 4, **i64), torch.empty(rows, 4, **f32)
        for call in (lambda: txl.softmax_xent_fwd(h, w, y), lambda: txl.softmax_xent_bwd(h, w, y, f, f),
                     lambda: txl.distill_fwd(h, w, idx, t), lambda: txl.distill_bwd(h, w, idx, t, f, f)):
            with pytest.raises(txl.TxlError, match="unsupported"):
                call()
    with pytest.raises(txl.TxlError, match="unsupported"):
        txl.distill_workspace_bytes(8, 8, 16, far, txl.TXL_BF16)
    h, w = torch.empty(8, 8, **bf), torch.empty(16, 8, **bf)
    with pytest.raises(txl.TxlError, match="unsupported"):
        txl.distill_fwd(h, w, torch.empty(8, far, **i64), torch.empty(8, far, **f32))


@pytest.mark.parametrize("op,backward", [(o, b) for o in ("xent", "distill") for b in (False, True)])
def test_rows_wider_than_a_bounded_wait(op, backward):
    """A tile's sum over d_model has to end well within the kernels' limit of 2 s per wait."""
    from transformer_xl_relative_rel_gb300 import abi
    for d in ((1 << 24) + 1, 1 << 29):
        assert _call(op, backward, d=d, nws=1 << 60) == UNSUPPORTED
        with pytest.raises(txl.TxlError, match="unsupported"):
            txl.softmax_xent_workspace_bytes(10, d, 100, abi.TXL_BF16, backward=backward)
    assert txl.softmax_xent_workspace_bytes(10, 1 << 24, 100, abi.TXL_BF16, backward=backward) > 0
