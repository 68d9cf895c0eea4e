"""Calls of the output-layer losses that no kernel could answer rightly are
refused on the host.  No compute call is made."""
import pytest
import torch

import transformer_xl_relative_rel_gb300 as txl
from tests.test_output_loss_host import CUDA, INVALID, _call, lib  # noqa: F401 (lib: a fixture)


@pytest.mark.parametrize("backward", [False, True])
def test_temperatures_whose_square_is_no_float(backward):
    """t^2 scales the loss: 2^64 and more would make it infinite or NaN, below
    2^-63 it would lose bits and vanish."""
    for t in (2.0 ** 64, 1e38, 2.0 ** -64, 1e-30):
        assert _call("distill", backward, t=t) == INVALID, t
    if not torch.cuda.is_available():           # accepted: only the launch fails
        for t in (2.0 ** 63, 2.0 ** -63, 1.0):
            assert _call("distill", backward, t=t) == CUDA, t
