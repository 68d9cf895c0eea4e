"""Workspace queries of the output-layer losses at the ends of their ranges:
batches without rows (which need nothing, whatever the vocabulary), and sizes
from one element to the largest that are taken.  No compute call is made."""
import itertools
import random

import pytest

import transformer_xl_relative_rel_gb300 as txl

DTYPES = (txl.TXL_BF16, txl.TXL_F32)


@pytest.fixture(scope="module", autouse=True)
def lib():
    from transformer_xl_relative_rel_gb300 import _build, abi
    _build.build()
    abi.load_library()


@pytest.mark.parametrize("vocab", [1, 100, 257, 5003, 32768, 1 << 30])
@pytest.mark.parametrize("dtype", DTYPES)
def test_no_rows(vocab, dtype):
    for d, backward in itertools.product((1, 64, 410, 1024), (False, True)):
        assert 0 < txl.softmax_xent_workspace_bytes(0, d, vocab, dtype, backward=backward) <= 4096
        assert 0 < txl.distill_workspace_bytes(0, d, vocab, 5, dtype, backward=backward) <= 4096


def test_any_sizes():
    """Every size that is taken has an answer: the backward's serves the
    forward, and holds at least a piece's dz or the few rows' parts of dh."""
    rng = random.Random(5)
    edge = [1, 2, 8, 9, 16, 17, 127, 128, 129, 255, 256, 257, 1 << 16, 1 << 20, 1 << 30]
    for x in range(1500):
        pick = lambda most: min(most, rng.choice(edge) if rng.random() < 0.4 else int(2 ** rng.uniform(0, 30)))
        d = pick(1 << 14)
        rows, vocab = pick((1 << 40) // d), pick((1 << 40) // d)
        dtype, k = rng.choice(DTYPES), rng.choice([0, 1, 7, 256])
        size = lambda b: txl.distill_workspace_bytes(rows, d, vocab, k, dtype, backward=b) if k else \
            txl.softmax_xent_workspace_bytes(rows, d, vocab, dtype, backward=b)
        fwd, bwd = size(False), size(True)
        assert 0 < fwd <= bwd, (rows, d, vocab, dtype, k)
        assert bwd >= rows * min(vocab, 256) * 2 or bwd >= rows * d * 4, (rows, d, vocab, dtype, k)
