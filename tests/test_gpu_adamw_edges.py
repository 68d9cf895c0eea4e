"""The optimiser step where a value leaves fp32, or a tensor its memory."""
import pytest
import torch

import transformer_xl_relative_rel_gb300 as txl
from tests.test_gpu_adamw import HYPER, KINDS, _copy, _model, _step
from tests.train_helpers import BF, H, U, adamw_reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from transformer_xl_relative_rel_gb300 import _build
    _build.build()


@pytest.mark.parametrize("small", [False, True])
@pytest.mark.parametrize("decay", [0.0, 0.1])
@pytest.mark.parametrize("kind", ["f32", "master", "8 bits", "8 bits f32", "8 bits bf16"])
def test_a_second_moment_past_the_largest_number(kind, decay, small):
    """A finite gradient of 1e25, whose square is not: v is infinite, and the
    update m / (sqrt(v) + eps) is 0, whatever its neighbours are (small: some
    of them have moments among the smallest numbers)."""
    model = _model([2000], 41, KINDS[kind])
    bits8 = model["exp_avg_scales"][0] is not None
    if small:
        for name in ("exp_avgs", "exp_avg_sqs"):
            model[name][0].zero_()
        model["grads"][0][296:300] = 1e-19
    model["grads"][0][300] = 1e25
    before = _copy(model)
    _step(model, decay=decay)
    txl.check()
    p = before["masters"][0] if before["masters"][0] is not None else before["params"][0]
    got = (model["masters"][0] if before["masters"][0] is not None else model["params"][0]).double()
    if before["masters"][0] is not None:
        assert torch.equal(model["params"][0], model["masters"][0].to(BF))
    m, v = before["exp_avgs"][0].double(), before["exp_avg_sqs"][0].double()
    if bits8:
        wide = lambda s: s.double().repeat_interleave(256)[:2000]
        m, v = m * wide(before["exp_avg_scales"][0]), (v * wide(before["exp_avg_sq_scales"][0])) ** 2
    want, tol = adamw_reference(p, before["grads"][0], m, v, HYPER["lr"], HYPER["step"], HYPER["beta1"], HYPER["beta2"],
                                HYPER["eps"], decay)
    want["p"][300] = float(p[300]) * (1 - HYPER["lr"] * decay)
    tol["p"][300] = 6 * H * abs(float(p[300]))
    lim = tol["p"] + (U[BF] * want["p"].abs() * (1 + 2 * H) if p.dtype == BF else 0)
    assert torch.isfinite(got).all()
    assert float(((got - want["p"]).abs() - lim).max()) <= 0
    if bits8:       # the block's second moments are lost, its first ones and other blocks are not
        assert model["exp_avg_sq_scales"][0][1].isnan() and torch.isfinite(model["exp_avg_scales"][0]).all()
        assert int(torch.isfinite(model["exp_avg_sq_scales"][0]).sum()) == 7
    else:
        assert float(model["exp_avg_sqs"][0][300]) == float("inf")


@pytest.mark.parametrize("kind", ["master", "8 bits"])
def test_tensors_moved_elsewhere_leave_their_memory_to_the_step(kind):
    """A weight whose storage is replaced after the list was made: the step
    still acts on the memory it was given, which nobody else gets meanwhile."""
    n = 300_000
    model = _model([n], 42, KINDS[kind])
    twin = _copy(model)
    t = txl.AdamwTensors(**model)
    moved = {name: x[0].clone() for name, x in model.items() if x[0] is not None}
    sizes = [(x.shape, x.dtype) for x in moved.values()]
    for name, x in moved.items():
        model[name][0].data = x
    # what is allocated now would get the memory, had it been given back
    others = [torch.full(shape, 0.5, device="cuda").to(dt) for shape, dt in sizes * 3]
    torch.cuda.synchronize()
    txl.adamw_step(t, 1e-2, 3)
    txl.check()
    assert all((x.float() == 0.5).all() for x in others)
    for name in moved:      # the new places are not the list's
        assert torch.equal(model[name][0].view(torch.uint8), twin[name][0].view(torch.uint8)), name
