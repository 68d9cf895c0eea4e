"""The optimiser step over many tensors and the gradients' norm on the GPU
against float64 (tests/train_helpers.py has the formulas and bounds)."""
import pytest
import torch

from tests.train_helpers import BF, F32, H, U, adamw_reference, check_codes, random_fractions

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn
SIZES = [1, 7, 8, 255, 256, 257, 2047, 2048, 2049, 5000, 0, 100003, 33, 8192, 8193, 3]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from transformer_xl_relative_rel_gb300 import _build
    _build.build()


def _model(sizes, seed, kinds, shift=0):
    """kinds: per tensor (param type, with a master, gradient type, 8-bit moments)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda s: torch.randn(s, device="cuda", generator=g)
    u = lambda s: torch.rand(s, device="cuda", generator=g)

    def place(x):
        if not shift:
            return x
        flat = torch.empty(x.numel() + 8, dtype=x.dtype, device="cuda")
        y = flat[shift:shift + x.numel()]
        y.copy_(x)
        return y

    keys = ("params", "grads", "exp_avgs", "exp_avg_sqs", "masters", "exp_avg_scales", "exp_avg_sq_scales")
    out = {k: [] for k in keys}
    for k, s in enumerate(sizes):
        dt, with_master, g_dt, bits = kinds[k % len(kinds)]
        w, blocks = n(s), (s + 255) // 256
        row = dict(params=w.to(dt), grads=(0.01 * n(s)).to(g_dt), masters=w if with_master else None,
                   exp_avg_scales=None, exp_avg_sq_scales=None)
        if bits == 8:
            row.update(exp_avgs=(100 * n(s)).clamp(-448, 448).to(E4M3), exp_avg_sqs=(448 * u(s)).to(E4M3),
                       exp_avg_scales=1e-5 * (0.5 + u(blocks)), exp_avg_sq_scales=2e-5 * (0.5 + u(blocks)))
        else:
            row.update(exp_avgs=0.003 * n(s), exp_avg_sqs=(0.01 * u(s)) ** 2)
        for name in keys:
            out[name].append(None if row[name] is None else place(row[name]))
    return out


def _copy(model):
    return {k: [None if x is None else x.clone() for x in v] for k, v in model.items()}


HYPER = dict(lr=1e-2, step=7, beta1=0.9, beta2=0.98, eps=1e-6)


def _decay(n):
    return [0.1 * (k % 3) for k in range(n)]


def _step(model, hyper=HYPER, factor=None, seed=99, decay=None, **kw):
    import transformer_xl_relative_rel_gb300 as txl
    t = txl.AdamwTensors(**model, weight_decay=_decay(len(model["params"])) if decay is None else decay)
    h = dict(hyper)
    h.update(kw)
    scale = None if factor is None else torch.tensor([factor], device="cuda")
    txl.adamw_step(t, h.pop("lr"), h.pop("step"), grad_scale=scale, seed=seed, **h)


def _dense(codes, scales):
    return codes.double() * scales.double().repeat_interleave(256)[:codes.numel()]


def _check(before, after, hyper=HYPER, factor=1.0, seed=99):
    import transformer_xl_relative_rel_gb300 as txl
    txl.check()
    for k, p in enumerate(before["params"]):
        if p.numel() == 0:
            continue
        bits8 = before["exp_avg_scales"][k] is not None
        m, v = before["exp_avgs"][k], before["exp_avg_sqs"][k]
        if bits8:
            m, v = _dense(m, before["exp_avg_scales"][k]), _dense(v, before["exp_avg_sq_scales"][k]) ** 2
        master = before["masters"][k]
        h = dict(hyper)
        want, tol = adamw_reference(p if master is None else master, before["grads"][k], m, v, h["lr"], h["step"],
                                    h["beta1"], h["beta2"], h["eps"], _decay(len(before["params"]))[k], factor)
        got = after["params"][k] if master is None else after["masters"][k]
        lim = tol["p"] + (U[p.dtype] * want["p"].abs() * (1 + 2 * H) if master is None and p.dtype == BF else 0)
        off = (got.double() - want["p"]).abs() - lim
        assert float(off.max()) <= 0, (k, p.numel(), float(off.max()))
        if master is not None:
            assert torch.equal(after["params"][k], after["masters"][k].to(BF)), k
        assert torch.equal(before["grads"][k], after["grads"][k])
        if not bits8:
            for name, x in (("exp_avgs", "m"), ("exp_avg_sqs", "v")):
                off = (after[name][k].double() - want[x]).abs() - tol[x]
                assert float(off.max()) <= 1e-44, (k, name)
            continue
        um, uv = random_fractions(seed, k, h["step"], p.numel(), "cuda")
        check_codes(after["exp_avgs"][k], after["exp_avg_scales"][k], want["m"], tol["m"], um, False, f"{k} m")
        root = want["v"].sqrt()
        # off by half v's relative bound, a root and the scaled codes' squares
        check_codes(after["exp_avg_sqs"][k], after["exp_avg_sq_scales"][k], root, 12 * H * root, uv, True, f"{k} v")


KINDS = {"f32": [(F32, False, F32, 32)], "bf16": [(BF, False, BF, 32)], "master": [(BF, True, BF, 32)],
         "master f32 grads": [(BF, True, F32, 32)], "f32 bf16 grads": [(F32, False, BF, 32)],
         "8 bits": [(BF, True, BF, 8)], "8 bits f32": [(F32, False, F32, 8)], "8 bits bf16": [(BF, False, BF, 8)],
         "mixed": [(BF, True, BF, 8), (F32, False, F32, 32), (BF, False, F32, 8), (BF, True, BF, 32), (F32, False, BF, 8)]}


@pytest.mark.parametrize("shift", [0, 1, 4])
@pytest.mark.parametrize("kind", list(KINDS))
def test_types_and_sizes(kind, shift):
    model = _model(SIZES, 3, KINDS[kind], shift)
    before = _copy(model)
    _step(model)
    _check(before, model)


@pytest.mark.parametrize("kind", ["master", "8 bits", "mixed"])
def test_many_tensors(kind):
    """More than one launch takes, in one of them more than the small one."""
    for count in (47, 48, 49, 384, 385, 1000):
        model = _model([SIZES[(5 * k) % len(SIZES)] % 3000 for k in range(count)], count, KINDS[kind])
        before = _copy(model)
        _step(model)
        _check(before, model)


def test_a_large_tensor():
    """Several rounds per chunk."""
    for kind in ("8 bits", "f32"):
        model = _model([9_000_001, 100, 5_000_000], 4, KINDS[kind])
        before = _copy(model)
        _step(model)
        _check(before, model)


@pytest.mark.parametrize("kind", ["f32", "8 bits"])
def test_hyperparameters(kind):
    for change in (dict(step=1), dict(step=100000), dict(step=3, beta1=0.0), dict(step=2, beta2=0.0, beta1=0.5),
                   dict(lr=0.0), dict(eps=1.0), dict(step=2 ** 40, beta2=0.999999)):
        hyper = dict(HYPER, **change)
        model = _model([3000, 70], 5, KINDS[kind])
        before = _copy(model)
        _step(model, hyper)
        _check(before, model, hyper)


@pytest.mark.parametrize("size", [1e-15, 1e-18, 1e-19, 1e-20, 3e-22])
@pytest.mark.parametrize("kind", ["f32", "8 bits"])
def test_second_moments_near_the_smallest_numbers(kind, size):
    """From v of 2^-100 down to the denormals (whose few bits bound what a
    root's square can be told from): the root is still the root."""
    model = _model([3000], 33, KINDS[kind])
    for name in ("exp_avgs", "exp_avg_sqs"):
        model[name][0].zero_()
    g = torch.Generator(device="cuda").manual_seed(1)
    model["grads"][0].copy_(size * 30 * torch.randn(3000, device="cuda", generator=g))
    before = _copy(model)
    hyper = dict(HYPER, step=1, eps=2.0 ** -120, lr=1e-3)
    _step(model, hyper, decay=0.0)
    torch.cuda.synchronize()
    grad = before["grads"][0].double()
    v = (1 - 0.98) * grad ** 2
    # an update of m / sqrt(v) at the first step is the gradient's sign; v is off by half a denormal's step
    kept = v > 2.0 ** -149 * 64
    p = before["masters"][0] if before["masters"][0] is not None else before["params"][0]
    got = model["masters"][0] if before["masters"][0] is not None else model["params"][0]
    want = p.double() - 1e-3 * torch.sign(grad)
    assert int(kept.sum()) > (100 if size > 1e-21 else 10)
    # half of 1/64, one denormal's step in v, of an update of 1e-3, and p's own rounding
    assert float(((got.double() - want).abs() - 2.0 ** -22 * p.abs().double())[kept].max()) <= 1e-3 * (1 / 64 + 1e-4)
    if kind == "f32":
        return
    root = _dense(model["exp_avg_sqs"][0], model["exp_avg_sq_scales"][0])
    # a code is within a step (1/8, or 2^-9 of 448 for the smallest) of what it stands for
    off = (root - v.sqrt()).abs() - v.sqrt() / 7 - model["exp_avg_sq_scales"][0].double().repeat_interleave(256)[:3000] / 512
    assert float(off[kept].max()) <= float(v.sqrt().max()) / 60


@pytest.mark.parametrize("kind", ["f32", "8 bits"])
def test_from_zero_moments(kind):
    """The first step: moments and scales are zero; elements without a gradient do not move."""
    model = _model([5000, 300], 6, KINDS[kind])
    for name in ("exp_avgs", "exp_avg_sqs", "exp_avg_scales", "exp_avg_sq_scales"):
        for x in model[name]:
            if x is not None:
                x.zero_()
    model["grads"][0][256:600] = 0
    model["grads"][0][1000:1003] = 0
    before = _copy(model)
    hyper = dict(HYPER, step=1)
    _step(model, hyper, decay=0.0)
    still = torch.zeros(5000, dtype=torch.bool, device="cuda")
    still[256:600] = still[1000:1003] = True
    moved = (model["masters"][0] if model["masters"][0] is not None else model["params"][0]) != \
        (before["masters"][0] if before["masters"][0] is not None else before["params"][0])
    assert not moved[still].any() and moved[~still].float().mean() > 0.99
    for name in ("exp_avgs", "exp_avg_sqs"):
        assert not model[name][0].double()[still].any()
    # no denominator is lost
    g = before["grads"][0] != 0
    assert (model["exp_avg_sqs"][0].double()[g] > 0).all()


def test_plain_fp32_arithmetic_gives_the_same_codes():
    """The header's formulas, operation by operation in torch's fp32, to the bit."""
    import transformer_xl_relative_rel_gb300 as txl
    n, step, seed = 300_000, 12, 77
    model = _model([n], 30, KINDS["8 bits"])
    before = _copy(model)
    t = txl.AdamwTensors(**model)
    scale = torch.tensor([0.37], device="cuda")
    txl.adamw_step(t, 1e-3, step, grad_scale=scale, seed=seed)
    wide = lambda s: s.repeat_interleave(256)[:n]
    g = before["grads"][0].float() * scale
    m = before["exp_avgs"][0].float() * wide(before["exp_avg_scales"][0])
    r = before["exp_avg_sqs"][0].float() * wide(before["exp_avg_sq_scales"][0])
    b1, c1, b2, c2 = (torch.tensor(x, dtype=F32, device="cuda") for x in (0.9, 1 - 0.9, 0.999, 1 - 0.999))
    m = b1 * m + c1 * g
    root = (b2 * (r * r) + (c2 * g) * g).sqrt()
    for x, name, u, keep in ((m, "exp_avg", 0, False), (root, "exp_avg_sq", 1, True)):
        u = random_fractions(seed, 0, step, n, "cuda")[u].float()
        top = torch.nn.functional.pad(x, (0, -n % 256)).view(-1, 256).abs().amax(1)
        y = x.abs() * wide((1 / top.double()).float() * 448)
        e = torch.frexp(y)[1].clamp(min=-5) - 1
        unit = ((e - 3 + 127) << 23).view(F32)
        steps = (y / unit + u).floor()
        if keep:
            steps = torch.where(y > 0, steps.clamp(min=1), steps)
        want = torch.sign(x) * (steps * unit).clamp(max=448)
        assert torch.equal(model[name + "s"][0].float(), want), name
        inverse = torch.tensor(1 / 448, dtype=F32, device="cuda")
        assert torch.equal(model[name + "_scales"][0], top * inverse), name


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_gradients_that_are_not_finite_stay_in_their_block(bad):
    for kind in ("8 bits", "f32"):
        model = _model([2000, 500], 31, KINDS[kind])
        clean = _copy(model)
        model["grads"][0][300] = bad
        _step(model)
        _step(clean)
        lost = torch.zeros(2000, dtype=torch.bool, device="cuda")
        lost[300] = True
        for name in ("params", "masters"):
            if model[name][0] is not None:
                assert torch.equal(model[name][0][~lost], clean[name][0][~lost])
                assert torch.equal(model[name][1], clean[name][1])
        if kind == "f32":
            assert torch.equal(model["exp_avgs"][0][~lost], clean["exp_avgs"][0][~lost])
            continue
        lost[256:512] = True
        for name in ("exp_avg", "exp_avg_sq"):
            assert torch.equal(model[name + "s"][0].double()[~lost], clean[name + "s"][0].double()[~lost])
            s = model[name + "_scales"][0]
            assert s[1].isnan() and torch.equal(s[2:], clean[name + "_scales"][0][2:]) and s[0] == clean[name + "_scales"][0][0]
        # what the next step makes of the lost block is NaN, not a number
        _step(model, step=8)
        assert model["masters"][0][256:512].isnan().all() and torch.isfinite(model["masters"][0][512:]).all()


def test_values_on_the_device():
    """lr, step and grad_scale read when the kernel runs; the same results as host values."""
    import transformer_xl_relative_rel_gb300 as txl
    a = _model(SIZES, 7, KINDS["mixed"])
    b = _copy(a)
    before = _copy(a)
    _step(a, factor=0.3)
    t = txl.AdamwTensors(**b, weight_decay=_decay(len(SIZES)))
    lr, step = torch.tensor([HYPER["lr"]], device="cuda"), torch.tensor([HYPER["step"]], device="cuda")
    scale = torch.tensor([0.3], device="cuda")
    kw = dict(beta1=HYPER["beta1"], beta2=HYPER["beta2"], eps=HYPER["eps"], grad_scale=scale, seed=99)
    txl.adamw_step(t, lr, step, **kw)
    torch.cuda.synchronize()
    for name in a:
        for x, y in zip(a[name], b[name]):
            assert x is None and y is None or torch.equal(x.view(torch.uint8), y.view(torch.uint8)), name
    _check(before, a, factor=float(scale))


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_a_step_without_a_finite_factor_changes_nothing(value):
    import transformer_xl_relative_rel_gb300 as txl
    model = _model(SIZES, 8, KINDS["mixed"])
    before = _copy(model)
    _step(model, factor=value)
    t = txl.AdamwTensors(**model)
    for step in (0, -5):
        txl.adamw_step(t, 1e-2, torch.tensor([step], device="cuda"))
    torch.cuda.synchronize()
    for name in model:
        for x, y in zip(model[name], before[name]):
            assert x is None or torch.equal(x.view(torch.uint8), y.view(torch.uint8)), name


def test_rounding_depends_on_seed_step_and_tensor():
    model = _model([4096, 4096], 9, KINDS["8 bits"])
    for name in model:
        if model[name][0] is not None:
            model[name][1].copy_(model[name][0])
    runs = []
    for seed, step in ((1, 7), (1, 7), (2, 7), (1 + (1 << 40), 7), (1, 8)):
        m = _copy(model)
        _step(m, seed=seed, step=step, decay=0.0)
        runs.append(m["exp_avg_sqs"])
    same = lambda x, y: torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    assert same(runs[0][0], runs[1][0]) and same(runs[0][1], runs[1][1])
    assert not same(runs[0][0], runs[0][1])
    for other in runs[2:]:
        # codes that moved by a step: neither none nor nearly all
        share = float((other[0].double() != runs[0][0].double()).double().mean())
        assert 0.1 < share < 0.9


def test_small_changes_of_the_second_moment_add_up():
    """v decays by 0.1% a step, far below the distance of two codes: after 700
    steps of zero gradients half of it is left, on average over a block."""
    import transformer_xl_relative_rel_gb300 as txl
    n = 256 * 64
    model = _model([n], 10, KINDS["8 bits"])
    model["grads"][0].zero_()
    model["exp_avg_sqs"][0].fill_(104.0)
    model["exp_avg_sqs"][0][::256] = 448.0
    model["exp_avg_sq_scales"][0].fill_(1e-5)
    # the block's largest element keeps its size, so that the scale does
    model["grads"][0][::256] = 448e-5
    t = txl.AdamwTensors(**model)
    for step in range(1, 701):
        txl.adamw_step(t, 0.0, step, beta2=0.999, seed=5)
    torch.cuda.synchronize()
    root = _dense(model["exp_avg_sqs"][0], model["exp_avg_sq_scales"][0])
    rest = torch.ones(n, dtype=torch.bool, device="cuda")
    rest[::256] = False
    mean = float(root[rest].mean()) / (104e-5 * 0.999 ** 350)
    # codes are 8 apart at 104 and 4 below 64: a step's rounding has a variance of at most
    # 0.05 * 8 = 0.4, so 700 have 17^2 at most; the mean of 16000 is within 5 * 17 / 126 = 0.7 of 73
    assert abs(mean - 1) < 0.01 + 5 * 17 / 126.0 / 73, mean


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("sizes", [[1], [5000], SIZES, [9_000_001, 3], [64] * 1000, []])
def test_norm_and_clip(sizes, dtype):
    import transformer_xl_relative_rel_gb300 as txl
    model = _model(sizes, 11, [(F32, False, dtype, 32)])
    t = txl.AdamwTensors(**model)
    want = float(sum((g.double() ** 2).sum() for g in model["grads"])) ** 0.5 if sizes else 0.0
    for max_norm in (want * 0.5 + 1e-3, want * 4 + 1, float("inf")):
        norm, clip = txl.grad_norm(t, max_norm)
        # squares of 24 bits and one rounding of the root, two of the factor
        assert abs(float(norm) - want) <= 2 * H * want
        assert abs(float(clip) - min(1.0, max_norm / max(want, 1e-30))) <= 5 * H
    size = txl.grad_norm_workspace_bytes(t)
    first = txl.grad_norm(t, 0.1)
    for k in range(3):
        again = txl.grad_norm(t, 0.1, workspace=torch.full((size,), 255, dtype=torch.uint8, device="cuda"))
        assert torch.equal(again[0], first[0]) and torch.equal(again[1], first[1])
    txl.check()


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), 1e25])
def test_a_norm_that_is_not_finite_skips_the_step(bad):
    import transformer_xl_relative_rel_gb300 as txl
    model = _model([300, 70000], 12, KINDS["master"])
    model["grads"][1][69999] = bad
    before = _copy(model)
    t = txl.AdamwTensors(**model)
    norm, clip = txl.grad_norm(t, 1.0)
    assert not torch.isfinite(norm).any() and clip.isnan().all()
    txl.adamw_step(t, 1e-2, 1, grad_scale=clip)
    torch.cuda.synchronize()
    for name in model:
        for x, y in zip(model[name], before[name]):
            assert x is None or torch.equal(x.view(torch.uint8), y.view(torch.uint8)), name


def test_captured_steps():
    """A graph of clip and step, replayed with other gradients, rates and step
    numbers, against the same steps made one by one."""
    import transformer_xl_relative_rel_gb300 as txl
    a = _model(SIZES, 13, KINDS["mixed"])
    b = _copy(a)
    ta, tb = txl.AdamwTensors(**a), txl.AdamwTensors(**b)
    lr, step = torch.tensor([0.01], device="cuda"), torch.tensor([0], device="cuda")
    ws = torch.empty(txl.grad_norm_workspace_bytes(ta), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step += 1
        norm, clip = txl.grad_norm(ta, 0.5, workspace=ws)
        txl.adamw_step(ta, lr, step, grad_scale=clip, seed=3)
    for t in range(1, 6):
        for x, y in zip(a["grads"], b["grads"]):
            x.copy_(torch.randn(x.shape, device="cuda"))
            y.copy_(x)
        lr.fill_(0.01 / t)
        g.replay()
        _, c = txl.grad_norm(tb, 0.5)
        txl.adamw_step(tb, float(lr), t, grad_scale=c, seed=3)
        torch.cuda.synchronize()
        assert torch.equal(c, clip) and float(c) < 1
    for name in a:
        for x, y in zip(a[name], b[name]):
            assert x is None or torch.equal(x.view(torch.uint8), y.view(torch.uint8)), name


def test_first_calls_of_a_process_captured():
    """No call has to come before a capture, nor for a list of many tensors."""
    code = """
import torch
import transformer_xl_relative_rel_gb300 as txl
from tests.test_gpu_adamw import KINDS, _copy, _model
tok = torch.randint(-1, 90, (700,), device="cuda")
table, dout = torch.randn(90, 64, device="cuda").bfloat16(), torch.randn(700, 64, device="cuda").bfloat16()
gamma = torch.randn(64, device="cuda")
models = [_model([70 * k + 5 for k in range(n)], 3, KINDS[kind]) for n, kind in ((100, "mixed"), (3, "f32"))]
twins = [_copy(m) for m in models]

def calls(models):
    x = txl.embed_fwd(tok, table, 3.0)
    y, mean, rstd = txl.layer_norm_fwd(x, gamma, residual=dout)
    g = txl.layer_norm_bwd(dout, x, mean, rstd, gamma=gamma, residual=dout)
    out = [x, y, mean, rstd, g["dx"], g["dgamma"], g["dbeta"], txl.embed_bwd(tok, g["dx"], vocab=90)]
    for m in models:
        t = txl.AdamwTensors(**m)
        norm, clip = txl.grad_norm(t, 0.1)
        txl.adamw_step(t, 1e-2, 3, grad_scale=clip, seed=4)
        out += [norm, clip]
    return out

torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = calls(models)
graph.replay()
torch.cuda.synchronize()
for a, b in zip(got, calls(twins)):
    assert torch.equal(a, b)
for a, b in zip(models, twins):
    for n in a:
        for x, y in zip(a[n], b[n]):
            assert x is None or torch.equal(x.view(torch.uint8), y.view(torch.uint8)), n
txl.check()
print("FINE")
"""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300, cwd=root)
    assert r.returncode == 0 and "FINE" in r.stdout, r.stdout + r.stderr


def test_streams_and_host_threads_at_once():
    import threading
    import transformer_xl_relative_rel_gb300 as txl
    models = [_model(SIZES, 14 + k, KINDS["mixed"]) for k in range(3)]
    want = [_copy(m) for m in models]
    for m in want:
        t = txl.AdamwTensors(**m)
        for s in range(1, 11):
            txl.adamw_step(t, 1e-3, s, seed=1, grad_scale=txl.grad_norm(t, 0.1)[1])
    torch.cuda.synchronize()

    def work(x):
        s = torch.cuda.Stream()
        t = txl.AdamwTensors(**models[x])
        with torch.cuda.stream(s):
            for k in range(1, 11):
                txl.adamw_step(t, 1e-3, k, seed=1, grad_scale=txl.grad_norm(t, 0.1)[1])
            s.synchronize()

    threads = [threading.Thread(target=work, args=(x,)) for x in range(3)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for a, b in zip(models, want):
        for name in a:
            for x, y in zip(a[name], b[name]):
                assert x is None or torch.equal(x.view(torch.uint8), y.view(torch.uint8)), name


def test_offsets_past_32_bits():
    """One tensor of more than 2^32 elements: its last ones, and the random numbers there."""
    import transformer_xl_relative_rel_gb300 as txl
    n = 2 ** 32 + 5000
    zeros = lambda dt, s=n: torch.zeros(s, dtype=dt, device="cuda")
    model = dict(params=[zeros(BF)], grads=[zeros(BF)], exp_avgs=[zeros(E4M3)], exp_avg_sqs=[zeros(E4M3)],
                 masters=[None], exp_avg_scales=[zeros(F32, (n + 255) // 256)],
                 exp_avg_sq_scales=[zeros(F32, (n + 255) // 256)])
    tail = _model([5000], 20, [(BF, False, BF, 8)])
    ends = {}
    for name in model:
        if model[name][0] is None:
            continue
        size = tail[name][0].numel()
        ends[name] = [model[name][0][-size:]]
        ends[name][0].copy_(tail[name][0])
    ends["masters"] = [None]
    _step(model, decay=0.0)
    torch.cuda.synchronize()
    um, uv = random_fractions(99, 0, HYPER["step"], 5000, "cuda", first=2 ** 32)
    m, v = _dense(tail["exp_avgs"][0], tail["exp_avg_scales"][0]), _dense(tail["exp_avg_sqs"][0], tail["exp_avg_sq_scales"][0]) ** 2
    want, tol = adamw_reference(tail["params"][0], tail["grads"][0], m, v, HYPER["lr"], HYPER["step"], HYPER["beta1"],
                                HYPER["beta2"], HYPER["eps"], 0.0)
    got = ends["params"][0].double()
    assert ((got - want["p"]).abs() <= tol["p"] + U[BF] * want["p"].abs() * (1 + 2 * H)).all()
    check_codes(ends["exp_avgs"][0], ends["exp_avg_scales"][0], want["m"], tol["m"], um, False)
    root = want["v"].sqrt()
    check_codes(ends["exp_avg_sqs"][0], ends["exp_avg_sq_scales"][0], root, 12 * H * root, uv, True)
    norm, _ = txl.grad_norm(txl.AdamwTensors(**model), 1.0)
    assert abs(float(norm) - float(tail["grads"][0].double().norm())) <= 64 * H * float(norm)
    assert not model["params"][0][:2 ** 31].any()


def test_oracle():
    import numpy as np
    import oracle
    model = _model([700], 21, KINDS["f32"])
    before = _copy(model)
    _step(model, factor=0.5, decay=0.2)
    f = lambda n: before[n][0].double().cpu().numpy()
    want = oracle.adamw(f("params"), f("grads"), f("exp_avgs"), f("exp_avg_sqs"), HYPER["lr"], HYPER["step"],
                        HYPER["beta1"], HYPER["beta2"], HYPER["eps"], 0.2, 0.5)
    for name, x in zip(("params", "exp_avgs", "exp_avg_sqs"), want):
        assert np.allclose(model[name][0].cpu().numpy(), x, rtol=1e-5, atol=1e-9)
    u = oracle.moment_bits(99, 2, 7, 50)
    w = random_fractions(99, 2, 7, 50, "cpu")
    assert np.array_equal(u[0], w[0].numpy()) and np.array_equal(u[1], w[1].numpy())
