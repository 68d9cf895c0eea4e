"""Pins for the oracle's output-layer losses (``oracle.softmax_xent``,
``oracle.distill``): central differences of the forward for every element of
h, w and the bias; torch's float64 log_softmax and autograd; distillation with
one kept entry is cross entropy; empty rows; a planted mistake is caught."""
import numpy as np
import pytest
import torch

import oracle


def _problem(seed, n=5, d=4, v=7, k=3):
    g = np.random.Generator(np.random.PCG64(seed))
    h, w, b = g.standard_normal((n, d)), g.standard_normal((v, d)), g.standard_normal(v)
    target = g.integers(0, v, n)
    target[1] = -100
    idx = np.stack([g.permutation(v)[:k] for _ in range(n)])
    idx[2] = -1                    # an empty row
    idx[3, 1] = v                  # one entry left out
    idx[4, 1] = idx[4, 0]          # the same index twice
    y = g.standard_normal((n, k)) * 2
    y[0, 2] = -np.inf
    return h, w, b, target, idx, y, g.standard_normal(n)


def _differences(f, arrays, eps=1e-6):
    out = []
    for x in arrays:
        gx = np.zeros_like(x)
        for at in np.ndindex(*x.shape):
            keep = x[at]
            x[at] = keep + eps
            up = f()
            x[at] = keep - eps
            down = f()
            x[at] = keep
            gx[at] = (up - down) / (2 * eps)
        out.append(gx)
    return out


@pytest.mark.parametrize("op,temperature", [("xent", 1.0), ("distill", 1.0), ("distill", 2.5)])
def test_gradients_match_differences(op, temperature):
    h, w, b, target, idx, y, dloss = _problem(3)

    def call(dl=None):
        if op == "xent":
            return oracle.softmax_xent(h, w, target, bias=b, dloss=dl)
        return oracle.distill(h, w, idx, y, temperature, bias=b, dloss=dl)

    g = call(dloss)[2]
    fd = _differences(lambda: float((call()[0] * dloss).sum()), (h, w, b))
    # second-order error of the difference ~ eps^2, cancellation ~ 1e-16 / eps
    for name, d in zip(("dh", "dw", "db"), fd):
        assert np.abs(g[name] - d).max() < 1e-7, name
    # a sign or a factor of the temperature gone wrong would not pass
    assert np.abs(g["dh"] * 1.01 - fd[0]).max() > 1e-5


def test_matches_torch_in_float64():
    h, w, b, target, idx, y, dloss = _problem(4)
    th, tw, tb = (torch.from_numpy(x).requires_grad_() for x in (h, w, b))
    z = th @ tw.t() + tb
    loss, lse, g = oracle.softmax_xent(h, w, target, bias=b, dloss=dloss)
    ref = torch.nn.functional.cross_entropy(z, torch.from_numpy(target), ignore_index=-100, reduction="none")
    grads = torch.autograd.grad((ref * torch.from_numpy(dloss)).sum(), (th, tw, tb), retain_graph=True)
    assert np.abs(loss - ref.detach().numpy()).max() < 1e-12
    assert np.abs(lse - torch.logsumexp(z, 1).detach().numpy()).max() < 1e-12
    for name, t in zip(("dh", "dw", "db"), grads):
        assert np.abs(g[name] - t.numpy()).max() < 1e-12
    # whole-vocabulary teacher: torch's kl_div
    t = 2.0
    full = np.tile(np.arange(len(w)), (len(h), 1))
    yt = np.random.Generator(np.random.PCG64(9)).standard_normal(full.shape)
    loss, _, g = oracle.distill(h, w, full, yt, t, bias=b, dloss=dloss)
    ref = t * t * torch.nn.functional.kl_div(torch.log_softmax(z / t, 1), torch.softmax(torch.from_numpy(yt) / t, 1),
                                             reduction="none").sum(1)
    grads = torch.autograd.grad((ref * torch.from_numpy(dloss)).sum(), (th, tw, tb))
    assert np.abs(loss - ref.detach().numpy()).max() < 1e-12
    for name, x in zip(("dh", "dw", "db"), grads):
        assert np.abs(g[name] - x.numpy()).max() < 1e-12


def test_one_entry_is_cross_entropy_and_empty_rows():
    h, w, b, target, idx, y, dloss = _problem(5)
    a = oracle.softmax_xent(h, w, target, bias=b, dloss=dloss)
    c = oracle.distill(h, w, target[:, None], np.full((len(h), 1), 3.7), 1.0, bias=b, dloss=dloss)
    assert np.allclose(a[0], c[0], atol=1e-14) and np.allclose(a[2]["dw"], c[2]["dw"], atol=1e-14)
    assert a[0][1] == 0 and not a[2]["dh"][1].any()
    loss, _, g = oracle.distill(h, w, idx, y, 2.0, bias=b, dloss=dloss)
    assert loss[2] == 0 and not g["dh"][2].any()
    loss, lse, g = oracle.softmax_xent(h, w, target, bias=np.full(len(w), -np.inf), dloss=dloss)
    assert not loss.any() and (lse == -np.inf).all() and not g["dw"].any()
