"""The output-layer losses in float64 torch (the oracle's formulas, vectorised)
and elementwise bounds on what the library's arithmetic may be off.

Bounds.  A logit is a sum of d products accumulated in fp32: at most
``acc_steps(d)`` additions, each off by at most 2^-23 of the largest partial
sum (a tensor core may truncate where it adds), which is at most
s = max sum_k |h_k w_k|.  So |delta z| <= Z = acc_steps(d) 2^-23 s, plus the
fp32 roundings of z's scaling, the bias and exp2's argument (a few 2^-23 |z|).
lse moves by at most Z + 2^-20 (the sum of positive terms, log2), loss by
twice that per unit of teacher weight, times t^2 (and Z / t).
With q = softmax, |delta q| <= q (2 Z/t + 2^-20).  dz is rounded to the
products' type (u = 2^-8 for bf16, 2^-16 with up to 128 rows, which keep it in
two bf16 parts; fp32 operands lose at most 2^-22), sums
add at most acc_steps(K) 2^-23 of the sum of absolute values, and the result
is rounded once (u of the output type).
"""
import torch

U = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
U_DZ = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -22}


def acc_steps(k):
    # an addition per 16-wide product step, six of them per step for fp32
    # operands held as three bf16 parts, or k additions half as far off
    return 8 * ((k + 15) // 16) + 16


def reference(h, w, bias, idx, weights, t, dloss=None):
    """idx [n, k] int64 with weights [n, k] float64 (0 for an entry left out);
    a row without a positive weight is empty."""
    h64, w64 = h.double(), w.double()
    live = (weights > 0).any(1)
    h64 = torch.where(live[:, None], h64, torch.zeros_like(h64)) if dloss is not None else h64
    z = h64 @ w64.t()
    if bias is not None:
        z = z + bias.double()
    z = z / t
    lse = torch.logsumexp(z, 1)
    at = idx.clamp(0, w.shape[0] - 1)
    zk = z.gather(1, at)
    logp = torch.where(weights > 0, weights.clamp(min=1e-300).log(), torch.zeros_like(weights))
    terms = torch.where(weights > 0, weights * (logp - (zk - lse[:, None])), torch.zeros_like(weights))
    ok = live & (lse != -float("inf"))
    loss = torch.where(ok, t * t * terms.sum(1), torch.zeros_like(lse))
    s = float((h64.nan_to_num().abs() @ w64.abs().t()).max()) if z.numel() else 0.0
    d = h.shape[1]
    zmax = float(z[z.isfinite()].abs().max()) if z.isfinite().any() else 0.0
    Z = acc_steps(d) * 2.0 ** -23 * s / t + 8 * 2.0 ** -23 * zmax
    tol = dict(lse=Z + 2.0 ** -20 * (1 + zmax), loss=t * t * (2 * Z + 2.0 ** -19 * (1 + zmax)))
    out = dict(loss=loss, lse=lse)
    if dloss is None:
        return out, tol
    coef = torch.where(ok, dloss.double() * t, torch.zeros_like(lse))
    q = torch.where((coef != 0)[:, None], (z - lse[:, None]).exp(), torch.zeros_like(z))
    dz = q.clone()
    dz.scatter_add_(1, at, -torch.where((coef != 0)[:, None], weights, torch.zeros_like(weights)))
    dz = dz * coef[:, None]
    out.update(dh=dz @ w64, dw=dz.t() @ h64, db=dz.sum(0))
    dt = h.dtype
    raw = coef.abs()[:, None] * q * (2 * Z + 2.0 ** -19) + dz.abs() * 2.0 ** -20
    # an entry's weight is an fp32 softmax: off by at most 2^-20 of itself
    raw.scatter_add_(1, at, coef.abs()[:, None] * weights * 2.0 ** -20)
    n, v = z.shape
    err = raw + (2.0 ** -16 if dt == torch.bfloat16 and n <= 128 else U_DZ[dt]) * dz.abs()
    tol["dh"] = err @ w64.abs() + acc_steps(v) * 2.0 ** -23 * (dz.abs() @ w64.abs()) + U[dt] * out["dh"].abs()
    tol["dw"] = err.t() @ h64.abs() + acc_steps(n) * 2.0 ** -23 * (dz.abs().t() @ h64.abs()) + U[dt] * out["dw"].abs()
    tol["db"] = raw.sum(0) + (n + 16) * 2.0 ** -23 * dz.abs().sum(0)
    return out, tol


def xent_reference(h, w, bias, target, dloss=None):
    live = (target >= 0) & (target < w.shape[0])
    return reference(h, w, bias, target[:, None], live.double()[:, None], 1.0, dloss)


def distill_reference(h, w, bias, idx, logits, t, dloss=None):
    y = logits.double() / t
    keep = (idx >= 0) & (idx < w.shape[0]) & (y != -float("inf"))
    y = torch.where(keep, y, torch.full_like(y, -float("inf")))
    p = torch.where(keep.any(1)[:, None], torch.softmax(y, 1), torch.zeros_like(y))
    return reference(h, w, bias, idx, torch.nan_to_num(p), t, dloss)


def check(got, want, tol, what=""):
    """Every element within its bound (empty slack of 1e-30 for exact zeros);
    infinities and NaN at the same places."""
    for name, ref in want.items():
        if got.get(name) is None:
            continue
        x = got[name].double().cpu()
        y = ref.cpu()
        assert x.shape == y.shape, (what, name)
        fine = torch.isfinite(y)
        assert torch.equal(torch.isfinite(x), fine), f"{what} {name}: finite elsewhere"
        assert torch.equal(x[~fine & ~y.isnan()], y[~fine & ~y.isnan()]), f"{what} {name}: infinities"
        lim = tol[name] if torch.is_tensor(tol[name]) else torch.full_like(y, tol[name])
        over = ((x - y).abs() - lim.cpu())[fine]
        assert over.numel() == 0 or float(over.max()) <= 1e-30, \
            f"{what} {name}: {float(((x - y).abs()[fine]).max()):.3e} off, {float(over.max()):.3e} over the bound"
