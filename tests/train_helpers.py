"""The embedding, layer norm and optimiser step in float64 torch (the oracle's
formulas, vectorised) and elementwise bounds on what the library's arithmetic
may be off.  One fp32 operation is off by at most h = 2^-24 of its result, a
rounding to bf16 by 2^-8.

Embedding: a product and a rounding; a gradient's n additions are each off by
h times a partial sum, at most the sum of absolute values, then a product, an
addition (accumulating) and a rounding.

Layer norm, per row, a = max |s|: a sum over a row adds at most 32 values in a
thread and then in trees of at most 5 + 5 + 5 levels, and s itself is rounded
once: mean, and s - mean with it, is off by at most 64 h a.  With
c = 64 h a rstd, rstd is off by c + 2^-19 of itself (var's own sum 48 h, rsqrt
and the division 4 h, halved; the rest is slack for c's square), and xh by
c + |xh| (c + 2^-19).  The backward's sums over a row add as the mean's; sums over
rows add at most rows / 152 + 64 terms one after another.

Optimiser: moments take three products, an addition and betas rounded to fp32
(8 h of the terms' sizes); an update's factors (1 - beta^t by expm1, its
root, the root of v, a division) are off by at most 48 h together.
"""
import torch

H = 2.0 ** -24
U = {torch.bfloat16: 2.0 ** -8, torch.float32: H}
F32, BF = torch.float32, torch.bfloat16


def embed_reference(tokens, table, scale, dout=None, dtable=None):
    """tokens [n], table [v, d]; dtable: what the gradient is added to."""
    v, dt = table.shape[0], table.dtype
    good = (tokens >= 0) & (tokens < v)
    at = tokens.clamp(0, v - 1)
    out = torch.where(good[:, None], scale * table.double()[at], torch.zeros((), dtype=torch.float64, device=table.device))
    want, tol = dict(out=out), dict(out=out.abs() * (U[dt] * (1 + 2 * H) + 2 * H))
    if dout is None:
        return want, tol
    rows = torch.nonzero(good)[:, 0]
    grad, size = (torch.zeros(table.shape, dtype=torch.float64, device=table.device) for _ in range(2))
    count = torch.zeros(v, dtype=torch.float64, device=table.device)
    g = dout[rows].double()
    grad.index_add_(0, tokens[rows], g)
    size.index_add_(0, tokens[rows], g.abs())
    count.index_add_(0, tokens[rows], torch.ones_like(g[:, 0]))
    grad, size = grad * scale, size * abs(scale)
    if dtable is not None:
        grad = grad + dtable.double()
    # the table's gradient (for the tests also the tokens that have no row)
    err = (count[:, None] + 4) * H * size + 2 * H * grad.abs()
    want["dtable"], tol["dtable"] = grad, err + U[dt] * (grad.abs() + err)
    return want, tol


def norm_reference(x, gamma, beta, eps, residual=None, keep_sum=False, dy=None, dsum=None):
    d, dt = x.shape[1], x.dtype
    s = x.double() if residual is None else x.double() + residual.double()
    want, tol = dict(), dict()
    if keep_sum:
        want["sum"] = (x.float() if residual is None else x.float() + residual.float()).to(dt).double()
        tol["sum"] = torch.zeros_like(s)
        s = want["sum"]
    mean = s.mean(1, keepdim=True)
    rstd = ((s - mean).square().mean(1, keepdim=True) + eps).rsqrt()
    hat = (s - mean) * rstd
    a = s.abs().amax(1, keepdim=True)
    c = 64 * H * a * rstd
    e_hat = c + hat.abs() * (c + 2.0 ** -19)
    one = torch.ones(d, dtype=torch.float64, device=x.device)
    gm = one if gamma is None else gamma.double()
    bt = 0 * one if beta is None else beta.double()
    y = hat * gm + bt
    want.update(y=y, mean=mean[:, 0], rstd=rstd[:, 0])
    err = gm.abs() * e_hat + 2 * H * (y.abs() + bt.abs())
    tol.update(y=err + U[dt] * (y.abs() + err), mean=(64 * H * a)[:, 0], rstd=(rstd * (c + 2.0 ** -19))[:, 0])
    if dy is None:
        return want, tol
    dy = dy.double()
    g = dy * gm
    m1, m2 = g.mean(1, keepdim=True), (g * hat).mean(1, keepdim=True)
    d0 = rstd * (g - m1 - hat * m2)
    add = 0 * d0 if dsum is None else dsum.double()
    dx = d0 + add
    e1 = 64 * H * g.abs().mean(1, keepdim=True)
    e2 = (g.abs() * e_hat).mean(1, keepdim=True) + 64 * H * (g * hat).abs().mean(1, keepdim=True)
    size = g.abs() + m1.abs() + (hat * m2).abs()
    err = rstd * (e1 + e_hat * m2.abs() + hat.abs() * e2 + e_hat * e2 + 8 * H * size) + \
        (c + 2.0 ** -19) * rstd * size + 2 * H * (add.abs() + dx.abs())
    want.update(dx=dx, dgamma=(dy * hat).sum(0), dbeta=dy.sum(0))
    steps = (x.shape[0] / 152 + 64) * H
    tol.update(dx=err + U[dt] * (dx.abs() + err),
               dgamma=(dy.abs() * e_hat).sum(0) + steps * (dy * hat).abs().sum(0), dbeta=steps * dy.abs().sum(0))
    return want, tol


def adamw_reference(p, grad, m, v, lr, step, beta1, beta2, eps, decay, factor=1.0):
    """The new (p, m, v) of flat tensors in float64 and their bounds."""
    p, g, m, v = (x.double() for x in (p, grad, m, v))
    g = g * factor
    m1, v1 = beta1 * m + (1 - beta1) * g, beta2 * v + (1 - beta2) * g * g
    em = 8 * H * (beta1 * m.abs() + (1 - beta1) * g.abs())
    ev = 8 * H * v1
    c1, c2 = 1 - beta1 ** step, 1 - beta2 ** step
    den = (v1 / c2).sqrt() + eps
    up = m1 / c1 / den
    e_up = em / c1 / den + 48 * H * up.abs()
    new = p - lr * (decay * p + up)
    ep = lr * (e_up + 4 * H * (decay * p.abs() + up.abs())) + 2 * H * new.abs()
    return dict(p=new, m=m1, v=v1), dict(p=ep, m=em, v=ev)


def random_fractions(seed, tensor, step, n, device, first=0):
    """oracle.moment_bits as torch tensors."""
    word = 0xffffffff

    def mix(x):
        x = ((x ^ (x >> 16)) * 0x7feb352d) & word
        x = ((x ^ (x >> 15)) * 0x846ca68b) & word
        return x ^ (x >> 16)

    key = mix((mix((mix((mix(seed & word) + (seed >> 32)) & word) + tensor) & word) + step) & word)
    i = torch.arange(first, first + n, device=device)
    h = mix((key + i + (i >> 32) * 0x9e3779b9) & word)
    return (h & 0xffff).double() / 65536, (h >> 16).double() / 65536


def check_codes(codes, scales, x, ex, u, keep, what=""):
    """Codes (float8_e4m3fn) and scales of a tensor's new moment x (float64,
    off by at most ex in the library's fp32)."""
    n = x.numel()
    pad = torch.nn.functional.pad
    blocks = lambda t: pad(t, (0, -n % 256)).view(-1, 256)
    xb = blocks(x)
    top = xb.abs().amax(1)
    live = top >= 2.0 ** -100
    top = torch.where(live, top, torch.zeros_like(top))
    e_top = torch.where(live, blocks(ex).amax(1), torch.zeros_like(top))
    off = (scales.double() - top / 448).abs() - (e_top / 448 + 4 * H * top / 448)
    assert scales.numel() == 0 or float(off.max()) <= 1e-44, f"{what}: scales"
    inverse = torch.where(live, 448 / top.clamp(min=1e-300), torch.zeros_like(top))
    rep = lambda t: t.repeat_interleave(256)[:n]
    y = x * rep(inverse)
    e = torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6)))
    unit = ((e.long() - 3 + 1023) << 52).view(torch.float64)      # 2^(e - 3) (** and ldexp are not exact on a GPU)
    steps = y.abs() / unit + u
    # y's error: the moment's, the largest one's, two roundings
    slack = ((ex * rep(inverse)) + y.abs() * (rep(e_top / top.clamp(min=1e-300)) + 4 * H)) / unit + 20 * H
    got = codes.double()
    assert torch.equal(torch.sign(got)[got != 0], torch.sign(x)[got != 0]), f"{what}: signs"

    def value(k):
        k = torch.floor(k)
        if keep:
            k = torch.where((y > 0) & (k < 1), torch.ones_like(k), k)
        return (k * unit).clamp(max=448.0)

    low, high = value(steps - slack), value(steps + slack)
    # (near a power of two y may lie on the other side, where steps differ in size: the neighbour's value)
    edge = torch.minimum((y.abs() / unit - 8).abs(), (16 - y.abs() / unit).abs()) <= slack
    fine = (got.abs() == low) | (got.abs() == high)
    near = edge & ((got.abs() - y.abs()).abs() <= unit * (1 + slack))
    bad = torch.nonzero(~(fine | near))[:, 0][:3].tolist()
    assert not bad, (what, [[float(t[b]) for t in (y, unit, u, steps, slack, got, low, high)] for b in bad])
    return float((low != high).double().mean())
