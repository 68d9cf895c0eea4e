"""Measured cases of what a training step needs around the attention and the
output layer: the token embedding and its table's gradient, layer norm over a
residual sum with its gradients, and the optimiser step (AdamW over all of a
model's tensors, states in 32 or 8 bits, with the gradients' global norm).

A case names the operator (``op``), whether the backward pass is wanted
(``train``), the element type and sizes.  ``run`` computes the plain form with
elementary torch operations in fp32, or, where ``own`` is true, calls the
library.
"""
import math

import torch

own = False

BF16, F32 = "bf16", "f32"
DTYPES = {BF16: torch.bfloat16, F32: torch.float32}
BETA1, BETA2, EPS = 0.9, 0.999, 1e-8
BLOCK = 256          # elements that share a scale of an 8-bit state
TOP = 448.0          # the largest e4m3 value


def _embed(name, train, dtype, rows, d_model, vocab, accumulate=False):
    return dict(name=name, op="embed", train=train, dtype=dtype, rows=rows, d_model=d_model, vocab=vocab,
                accumulate=accumulate)


def _norm(name, train, dtype, rows, d_model, pre=False):
    return dict(name=name, op="norm", train=train, dtype=dtype, rows=rows, d_model=d_model, pre=pre)


def _adamw(name, bits, dtype, layers, d_model, vocab, clip):
    return dict(name=name, op="adamw", bits=bits, dtype=dtype, layers=layers, d_model=d_model, vocab=vocab, clip=clip)


def listed():
    return [
        # one generated token of a character model: launch latency
        _embed("embed_one_token", False, BF16, 1, 512, 256),
        # character training (22 x 768 tokens): few tokens of many rows each, added to the tied output layer's gradient
        _embed("embed_train_char", True, BF16, 22 * 768, 512, 256, True),
        # base-LM training (d_model 410, 60 x 150 tokens): odd pitch, odd vocabulary
        _embed("embed_train_base", True, BF16, 60 * 150, 410, 50021),
        # large-LM training (16 x 384 tokens): the table's bytes
        _embed("embed_train_large", True, BF16, 16 * 384, 1024, 131072),
        # the norm after one generated token's sub-layer
        _norm("norm_one_token", False, BF16, 1, 512),
        # after a character model's sub-layer, x + f(x) normalised
        _norm("norm_train_char", True, BF16, 22 * 768, 512),
        # before a large model's sub-layer: the sum is kept, its gradient has a second path
        _norm("norm_train_pre", True, BF16, 16 * 384, 1024, True),
        # fp32, ragged
        _norm("norm_train_f32", True, F32, 1111, 410),
        # a small fp32 model: launch latency
        _adamw("adamw_small", 32, F32, 2, 128, 256, False),
        # large-LM (18 layers, d_model 1024): bf16 weights with fp32 masters, clipped
        _adamw("adamw_large", 32, BF16, 18, 1024, 131072, True),
        # character model (24 layers, d_model 512), states in 8 bits, clipped
        _adamw("adamw_char_8bit", 8, BF16, 24, 512, 256, True),
        # base-LM (16 layers, d_model 410), states in 8 bits: tensors that end inside a block
        _adamw("adamw_base_8bit", 8, BF16, 16, 410, 50021, False),
    ]


def draw(rng):
    def log_uniform(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["embed", "norm", "adamw"])
    dtype = BF16 if rng.random() < 0.75 else F32
    # aligned widths and odd ones (heads x head size, unaligned pitches)
    d_model = rng.choice([64, 128, 256, 410, 512, 768, 1024, rng.randrange(33, 1024)])
    if op == "adamw":
        layers = log_uniform(1, 24)
        most = 18 * 5 * 1024 ** 2 + 131072 * 1024        # the largest listed case's weights
        vocab = min(log_uniform(130, 131072), max(130, (most - 5 * layers * d_model ** 2) // d_model // 2))
        return dict(op=op, bits=rng.choice([8, 32]), dtype=dtype, layers=layers, d_model=d_model, vocab=vocab,
                    clip=rng.random() < 0.5)
    train = rng.random() < 0.75
    rows = log_uniform(1, 32768)
    if op == "norm":
        return dict(op=op, train=train, dtype=dtype, rows=rows, d_model=rng.choice([d_model, 2 * d_model]),
                    pre=rng.random() < 0.5)
    return dict(op=op, train=train, dtype=dtype, rows=rows, d_model=d_model, vocab=log_uniform(130, 131072),
                accumulate=rng.random() < 0.5)


def _shapes(case):
    """The tensors of a model: per layer the projections, the global biases
    and two norms, then the tied embedding and the output bias."""
    d, out = case["d_model"], []
    for _ in range(case["layers"]):
        out += [(d, d)] * 5 + [(d,)] * 6
    return out + [(case["vocab"], d), (case["vocab"],)]


def _layout(case):
    """(shape, elements, first element) of each tensor in a flat buffer, and the buffer's size."""
    at, out = 0, []
    for shape in _shapes(case):
        n = math.prod(shape)
        out.append((shape, n, at))
        at += (n + BLOCK - 1) // BLOCK * BLOCK
    return out, at


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    dt = DTYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, device="cuda", generator=g)

    def uniform(*shape):
        return torch.rand(*shape, device="cuda", generator=g)

    s = dict(case=dict(case))
    if case["op"] == "embed":
        n, d, v = case["rows"], case["d_model"], case["vocab"]
        # tokens by Zipf's law, and padding rows in a batch
        tok = (v ** uniform(n).double()).long().clamp_(1, v) - 1
        if n > 8:
            tok = torch.where(uniform(n) > 0.05, tok, torch.full_like(tok, -100))
        s.update(tokens=tok, table=(normal(v, d) / math.sqrt(d)).to(dt), scale=math.sqrt(d))
        if case["train"]:
            s["dout"] = (normal(n, d) / n).to(dt)
            # the tied output layer's gradient, which the table's is added to
            s["dtable"] = ((normal(v, d) / n).to(dt) if case["accumulate"] else torch.empty_like(s["table"]))
        return s
    if case["op"] == "norm":
        n, d = case["rows"], case["d_model"]
        s.update(x=(normal(n, d) + 0.5).to(dt), residual=(0.5 * normal(n, d)).to(dt), gamma=1 + 0.2 * normal(d),
                 beta=0.1 * normal(d), eps=1e-5)
        if case["train"]:
            s["dy"] = normal(n, d).to(dt)
            s["dsum"] = normal(n, d).to(dt) if case["pre"] else None
        return s
    layout, total = _layout(case)
    live = torch.zeros(total, dtype=torch.bool, device="cuda")
    decay = torch.zeros(total, device="cuda")
    for shape, n, at in layout:
        live[at:at + n] = True
        decay[at:at + n] = 0.01 if len(shape) == 2 else 0.0      # matrices decay, vectors do not

    def flat(x):
        return torch.where(live, x, torch.zeros_like(x))

    weights = flat(0.02 * normal(total))
    s.update(layout=layout, param=weights.to(dt), grad=flat(1e-3 * normal(total)).to(dt))
    s["master"] = weights if dt == torch.bfloat16 else None
    if case["bits"] == 32:
        s.update(exp_avg=flat(3e-4 * normal(total)), exp_avg_sq=flat((5e-4 + 1e-3 * uniform(total)) ** 2))
        s["exp_avg_scale"] = s["exp_avg_sq_scale"] = None
    else:
        e4m3 = torch.float8_e4m3fn
        s.update(exp_avg=flat((120 * normal(total)).clamp_(-TOP, TOP)).to(e4m3),
                 exp_avg_sq=flat(100 + 348 * uniform(total)).to(e4m3),
                 exp_avg_scale=2e-6 * (0.5 + uniform(total // BLOCK)),
                 exp_avg_sq_scale=4e-6 * (0.5 + uniform(total // BLOCK)))
        # each element's tensor and its place there, for the random numbers
        starts = torch.tensor([at for _, _, at in layout], device="cuda")
        place = torch.arange(total, device="cuda")
        s["tensor"] = torch.searchsorted(starts, place, right=True) - 1
        s["index"] = place - starts[s["tensor"]]
    s.update(decay=decay, weight_decay=[0.01 if len(shape) == 2 else 0.0 for shape, _, _ in layout], lr=2.5e-4, step=1000,
             seed=1234567 + int(seed), max_norm=0.25)
    return s


# ------------------------------------------------------------------ plain forms

def _plain_embed(s):
    c, dt = s["case"], s["table"].dtype
    good = ((s["tokens"] >= 0) & (s["tokens"] < c["vocab"]))[:, None]
    at = s["tokens"].clamp(0, c["vocab"] - 1)
    rows = s["table"][at].float() * s["scale"]
    out = dict(out=torch.where(good, rows, torch.zeros_like(rows)).to(dt))
    if c["train"]:
        dout = s["dout"].float()
        acc = torch.zeros(c["vocab"], c["d_model"], device=dout.device)
        acc.index_add_(0, at, torch.where(good, dout, torch.zeros_like(dout)))
        acc *= s["scale"]
        if c["accumulate"]:
            acc += s["dtable"].float()
        s["dtable"].copy_(acc)
        out["dtable"] = s["dtable"]
    return out


def _plain_norm(s):
    c, dt = s["case"], s["x"].dtype
    a = s["x"].float() + s["residual"].float()
    out = dict()
    if c["pre"]:
        out["sum"] = a.to(dt)
        a = out["sum"].float()
    mean = a.mean(1, keepdim=True)
    rstd = ((a - mean).square().mean(1, keepdim=True) + s["eps"]).rsqrt()
    hat = (a - mean) * rstd
    out.update(y=(hat * s["gamma"] + s["beta"]).to(dt), mean=mean[:, 0], rstd=rstd[:, 0])
    if c["train"]:
        dy = s["dy"].float()
        t = dy * s["gamma"]
        dx = rstd * (t - t.mean(1, keepdim=True) - hat * (t * hat).mean(1, keepdim=True))
        if s["dsum"] is not None:
            dx = dx + s["dsum"].float()
        out.update(dx=dx.to(dt), dgamma=(dy * hat).sum(0), dbeta=dy.sum(0))
    return out


def _mix(x):
    """A mixing permutation of 32-bit numbers, here in int64 tensors."""
    x = x & 0xffffffff
    x = ((x ^ (x >> 16)) * 0x7feb352d) & 0xffffffff
    x = ((x ^ (x >> 15)) * 0x846ca68b) & 0xffffffff
    return x ^ (x >> 16)


def _random(seed, tensor, step, index):
    """Two uniform 16-bit fractions for each element of a tensor."""
    h = _mix(_mix(_mix(_mix(_mix(seed) + (seed >> 32)) + tensor) + step) + index)
    return (h & 0xffff).float() / 65536, (h >> 16).float() / 65536


def _plain_quantise(x, u, keep):
    """x rounded up or down to e4m3 times its block's scale, by the random
    fractions u; ``keep``: what is not zero does not become zero."""
    b = x.view(-1, BLOCK)
    top = b.abs().amax(1, keepdim=True)
    top = torch.where(top < 2.0 ** -100, torch.zeros_like(top), top)
    inverse = torch.where(top > 0, TOP / top, torch.zeros_like(top))
    y = (b * inverse).view(-1)
    exponent = torch.frexp(y)[1].clamp(min=-5) - 1
    unit = torch.ldexp(torch.ones_like(y), exponent - 3)
    steps = (y.abs() / unit + u).floor()
    if keep:
        steps = torch.where(y > 0, steps.clamp(min=1), steps)
    value = (steps * unit).clamp(max=TOP)
    return torch.where(y < 0, -value, value).to(torch.float8_e4m3fn), (top / TOP)[:, 0]


def _plain_step(s, factor):
    """The step over the flat buffers, in place (what lies between two tensors
    is zero and stays zero)."""
    p = s["param"] if s["master"] is None else s["master"]
    grad = s["grad"].float() * factor
    m, v = s["exp_avg"].float(), s["exp_avg_sq"].float()
    if s["case"]["bits"] == 8:
        m = (m.view(-1, BLOCK) * s["exp_avg_scale"][:, None]).view(-1)
        v = (v.view(-1, BLOCK) * s["exp_avg_sq_scale"][:, None]).view(-1).square()
    m = BETA1 * m + (1 - BETA1) * grad
    v = BETA2 * v + (1 - BETA2) * grad * grad
    update = (m / (1 - BETA1 ** s["step"])) / ((v / (1 - BETA2 ** s["step"])).sqrt() + EPS)
    p.copy_(p * (1 - s["lr"] * s["decay"]) - s["lr"] * update)
    if s["master"] is not None:
        s["param"].copy_(p)
    if s["case"]["bits"] == 8:
        um, uv = _random(s["seed"], s["tensor"], s["step"], s["index"])
        m, scale = _plain_quantise(m, um, False)
        s["exp_avg_scale"].copy_(scale)
        v, scale = _plain_quantise(v.sqrt(), uv, True)
        s["exp_avg_sq_scale"].copy_(scale)
    s["exp_avg"].copy_(m)
    s["exp_avg_sq"].copy_(v)


def _state_of(s):
    names = ("param", "master", "exp_avg", "exp_avg_sq", "exp_avg_scale", "exp_avg_sq_scale")
    return {name: s[name] for name in names if s[name] is not None}


def _plain_adamw(s):
    out, factor = dict(), 1.0
    if s["case"]["clip"]:
        # (what lies between the tensors is zero)
        norm = s["grad"].float().square().sum(dtype=torch.float64).sqrt().float().view(1)
        factor = (s["max_norm"] / norm).clamp(max=1.0)
        out.update(norm=norm, clip=factor)
    _plain_step(s, factor)
    out.update(_state_of(s))
    return out


# ------------------------------------------------------------------ the library's calls

def _own_embed(s):
    import transformer_xl_relative_rel_gb300 as txl
    c = s["case"]
    if "out" not in s:
        s["out"] = dict(out=torch.empty(c["rows"], c["d_model"], dtype=s["table"].dtype, device="cuda"))
        if c["train"]:
            code = txl.TXL_BF16 if s["table"].dtype == torch.bfloat16 else txl.TXL_F32
            size = txl.embed_bwd_workspace_bytes(c["rows"], c["d_model"], c["vocab"], code)
            s["workspace"] = torch.empty(size, dtype=torch.uint8, device="cuda")
            s["out"]["dtable"] = s["dtable"]
    out = s["out"]
    txl.embed_fwd(s["tokens"], s["table"], s["scale"], out=out["out"])
    if c["train"]:
        txl.embed_bwd(s["tokens"], s["dout"], out["dtable"], s["scale"], accumulate=c["accumulate"],
                      workspace=s["workspace"])
    return out


def _own_norm(s):
    import transformer_xl_relative_rel_gb300 as txl
    c, x = s["case"], s["x"]
    if "out" not in s:
        f32 = dict(dtype=torch.float32, device="cuda")
        out = dict(y=torch.empty_like(x), mean=torch.empty(c["rows"], **f32), rstd=torch.empty(c["rows"], **f32))
        if c["pre"]:
            out["sum"] = torch.empty_like(x)
        if c["train"]:
            out.update(dx=torch.empty_like(x), dgamma=torch.empty(c["d_model"], **f32),
                       dbeta=torch.empty(c["d_model"], **f32))
            code = txl.TXL_BF16 if x.dtype == torch.bfloat16 else txl.TXL_F32
            size = txl.layer_norm_bwd_workspace_bytes(c["rows"], c["d_model"], code)
            s["workspace"] = torch.empty(size, dtype=torch.uint8, device="cuda")
        s["out"] = out
    out = s["out"]
    txl.layer_norm_fwd(x, s["gamma"], s["beta"], residual=s["residual"], eps=s["eps"], y=out["y"], sum=out.get("sum"),
                       mean=out["mean"], rstd=out["rstd"])
    if c["train"]:
        # what was normalised: the kept sum, or the two summands again
        a, b = (out["sum"], None) if c["pre"] else (x, s["residual"])
        txl.layer_norm_bwd(s["dy"], a, out["mean"], out["rstd"], gamma=s["gamma"], residual=b, dsum=s["dsum"],
                           grads=out, workspace=s["workspace"])
    return out


def _own_adamw(s):
    import transformer_xl_relative_rel_gb300 as txl
    if "tensors" not in s:
        def views(name, per=1):
            if s[name] is None:
                return None
            return [s[name][at // per:at // per + (n + per - 1) // per] for _, n, at in s["layout"]]

        s["tensors"] = txl.AdamwTensors(
            views("param"), views("grad"), views("exp_avg"), views("exp_avg_sq"), masters=views("master"),
            exp_avg_scales=views("exp_avg_scale", BLOCK), exp_avg_sq_scales=views("exp_avg_sq_scale", BLOCK),
            weight_decay=s["weight_decay"])
        s["out"] = _state_of(s)
        if s["case"]["clip"]:
            s["out"].update(norm=torch.empty(1, device="cuda"), clip=torch.empty(1, device="cuda"))
            s["workspace"] = torch.empty(txl.grad_norm_workspace_bytes(s["tensors"]), dtype=torch.uint8, device="cuda")
    out = s["out"]
    if s["case"]["clip"]:
        txl.grad_norm(s["tensors"], s["max_norm"], norm=out["norm"], clip=out["clip"], workspace=s["workspace"])
    txl.adamw_step(s["tensors"], s["lr"], s["step"], beta1=BETA1, beta2=BETA2, eps=EPS, grad_scale=out.get("clip"),
                   seed=s["seed"])
    return out


def run(state):
    op = state["case"]["op"]
    if own:
        return _own_embed(state) if op == "embed" else _own_norm(state) if op == "norm" else _own_adamw(state)
    return _plain_embed(state) if op == "embed" else _plain_norm(state) if op == "norm" else _plain_adamw(state)


def work(case):
    e = 2 if case["dtype"] == BF16 else 4
    if case["op"] == "embed":
        n, d, v = case["rows"], case["d_model"], case["vocab"]
        # different tokens among n by Zipf's law: each one's row is read once
        t = torch.arange(1, v, dtype=torch.float64)
        distinct = int((1 - (1 - ((t + 1) / t).log() / math.log(v)) ** n).sum()) + 1
        nbytes, flops = e * d * (distinct + n) + 8 * n, n * d
        if case["train"]:
            nbytes += e * d * (n + (2 * distinct if case["accumulate"] else v))
            flops += 2 * n * d
        return dict(bytes=nbytes, flops=flops)
    if case["op"] == "norm":
        n, d = case["rows"], case["d_model"]
        nbytes, flops = n * d * e * (4 if case["pre"] else 3) + 8 * n + 8 * d, 9 * n * d
        if case["train"]:
            nbytes += n * d * e * 4 + 8 * n + 12 * d
            flops += 16 * n * d
        return dict(bytes=nbytes, flops=flops)
    n = sum(math.prod(shape) for shape in _shapes(case))
    # weights (and masters) read and written or written, gradients read, states read and written
    per = (2 + 8 if case["dtype"] == BF16 else 8) + e + (16 if case["bits"] == 32 else 4 + 16 / BLOCK)
    return dict(bytes=n * per, flops=16 * n)


# ------------------------------------------------------------------ values in 64 bits

def _exact_embed(case, s):
    c = case
    table, tok = s["table"].double(), s["tokens"]
    rows = torch.nonzero((tok >= 0) & (tok < c["vocab"]))[:, 0]
    res = torch.zeros(c["rows"], c["d_model"], dtype=torch.float64, device=tok.device)
    res[rows] = table[tok[rows]] * s["scale"]
    out = dict(out=res)
    if c["train"]:
        # sums over sorted tokens by differences of running sums would lose bits: by runs instead
        order = rows[torch.sort(tok[rows], stable=True).indices]
        names, counts = torch.unique_consecutive(tok[order], return_counts=True)
        grad = torch.zeros_like(table)
        if len(rows):
            grad[names] = torch.segment_reduce(s["dout"].double()[order], "sum", lengths=counts, axis=0)
        grad *= s["scale"]
        out["dtable"] = grad + s["dtable"].double() if c["accumulate"] else grad
    return out


def _exact_norm(case, s):
    a = s["x"].double() + s["residual"].double()
    out = dict()
    if case["pre"]:
        out["sum"] = a
        a = a.float().to(s["x"].dtype).double()     # the stored sum is what is normalised
    mean = a.sum(1) / case["d_model"]
    var = (a * a).sum(1) / case["d_model"] - mean * mean
    rstd = 1 / torch.sqrt(var + s["eps"])
    hat = torch.einsum("nd,n->nd", a - mean[:, None], rstd)
    gamma = s["gamma"].double()
    out.update(y=hat * gamma + s["beta"].double(), mean=mean, rstd=rstd)
    if case["train"]:
        dy = s["dy"].double()
        t = torch.einsum("nd,d->nd", dy, gamma)
        along = torch.einsum("nd,nd->n", t, hat) / case["d_model"]
        dx = (t - t.sum(1)[:, None] / case["d_model"] - along[:, None] * hat) * rstd[:, None]
        out["dx"] = dx if s["dsum"] is None else dx + s["dsum"].double()
        out["dgamma"] = torch.einsum("nd,nd->d", dy, hat)
        out["dbeta"] = torch.einsum("nd->d", dy)
    return out


def _exact_round(y, u, floor_at):
    """|y| (at most 448) to a neighbour in e4m3: up where the fraction of the
    way to the next value and u make a whole."""
    mag = y.abs()
    exponent = torch.floor(torch.log2(mag.clamp(min=2.0 ** -6))).clamp(-6, 8)
    unit = torch.ldexp(torch.ones_like(mag), exponent.int() - 3)
    low = torch.floor(mag / unit)
    steps = low + ((mag / unit - low) + u >= 1)
    value = torch.minimum(torch.maximum(steps * unit, floor_at), torch.full_like(mag, TOP))
    return torch.sign(y) * value


def _exact_adamw(case, s):
    total = s["grad"].numel()
    device = s["grad"].device
    counts = torch.tensor([n for _, n, _ in s["layout"]], device=device)
    starts = torch.tensor([at for _, _, at in s["layout"]], device=device)
    span = torch.diff(starts, append=torch.tensor([total], device=device))
    tensor = torch.repeat_interleave(torch.arange(len(counts), device=device), span)
    index = torch.arange(total, device=device) - starts[tensor]
    live = index < counts[tensor]
    decay = torch.tensor(s["weight_decay"], dtype=torch.float64, device=device)[tensor]
    p = (s["param"] if s["master"] is None else s["master"]).double()
    grad = s["grad"].double()
    out = dict()
    if case["clip"]:
        norm = torch.linalg.vector_norm(grad).view(1)
        out.update(norm=norm, clip=torch.clamp(s["max_norm"] / norm, max=1.0))
        grad = grad * out["clip"]
    m, v = s["exp_avg"].double(), s["exp_avg_sq"].double()
    if case["bits"] == 8:
        m = m * s["exp_avg_scale"].double().repeat_interleave(BLOCK)
        v = (v * s["exp_avg_sq_scale"].double().repeat_interleave(BLOCK)) ** 2
    m = m * BETA1 + grad * (1 - BETA1)
    v = v * BETA2 + grad ** 2 * (1 - BETA2)
    t = s["step"]
    denominator = torch.sqrt(v) / math.sqrt(1 - BETA2 ** t) + EPS
    p = p - s["lr"] * (decay * p + m / (1 - BETA1 ** t) / denominator)
    p = torch.where(live, p, torch.zeros_like(p))
    out["param"] = p
    if s["master"] is not None:
        out["master"] = p
    if case["bits"] == 32:
        out.update(exp_avg=m, exp_avg_sq=v)
        return out
    word = 0xffffffff

    def mixed(x):
        for shift, factor in ((16, 0x7feb352d), (15, 0x846ca68b)):
            x = ((x ^ (x >> shift)) * factor) & word
        return x ^ (x >> 16)

    base = mixed((mixed(s["seed"] & word) + (s["seed"] >> 32)) & word)
    h = mixed((mixed((mixed((base + tensor) & word) + t) & word) + index) & word)
    zero = torch.zeros_like(m)
    for name, x, bits in (("exp_avg", m, h & 0xffff), ("exp_avg_sq", v.sqrt(), h >> 16)):
        top = x.view(-1, BLOCK).abs().max(1).values
        out[name + "_scale"] = top / TOP
        y = x / torch.where(top > 0, top / TOP, torch.ones_like(top)).repeat_interleave(BLOCK)
        least = zero if name == "exp_avg" else torch.where(x > 0, zero + 2.0 ** -9, zero)
        out[name] = _exact_round(y, bits.double() / 65536, least)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"embed": _exact_embed, "norm": _exact_norm, "adamw": _exact_adamw}[case["op"]](case, s)
