"""Measured cases of the output-layer losses: softmax cross entropy over a
vocabulary and distillation from a teacher's top logits, each forward alone
(evaluation, scoring) and forward with backward (a training step's last layer).

A case names the operator (``op``), whether gradients are wanted (``train``),
the element type, rows (tokens), d_model, vocabulary size, whether the output
layer has a bias and, for distillation, the number of teacher entries per row
and the temperature.  ``run`` computes the plain form with elementary torch
operations in fp32, or, where ``own`` is true, calls the library.
"""
import math

import torch

own = False

BF16, F32 = "bf16", "f32"
DTYPES = {BF16: torch.bfloat16, F32: torch.float32}


def _case(name, op, train, dtype, rows, d_model, vocab, bias, top_k=1, temperature=1.0):
    return dict(name=name, op=op, train=train, dtype=dtype, rows=rows, d_model=d_model, vocab=vocab, bias=bias,
                top_k=top_k, temperature=temperature)


def listed():
    return [
        # scoring one token of a character model: launch latency
        _case("xent_eval_one_token", "xent", False, BF16, 1, 512, 256, True),
        # scoring one 128-token segment (batch 1) against a word vocabulary: the weights' bytes
        _case("xent_eval_segment", "xent", False, BF16, 128, 1024, 65536, False),
        # evaluation of a 22 x 128 batch against a large vocabulary
        _case("xent_eval_batch", "xent", False, BF16, 22 * 128, 512, 131072, True),
        # character training: many rows, a small vocabulary
        _case("xent_train_char", "xent", True, BF16, 22 * 768, 512, 256, True),
        # base-LM training (d_model 410, 60 x 150 tokens): odd pitch, odd vocabulary
        _case("xent_train_base", "xent", True, BF16, 60 * 150, 410, 50021, True),
        # large-LM training (d_model 1024, 16 x 384 tokens): the largest
        _case("xent_train_large", "xent", True, BF16, 16 * 384, 1024, 131072, False),
        # fp32 training, ragged in every size
        _case("xent_train_f32", "xent", True, F32, 1111, 410, 20011, True),
        # distillation loss of a small evaluation batch
        _case("distill_eval", "distill", False, BF16, 64, 1024, 32768, False, 8, 1.0),
        # a short ragged batch of a small student
        _case("distill_train_small", "distill", True, BF16, 257, 256, 5003, True, 16, 2.0),
        # large-LM student, 16 x 384 tokens
        _case("distill_train_large", "distill", True, BF16, 16 * 384, 1024, 32768, True, 32, 2.0),
        # long batch of a narrower student with many teacher entries
        _case("distill_train_wide", "distill", True, BF16, 16384, 512, 65536, False, 64, 4.0),
        # fp32 student, odd sizes
        _case("distill_train_f32", "distill", True, F32, 900, 512, 10007, False, 32, 3.0),
    ]


def draw(rng):
    def log_uniform(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["xent", "distill"])
    train = rng.random() < 0.6
    dtype = BF16 if rng.random() < 0.75 else F32
    # aligned widths and odd ones (heads x head size, unaligned pitches)
    d_model = rng.choice([64, 128, 256, 410, 512, 768, 1024, rng.randrange(33, 1024)])
    rows = log_uniform(1, 16384)
    # at most the largest listed case's products (fp32: a twentieth of it, its plain form is as long)
    most = 16 * 384 * 1024 * 131072 // (1 if dtype == BF16 else 20)
    vocab = min(log_uniform(130, 131072), max(130, most // (rows * d_model)))
    top_k = rng.choice([1, 2, 5, 8, 16, 32, 50, 64]) if op == "distill" else 1
    temperature = rng.choice([1.0, 1.5, 2.0, 4.0]) if op == "distill" else 1.0
    return dict(op=op, train=train, dtype=dtype, rows=rows, d_model=d_model, vocab=vocab, bias=rng.random() < 0.5,
                top_k=top_k, temperature=temperature)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    n, d, v, k = case["rows"], case["d_model"], case["vocab"], case["top_k"]
    dt = DTYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, device="cuda", generator=g)

    def uniform(*shape):
        return torch.rand(*shape, device="cuda", generator=g)

    # an output layer whose logits have a spread of about 2 and lean towards the row's own token;
    # frequent tokens have low numbers
    w = normal(v, d) * (2.0 / math.sqrt(d))
    own_token = (v * uniform(n) ** 3).long().clamp_(0, v - 1)
    h = normal(n, d) + 0.5 * w[own_token]
    state = dict(case=dict(case), h=h.to(dt), w=w.to(dt), bias=normal(v) * 0.5 if case["bias"] else None)
    counted = torch.ones(n, dtype=torch.bool, device="cuda")
    if case["train"] and n > 8:
        counted = uniform(n) > 0.05      # padding rows of a batch carry no loss
    # the gradient of a mean over the counted tokens, each with its weight
    state["dloss"] = (0.5 + uniform(n)) / counted.sum().clamp(min=1)
    if case["op"] == "xent":
        state["target"] = torch.where(counted, own_token, torch.full_like(own_token, -100))
    else:
        # k different tokens per row, in the order of the teacher's logits (largest first)
        step = max(1, v // k)
        at = torch.arange(k, device="cuda") * step + (uniform(n, k) * step).long().clamp_(0, step - 1)
        at = (at + own_token[:, None]) % (step * k)
        at = torch.gather(at, 1, uniform(n, k).argsort(1))
        state["teacher_idx"] = torch.where(counted[:, None], at, torch.full_like(at, -1)).contiguous()
        # stored in the student's type, as teachers' logits are
        state["teacher_logits"] = (normal(n, k).sort(1, descending=True).values * 3.0 + 8.0).to(dt).contiguous()
    return state


def _plain_logits(s):
    z = s["h"].float() @ s["w"].float().t()
    return z if s["bias"] is None else z + s["bias"]


def _plain_lse(z):
    m = z.max(1, keepdim=True).values
    return (m + (z - m).exp().sum(1, keepdim=True).log())[:, 0]


def _plain_grads(s, dz):
    dt = s["h"].dtype
    out = dict(dh=(dz @ s["w"].float()).to(dt), dw=(dz.t() @ s["h"].float()).to(dt))
    if s["bias"] is not None:
        out["db"] = dz.sum(0)
    return out


def _plain_xent(s):
    z = _plain_logits(s)
    lse = _plain_lse(z)
    counted = s["target"] >= 0
    at = s["target"].clamp(min=0)[:, None]
    loss = torch.where(counted, lse - z.gather(1, at)[:, 0], torch.zeros_like(lse))
    out = dict(loss=loss, lse=lse)
    if s["case"]["train"]:
        dz = (z - lse[:, None]).exp()
        dz.scatter_add_(1, at, torch.full_like(loss, -1.0)[:, None])
        dz = dz * torch.where(counted, s["dloss"], torch.zeros_like(loss))[:, None]
        out.update(_plain_grads(s, dz))
    return out


def _plain_distill(s):
    t = s["case"]["temperature"]
    z = _plain_logits(s) / t
    lse = _plain_lse(z)
    idx = s["teacher_idx"]
    listed_ = idx >= 0
    counted = listed_.any(1)
    at = idx.clamp(min=0)
    y = s["teacher_logits"].float() / t
    top = torch.where(listed_, y, torch.full_like(y, -1e30)).max(1, keepdim=True).values
    e = torch.where(listed_, (y - top).exp(), torch.zeros_like(y))
    total = torch.where(counted[:, None], e.sum(1, keepdim=True), torch.ones_like(top))
    p = e / total
    terms = p * ((y - top - total.log()) - (z.gather(1, at) - lse[:, None]))
    loss = t * t * torch.where(listed_, terms, torch.zeros_like(terms)).sum(1)
    out = dict(loss=loss, lse=lse)
    if s["case"]["train"]:
        dz = (z - lse[:, None]).exp()
        dz.scatter_add_(1, at, -p)
        dz = dz * (t * torch.where(counted, s["dloss"], torch.zeros_like(loss)))[:, None]
        out.update(_plain_grads(s, dz))
    return out


def _buffers(s):
    """The outputs and the workspace, kept by the program from its first pass on."""
    if "out" not in s:
        import transformer_xl_relative_rel_gb300 as txl
        c, h = s["case"], s["h"]
        f32 = dict(dtype=torch.float32, device=h.device)
        out = dict(loss=torch.empty(c["rows"], **f32), lse=torch.empty(c["rows"], **f32))
        if c["train"]:
            out.update(dh=torch.empty_like(h), dw=torch.empty_like(s["w"]))
            if s["bias"] is not None:
                out["db"] = torch.empty(c["vocab"], **f32)
        code = txl.TXL_BF16 if h.dtype == torch.bfloat16 else txl.TXL_F32
        if c["op"] == "xent":
            size = txl.softmax_xent_workspace_bytes(c["rows"], c["d_model"], c["vocab"], code, backward=c["train"])
        else:
            size = txl.distill_workspace_bytes(c["rows"], c["d_model"], c["vocab"], c["top_k"], code,
                                               backward=c["train"])
        s["workspace"] = torch.empty(size, dtype=torch.uint8, device=h.device)
        s["out"] = out
    return s["out"], s["workspace"]


def _own(s):
    import transformer_xl_relative_rel_gb300 as txl
    c = s["case"]
    out, ws = _buffers(s)
    if c["op"] == "xent":
        txl.softmax_xent_fwd(s["h"], s["w"], s["target"], bias=s["bias"], loss=out["loss"], lse=out["lse"],
                             workspace=ws)
        if c["train"]:
            txl.softmax_xent_bwd(s["h"], s["w"], s["target"], out["lse"], s["dloss"], bias=s["bias"], grads=out,
                                 workspace=ws)
    else:
        txl.distill_fwd(s["h"], s["w"], s["teacher_idx"], s["teacher_logits"], c["temperature"], bias=s["bias"],
                        loss=out["loss"], lse=out["lse"], workspace=ws)
        if c["train"]:
            txl.distill_bwd(s["h"], s["w"], s["teacher_idx"], s["teacher_logits"], out["lse"], s["dloss"],
                            c["temperature"], bias=s["bias"], grads=out, workspace=ws)
    return out


def run(state):
    if own:
        return _own(state)
    return _plain_xent(state) if state["case"]["op"] == "xent" else _plain_distill(state)


def work(case):
    n, d, v, k = case["rows"], case["d_model"], case["vocab"], case["top_k"]
    e = 2 if case["dtype"] == BF16 else 4
    per_row = 8 if case["op"] == "xent" else (8 + e) * k
    nbytes = e * (n * d + v * d) + n * per_row + 8 * n + (4 * v if case["bias"] else 0)
    if case["train"]:
        nbytes += e * (n * d + v * d) + 4 * n + (4 * v if case["bias"] else 0)
    # the logits, and for training the products with the weights and with the hidden states
    return dict(bytes=nbytes, flops=(3 if case["train"] else 1) * 2 * n * v * d)


def exact(case, seed):
    s = prepare(case, seed)
    h, w = s["h"].double(), s["w"].double()
    n, v, t = case["rows"], case["vocab"], float(case["temperature"])
    z = torch.einsum("nd,vd->nv", h, w)
    if s["bias"] is not None:
        z += s["bias"].double()
    z /= t
    lse = torch.logsumexp(z, 1)
    logq = z.sub_(lse[:, None])
    if case["op"] == "xent":
        good = (s["target"] >= 0) & (s["target"] < v)
        rows = torch.nonzero(good)[:, 0]
        idx = s["target"][rows][:, None]
        p = torch.ones(len(rows), 1, dtype=torch.float64, device=h.device)
    else:
        # a row is listed whole or not at all
        rows = torch.nonzero(s["teacher_idx"][:, 0] >= 0)[:, 0]
        idx = s["teacher_idx"][rows]
        p = torch.softmax(s["teacher_logits"][rows].double() / t, 1)
    loss = torch.zeros(n, dtype=torch.float64, device=h.device)
    loss[rows] = t * t * (p * (p.log() - logq[rows[:, None], idx])).sum(1)
    out = dict(loss=loss, lse=lse)
    if case["train"]:
        scale = torch.zeros(n, dtype=torch.float64, device=h.device)
        scale[rows] = t * s["dloss"][rows].double()
        dz = logq.exp_()
        dz[rows[:, None], idx] -= p      # the listed tokens of a row differ from one another
        dz *= scale[:, None]
        out["dh"] = torch.einsum("nv,vd->nd", dz, w)
        out["dw"] = torch.einsum("nv,nd->vd", dz, h)
        if s["bias"] is not None:
            out["db"] = dz.sum(0)
    return out
