"""Training steps made of the library's calls alone: tokens to embeddings, a
layer (norm, projections, relative attention, residual and norm), the output
layer's cross entropy on the tied table, the backward pass through all of
them, clipping and AdamW.  Against the same steps in float64 torch autograd."""
import pytest
import torch

import transformer_xl_relative_rel_gb300 as txl
from tests.train_helpers import BF, F32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from transformer_xl_relative_rel_gb300 import _build
    _build.build()


B, H, D, L, M, V = 3, 2, 32, 24, 8, 211
DM, T = H * D, M + L
NAMES = ("table", "w_q", "w_k", "w_v", "g1", "b1", "g2", "b2", "bias", "u", "w")
HYPER = dict(beta1=0.9, beta2=0.98, eps=1e-6)


def _weights(seed):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g)
    p = dict(table=n(V, DM) * 0.125, w_q=n(DM, DM) * 0.2, w_k=n(DM, DM) * 0.2, w_v=n(DM, DM) * 0.2, g1=1 + 0.1 * n(DM),
             b1=0.1 * n(DM), g2=1 + 0.1 * n(DM), b2=0.1 * n(DM), bias=0.1 * n(V), u=0.1 * n(H, D), w=0.1 * n(H, D))
    rel = n(T, H, D) * 0.5      # the projected relative table: given, not trained here
    return {k: v.float().cuda() for k, v in p.items()}, rel.cuda()


def _batch(seed):
    g = torch.Generator().manual_seed(seed)
    tok = (V ** torch.rand(L, B, generator=g)).long().clamp(1, V) - 1
    target = torch.randint(0, V, (L, B), generator=g)
    tok[3, 1], target[5, 2], target[0, 0] = -100, -100, V      # padding
    return tok.cuda(), target.cuda(), torch.randn(M, B, DM, generator=g).cuda()


class Step:
    """One training step's buffers and calls (fp32 or bf16 weights, the latter with fp32 masters)."""

    def __init__(self, dtype, seed, bits, biases=True):
        self.dtype, self.biases = dtype, biases
        weights, rel = _weights(seed)
        small = ("g1", "b1", "g2", "b2", "bias", "u", "w")     # vectors stay fp32
        self.master = {n: w.clone() for n, w in weights.items() if n not in small and dtype == BF}
        self.p = {n: w.to(F32 if n in small else dtype).contiguous() for n, w in weights.items()}
        self.g = {n: torch.zeros_like(w) for n, w in self.p.items()}
        self.rel = rel.to(dtype)
        zeros = lambda n, d: torch.zeros(n, dtype=d, device="cuda")
        codes = {n: bits == 8 and n not in small for n in NAMES}
        state = {n: torch.float8_e4m3fn if codes[n] else F32 for n in NAMES}
        size = {n: self.p[n].numel() for n in NAMES}
        self.m, self.v = ({n: zeros(size[n], state[n]).view(self.p[n].shape) for n in NAMES} for _ in range(2))
        self.ms, self.vs = ({n: zeros((size[n] + 255) // 256, F32) if codes[n] else None for n in NAMES} for _ in range(2))
        lists = lambda d: [d.get(n) for n in NAMES]
        self.tensors = txl.AdamwTensors(lists(self.p), lists(self.g), lists(self.m), lists(self.v), lists(self.master),
                                        lists(self.ms), lists(self.vs),
                                        weight_decay=[0.01 if self.p[n].dim() == 2 and n not in ("u", "w") else 0.0
                                                      for n in NAMES])
        self.lr = torch.tensor([0.01], device="cuda")
        self.number = torch.zeros(1, dtype=torch.int64, device="cuda")
        self.lse_a = torch.empty(B, H, L, device="cuda") if dtype == BF else None

    def __call__(self, tok, target, mem):
        p, g, dt = self.p, self.g, self.dtype
        x = txl.embed_fwd(tok, p["table"], DM ** 0.5)
        h, mean1, rstd1 = txl.layer_norm_fwd(x, p["g1"], p["b1"])
        ctx = torch.cat([mem.to(dt), h])
        q, k, v = txl.project_qkv(ctx, p["w_q"], p["w_k"], p["w_v"], H, D, D, q_from=M)
        a = txl.rel_attn_fwd(q, k, v, self.rel, p["u"], p["w"], mem_len=M, lse=self.lse_a)
        y, mean2, rstd2 = txl.layer_norm_fwd(x, p["g2"], p["b2"], residual=a.view(L, B, DM))
        loss, lse = txl.softmax_xent_fwd(y, p["table"], target, bias=p["bias"])
        dloss = torch.full((L, B), 1.0 / (L * B), device="cuda")
        txl.softmax_xent_bwd(y, p["table"], target, lse, dloss, bias=p["bias"],
                             grads=dict(dh=(dy := torch.empty_like(y)), dw=g["table"], db=g["bias"]))
        r = txl.layer_norm_bwd(dy, x, mean2, rstd2, gamma=p["g2"], residual=a.view(L, B, DM),
                               grads=dict(dgamma=g["g2"], dbeta=g["b2"]))
        s = txl.rel_attn_bwd(q, k, v, self.rel, p["u"], p["w"], r["dx"].view(L, B, H, D), mem_len=M,
                             out=a if dt == BF else None, lse=self.lse_a)
        # the projections' gradients, products of fp32 matrices
        f = lambda t: t.reshape(-1, DM).float()
        product = lambda a, b: txl.project_heads(a.contiguous(), b.contiguous(), 1, b.shape[0], b.shape[0])[:, 0]   # a b^T
        for n, d, inp in (("w_q", s["dq"], h), ("w_k", s["dk"], ctx), ("w_v", s["dv"], ctx)):
            g[n].copy_(product(f(d).t(), f(inp).t()))
        dh = sum(product(f(d)[-L * B:], p[n].float().t()) for n, d in (("w_q", s["dq"]), ("w_k", s["dk"]), ("w_v", s["dv"])))
        if self.biases:
            g["u"].copy_(s["du"])
            g["w"].copy_(s["dw"])
        # x reaches the loss through the first norm and as the second one's summand
        d1 = txl.layer_norm_bwd(dh.to(dt).view(L, B, DM), x, mean1, rstd1, gamma=p["g1"], dsum=r["dx"],
                                grads=dict(dgamma=g["g1"], dbeta=g["b1"]))
        txl.embed_bwd(tok, d1["dx"], g["table"], DM ** 0.5, accumulate=True)
        norm, clip = txl.grad_norm(self.tensors, 0.25)
        self.number += 1
        txl.adamw_step(self.tensors, self.lr, self.number, grad_scale=clip, seed=11, **HYPER)
        return loss, norm, clip


def _reference(weights, rel, tok, target, mem):
    """The mean loss in float64 and the leaves it depends on."""
    leaf = {n: w.double().clone().requires_grad_(True) for n, w in weights.items()}
    rel = rel.double()
    good = (tok >= 0)[..., None]
    x = leaf["table"][tok.clamp(0)] * DM ** 0.5 * good
    ln = lambda t, g, b: torch.nn.functional.layer_norm(t, (DM,), leaf[g], leaf[b], 1e-5)
    ctx = torch.cat([mem.double(), ln(x, "g1", "b1")])
    heads = lambda t, n: (t @ leaf[n].t()).view(t.shape[0], B, H, D)
    q, k, v = heads(ctx[M:], "w_q"), heads(ctx, "w_k"), heads(ctx, "w_v")
    i, j = torch.arange(L, device="cuda")[:, None], torch.arange(T, device="cuda")[None, :]
    off = M + i - j
    s = torch.einsum("ibhd,jbhd->bhij", q + leaf["u"], k) + \
        torch.einsum("ibhd,ijhd->bhij", q + leaf["w"], rel[(T - 1 - off).clamp(0, T - 1)])
    s = (s / D ** 0.5).masked_fill(off < 0, -float("inf"))
    a = torch.einsum("bhij,jbhd->ibhd", s.softmax(-1), v).reshape(L, B, DM)
    y = ln(x + a, "g2", "b2")
    z = y @ leaf["table"].t() + leaf["bias"]
    ok = (target >= 0) & (target < V)
    loss = torch.where(ok, z.logsumexp(-1) - z.gather(-1, target.clamp(0, V - 1)[..., None])[..., 0], 0.0)
    return loss, leaf


@pytest.mark.parametrize("dtype,bits", [(F32, 32), (BF, 32), (BF, 8)])
def test_steps_against_autograd(dtype, bits):
    """Every step's loss, gradients and clip, with the library's own weights
    of that step in the reference.  fp32 calls are within 1e-5 and bf16 ones
    within 2^-8 of their operands' sizes each; the chain has about ten."""
    from tests.train_helpers import adamw_reference
    step = Step(dtype, 5, bits)
    tol = 2e-4 if dtype == F32 else 10 * 2.0 ** -7
    for t in range(1, 4):
        tok, target, mem = _batch(20 + t)
        before = {n: step.p[n].clone() for n in NAMES}
        masters = {n: w.clone() for n, w in step.master.items()}
        state = {n: (step.m[n].clone(), step.v[n].clone()) for n in NAMES}
        loss, norm, clip = step(tok, target, mem.to(dtype).float())
        torch.cuda.synchronize()
        txl.check()
        want, leaf = _reference(before, step.rel, tok, target, mem.to(dtype))
        (want.sum() / (L * B)).backward()
        want = want.detach()
        assert float((loss.double() - want).abs().max()) <= tol * (1 + float(want.abs().max()))
        for n in NAMES:
            ref, got = leaf[n].grad, step.g[n].double()
            # against the gradient's norm: elements of a matrix differ in what they sum
            assert float((got - ref).norm()) <= tol * float(ref.norm()) + 1e-12, (t, n, float((got - ref).norm() / ref.norm()))
        total = float(sum((step.g[n].double() ** 2).sum() for n in NAMES)) ** 0.5
        assert abs(float(norm) - total) <= 1e-6 * total and abs(float(clip) - min(1.0, 0.25 / total)) <= 1e-6
        for n in NAMES:
            if step.ms[n] is not None:
                continue
            decay = 0.01 if before[n].dim() == 2 and n not in ("u", "w") else 0.0
            new, lim = adamw_reference(masters.get(n, before[n]), step.g[n], *state[n], 0.01, t, 0.9, 0.98, 1e-6, decay,
                                       float(clip))
            got = step.master.get(n, step.p[n]).double()
            # (the rate is a float32 tensor)
            assert ((got - new["p"]).abs() <= lim["p"] + 2.0 ** -23 * new["p"].abs() + 0.01 * 2.0 ** -20).all(), (t, n)
    assert float(step.number) == 3


@pytest.mark.parametrize("dtype,bits", [(F32, 32), (BF, 8)])
def test_a_captured_step_replays_as_steps_made_one_by_one(dtype, bits):
    """To the bit, with u and w kept: the attention's backward adds their
    gradients with atomics, so that two runs of it differ in their last bits."""
    a, b, warm = (Step(dtype, 6, bits, biases=False) for _ in range(3))
    batches = [_batch(30 + t) for t in range(5)]
    warm(*batches[0])       # (the attention's scratch is allocated outside capture)
    s = torch.cuda.Stream()
    tok, target, mem = (x.clone() for x in batches[0])
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        warm(tok, target, mem)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        loss, norm, clip = a(tok, target, mem)
    for t, batch in enumerate(batches):
        for x, y in zip((tok, target, mem), batch):
            x.copy_(y)
        rate = torch.tensor([0.01 / (1 + t)], device="cuda")
        a.lr.copy_(rate)
        b.lr.copy_(rate)
        g.replay()
        want = b(*batch)
        torch.cuda.synchronize()
        for x, y in zip((loss, norm, clip), want):
            assert torch.equal(x, y), t
    for n in NAMES:
        assert torch.equal(a.p[n], b.p[n]) and torch.equal(a.g[n], b.g[n]), n
        assert torch.equal(a.m[n].view(torch.uint8), b.m[n].view(torch.uint8)), n
    txl.check()
