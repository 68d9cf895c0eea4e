"""The token embedding and its table's gradient on the GPU against float64
(tests/train_helpers.py has the formulas and bounds)."""
import pytest
import torch

from tests.loss_helpers import check
from tests.train_helpers import BF, F32, embed_reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from transformer_xl_relative_rel_gb300 import _build
    _build.build()


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _tokens(kind, rows, vocab, g):
    """Padding rows and tokens far outside among the first ones."""
    u = torch.rand(rows, device="cuda", generator=g, dtype=torch.float64)
    if kind == "zipf":
        t = (vocab ** u).long().clamp(1, vocab) - 1
        t[::7] = -100
        if rows > 20:
            t[3], t[4], t[5], t[6] = vocab, 2 ** 40, -2 ** 63, 2 ** 63 - 1
            t[8], t[9] = 0, vocab - 1
        return t
    if kind == "one":
        return torch.full((rows,), vocab - 1, dtype=torch.int64, device="cuda")
    if kind == "none":
        return torch.full((rows,), vocab, dtype=torch.int64, device="cuda")
    if kind == "two":          # halves of a chunk, ends on its boundaries
        return torch.where(torch.arange(rows, device="cuda") % 3 == 0, 0, vocab // 2)
    return (u * vocab).long().clamp(0, vocab - 1)


def _shifted(x, by):
    """x, `by` elements behind a 16-byte boundary."""
    flat = torch.empty(x.numel() + 8, dtype=x.dtype, device=x.device)
    y = flat[by:by + x.numel()].view(x.shape)
    y.copy_(x)
    return y


def _inputs(rows, d, vocab, dtype, seed, kind="zipf", shift=0):
    g = _gen(seed)
    n = lambda *s: torch.randn(*s, device="cuda", generator=g)
    p = dict(tokens=_tokens(kind, rows, vocab, g), table=n(vocab, d).to(dtype), dout=n(rows, d).to(dtype),
             dtable=n(vocab, d).to(dtype))
    for name in ("table", "dout", "dtable"):
        p[name] = _shifted(p[name], shift) if shift else p[name]
    return p


def _run(p, scale=1.5, accumulate=False, workspace=None):
    import transformer_xl_relative_rel_gb300 as txl
    out = _shifted(torch.full_like(p["dout"], 7.0), 1) if p["table"].data_ptr() % 16 else None
    out = txl.embed_fwd(p["tokens"], p["table"], scale, out=out)
    grad = p["dtable"].clone() if p["dtable"].data_ptr() % 16 == 0 else _shifted(p["dtable"], 1)
    if not accumulate:
        grad.fill_(float("nan"))
    txl.embed_bwd(p["tokens"], p["dout"], grad, scale, accumulate=accumulate, workspace=workspace)
    return dict(out=out, dtable=grad)


def _check(p, scale=1.5, accumulate=False, got=None):
    import transformer_xl_relative_rel_gb300 as txl
    got = _run(p, scale, accumulate) if got is None else got
    want, tol = embed_reference(p["tokens"], p["table"], scale, p["dout"], p["dtable"] if accumulate else None)
    check(got, want, tol)
    txl.check()


SIZES = [(1, 1, 1), (1, 512, 256), (3, 8, 2), (31, 64, 5), (32, 64, 5), (33, 64, 700), (64, 40, 3), (257, 256, 5003),
         (1000, 410, 511), (1023, 72, 512), (1024, 33, 513), (1025, 1024, 131072), (2049, 128, 262143),
         (5000, 64, 262144), (3000, 24, 300001), (9000, 410, 50021), (16896, 512, 256), (70000, 33, 1000)]


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,d,vocab", SIZES)
def test_sizes(rows, d, vocab, dtype, accumulate):
    p = _inputs(rows, d, vocab, dtype, rows + d)
    p["dout"][::7] = float("nan")        # what padding rows hold does not matter
    if rows > 20:
        p["dout"][3:7] = float("inf")
    else:
        p["tokens"][::7] = -1
    _check(p, 1.5, accumulate)


@pytest.mark.parametrize("shift", [0, 1, 2, 4])
@pytest.mark.parametrize("kind", ["zipf", "one", "none", "two", "even"])
@pytest.mark.parametrize("dtype,rows,d,vocab", [(BF, 2000, 64, 77), (F32, 777, 24, 1000), (BF, 300, 41, 20),
                                                (BF, 1, 512, 256), (F32, 2, 3, 1),
                                                (BF, 100000, 24, 77), (F32, 300001, 9, 5), (F32, 33000, 300, 40)])
def test_tokens_and_alignments(dtype, rows, d, vocab, kind, shift):
    p = _inputs(rows, d, vocab, dtype, 5, kind, shift)
    for accumulate in (False, True):
        _check(p, -0.37, accumulate)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows", [2047 * 16 + 1, 2048 * 16, 2049 * 16 - 3, 140000])
def test_runs_that_end_around_groups_of_chunks(rows, dtype):
    """Sorted tokens whose rows begin and end at, just before and just behind
    the ends of 16 rows and of 32 times 16."""
    import transformer_xl_relative_rel_gb300 as txl
    g = _gen(rows)
    lengths, total = [], 0
    near = [1, 15, 16, 17, 31, 511, 512, 513, 1023, 1024, 1025, 528, 496, 5000, 2560, 33 * 16, 3, 13, 498]
    while total < rows:
        lengths.append(near[len(lengths) % len(near)] + (len(lengths) // len(near)) % 5)
        total += lengths[-1]
    tok = torch.repeat_interleave(torch.arange(len(lengths)), torch.tensor(lengths))[:rows].cuda()
    vocab = len(lengths)
    dout = torch.randint(-4, 5, (rows, 140), device="cuda", generator=g).to(dtype)
    want = torch.zeros(vocab, 140, dtype=torch.float64, device="cuda").index_add_(0, tok, dout.double())
    order = torch.randperm(rows, device="cuda", generator=g)
    for t, x in ((tok, dout), (tok[order], dout[order].contiguous())):
        grad = txl.embed_bwd(t, x, vocab=vocab)
        # whole numbers below 2^24: exact sums, one rounding
        assert torch.equal(grad, want.to(dtype))
        old = torch.ones(vocab, 140, dtype=dtype, device="cuda")
        assert torch.equal(txl.embed_bwd(t, x, old, accumulate=True), (want + 1).to(dtype))
    txl.check()


def test_rows_of_other_tokens_stay_as_they_are():
    p = _inputs(500, 64, 3000, BF, 6)
    p["dtable"][:] = torch.randint(-32768, 32767, (3000, 64), device="cuda", generator=_gen(1)).to(torch.int16).view(BF)
    absent = torch.ones(3000, dtype=torch.bool, device="cuda")
    good = p["tokens"][(p["tokens"] >= 0) & (p["tokens"] < 3000)]
    absent[good] = False
    got = _run(p, accumulate=True)["dtable"]
    assert torch.equal(got.view(torch.int16)[absent], p["dtable"].view(torch.int16)[absent])
    assert absent.sum() > 2000
    got = _run(p)["dtable"]
    assert not got[absent].any()


def test_values_that_are_not_finite():
    """They reach their token's columns and nothing else."""
    p = _inputs(900, 48, 40, F32, 7, "even")
    p["dout"][5, 3], p["dout"][6, 4] = float("inf"), float("nan")
    p["table"][2, 1] = float("-inf")
    got = _run(p)
    bad = torch.zeros(40, 48, dtype=torch.bool, device="cuda")
    bad[p["tokens"][5], 3] = bad[p["tokens"][6], 4] = True
    assert torch.equal(~torch.isfinite(got["dtable"]), bad)
    assert float(got["dtable"][p["tokens"][5], 3]) == float("inf") and bool(got["dtable"][p["tokens"][6], 4].isnan())
    assert torch.equal(got["out"] == -float("inf"), (p["tokens"] == 2)[:, None] & (torch.arange(48, device="cuda") == 1))


@pytest.mark.parametrize("rows,d,vocab,kind", [(16896, 64, 256, "zipf"), (5000, 128, 9, "two"), (40000, 40, 100000, "zipf")])
def test_the_same_call_gives_the_same_bits(rows, d, vocab, kind):
    import transformer_xl_relative_rel_gb300 as txl
    p = _inputs(rows, d, vocab, F32, 8, kind)
    size = txl.embed_bwd_workspace_bytes(rows, d, vocab, txl.TXL_F32)
    first = _run(p)
    for k in range(5):
        ws = torch.full((size // 4,), float("nan") if k % 2 else float(k), device="cuda")
        again = _run(p, workspace=ws)
        assert torch.equal(again["dtable"], first["dtable"]) and torch.equal(again["out"], first["out"])


def test_rows_add_in_their_order():
    """A row that cancels what came before it leaves what comes behind it."""
    big = torch.tensor([1e30, -1e30, 1.0, 2.0], device="cuda").repeat(2)[:, None].repeat(1, 8).contiguous()
    tok = torch.full((8,), 3, dtype=torch.int64, device="cuda")
    import transformer_xl_relative_rel_gb300 as txl
    got = txl.embed_bwd(tok, big, vocab=5)
    want = 0.0
    for x in big[:, 0].tolist():
        want = float(torch.tensor(want, dtype=F32) + torch.tensor(x, dtype=F32))
    assert (got[3] == want).all()


def test_no_rows():
    import transformer_xl_relative_rel_gb300 as txl
    tok, dout = torch.empty(0, dtype=torch.int64, device="cuda"), torch.empty(0, 16, device="cuda", dtype=BF)
    table = torch.ones(30, 16, device="cuda", dtype=BF)
    assert txl.embed_fwd(tok, table).shape == (0, 16)
    grad = torch.full_like(table, 3.0)
    assert (txl.embed_bwd(tok, dout, grad, accumulate=True) == 3).all()
    assert not txl.embed_bwd(tok, dout, grad).any()
    assert not txl.embed_bwd(tok, dout, vocab=7).any()
    txl.check()


def test_shapes_of_more_dimensions():
    import transformer_xl_relative_rel_gb300 as txl
    p = _inputs(60, 32, 50, F32, 9)
    tok, dout = p["tokens"].view(3, 4, 5), p["dout"].view(3, 4, 5, 32)
    out = txl.embed_fwd(tok, p["table"], 2.0)
    assert out.shape == (3, 4, 5, 32)
    grad = txl.embed_bwd(tok, dout, vocab=50, scale=2.0)
    check(dict(out=out.view(60, 32), dtable=grad), *embed_reference(p["tokens"], p["table"], 2.0, p["dout"]))
    one = txl.embed_fwd(tok[0, 0, 1], p["table"], 2.0)
    assert torch.equal(one, out[0, 0, 1])


@pytest.mark.parametrize("rows", [5000, 131072, 131073, 300000])
@pytest.mark.parametrize("vocab", [1 << 27, (1 << 28) + 1])
def test_tokens_of_many_digits(rows, vocab):
    """Vocabularies whose tokens are sorted by four digits, in one cluster and
    by launches: tokens that differ in one digit only, each once and twice."""
    import transformer_xl_relative_rel_gb300 as txl
    g = _gen(12)
    tok = torch.randint(0, vocab, (rows,), device="cuda", generator=g)
    tok[:256] = torch.arange(256, device="cuda")
    tok[256:512] = torch.arange(256, device="cuda") << 8
    tok[512:768] = torch.arange(256, device="cuda") << 16
    tok[768:776] = torch.arange(8, device="cuda") << 24
    tok[776], tok[777], tok[778] = vocab - 1, vocab, vocab - 2
    dout = torch.randint(-8, 9, (rows, 2), device="cuda", generator=g).to(BF)
    grad = txl.embed_bwd(tok, dout, torch.full((vocab, 2), 3.0, dtype=BF, device="cuda"))
    good = tok < vocab
    names, at = torch.unique(tok[good], return_inverse=True)
    want = torch.zeros(len(names), 2, dtype=torch.float64, device="cuda").index_add_(0, at, dout[good].double())
    assert torch.equal(grad[names].double(), want)
    grad[names] = 0
    assert not grad.any()
    txl.check()


@pytest.mark.parametrize("rows,d,vocab", [(40, 2100, 1 << 20), (2200000, 1000, 3)])
def test_offsets_past_32_bits(rows, d, vocab):
    """A table, and rows, of more than 2^31 elements."""
    import transformer_xl_relative_rel_gb300 as txl
    g = _gen(10)
    tok = torch.randint(0, vocab, (rows,), device="cuda", generator=g)
    if vocab > 1000:
        tok[5], tok[6] = vocab - 1, vocab - 2
        table = torch.zeros(vocab, d, dtype=BF, device="cuda")
        table[tok] = torch.randn(rows, d, device="cuda", generator=g).to(BF)
        out = txl.embed_fwd(tok, table, 2.0)
        assert torch.equal(out, table[tok] * 2)
        grad = txl.embed_bwd(tok, out, torch.full_like(table, 5.0), 0.5)
        present = torch.unique(tok)
        assert len(present) == rows and torch.equal(grad[tok], table[tok])
        grad[tok] = 0
        assert not any(part.any() for part in grad.split(1 << 17))
        return
    table = torch.randn(vocab, d, device="cuda", generator=g).to(BF)
    out = txl.embed_fwd(tok, table)
    for part in range(0, rows, 1 << 18):
        assert torch.equal(out[part:part + (1 << 18)], table[tok[part:part + (1 << 18)]])
    # sums of equal values: exact in fp32 up to 2^24 terms of 8 bits
    out.fill_(0.5)
    out[-1] = 64.0
    grad = txl.embed_bwd(tok, out, vocab=vocab)
    want = 0.5 * torch.bincount(tok, minlength=vocab).double()
    want[tok[-1]] += 63.5
    assert torch.equal(grad, want.float().to(BF)[:, None].expand(vocab, d))
    txl.check()


def test_captured_and_replayed():
    """Two graphs with workspaces of their own and tokens of other draws."""
    import transformer_xl_relative_rel_gb300 as txl
    ps = [_inputs(2500, 64, 300, BF, 11), _inputs(40, 41, 5000, F32, 12)]
    ws = [torch.empty(txl.embed_bwd_workspace_bytes(*p["dout"].shape, len(p["table"]), c), dtype=torch.uint8, device="cuda")
          for p, c in zip(ps, (txl.TXL_BF16, txl.TXL_F32))]
    outs, graphs = [], []
    torch.cuda.synchronize()
    for p, w in zip(ps, ws):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(_run(p, workspace=w))
        graphs.append(g)
    for seed in (13, 14):
        for p, kind in zip(ps, ("one", "even")):
            q = _inputs(*p["dout"].shape, len(p["table"]), p["table"].dtype, seed, kind)
            for n in p:
                p[n].copy_(q[n])
        for g in graphs + graphs:
            g.replay()
        torch.cuda.synchronize()
        for p, out in zip(ps, outs):
            _check(p, got=out)


def test_streams_and_host_threads_at_once():
    import threading
    ps = [_inputs(3000, 64, 200, BF, 20), _inputs(500, 40, 70000, F32, 21), _inputs(9000, 72, 9, BF, 22, "two")]
    want = [_run(p) for p in ps]
    torch.cuda.synchronize()
    wrong = []

    def work(x):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(20):
                got = _run(ps[x])
            s.synchronize()
        wrong.extend((x, n) for n in got if not torch.equal(got[n], want[x][n]))

    threads = [threading.Thread(target=work, args=(x,)) for x in range(len(ps))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong, wrong


def test_a_stream_given_as_an_argument():
    import transformer_xl_relative_rel_gb300 as txl
    p = _inputs(3000, 64, 200, BF, 23)
    want = _run(p)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(10):
        out = txl.embed_fwd(p["tokens"], p["table"], 1.5, stream=s)
        grad = txl.embed_bwd(p["tokens"], p["dout"], vocab=200, scale=1.5, stream=s)
    s.synchronize()
    assert torch.equal(out, want["out"]) and torch.equal(grad, want["dtable"])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_calls_back_to_back_in_one_workspace(dtype):
    import transformer_xl_relative_rel_gb300 as txl
    ps = [_inputs(r, d, v, dtype, 30 + r, k) for r, d, v, k in
          [(5, 72, 300, "even"), (5000, 64, 4000, "zipf"), (33, 64, 70000, "two"), (9000, 40, 7, "zipf"), (600, 512, 100, "one")]]
    code = txl.TXL_BF16 if dtype == BF else txl.TXL_F32
    ws = torch.empty(max(txl.embed_bwd_workspace_bytes(*p["dout"].shape, len(p["table"]), code) for p in ps),
                     dtype=torch.uint8, device="cuda")
    want = [_run(p) for p in ps]
    torch.cuda.synchronize()
    order = [0, 1, 2, 3, 4, 3, 1, 4, 0, 2] * 3
    got = [_run(ps[k], workspace=ws) for k in order]
    torch.cuda.synchronize()
    for k, x in zip(order, got):
        assert torch.equal(x["out"], want[k]["out"]) and torch.equal(x["dtable"], want[k]["dtable"])


def test_oracle():
    import numpy as np
    import oracle
    p = _inputs(90, 16, 30, F32, 40)
    got = _run(p, 3.0)
    out, grad = oracle.embed(p["tokens"].cpu().numpy(), p["table"].double().cpu().numpy(), 3.0,
                             p["dout"].double().cpu().numpy())
    assert np.abs(got["out"].cpu().numpy() - out).max() < 1e-5
    assert np.abs(got["dtable"].cpu().numpy() - grad).max() < 1e-4
