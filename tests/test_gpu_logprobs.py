"""GPU: gdn_logprobs against log_softmax in 64 bits and a stable order."""
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
INF = float("inf")


@pytest.fixture(scope="module")
def g():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import gated_deltanet_decode_amd as g
    return g


def call(g, x, tokens, top, ws=None, stream=None):
    r, v = x.shape
    n = g.logprobs_workspace_bytes(r, v, top)
    if ws is None:
        ws = torch.empty(n, dtype=torch.uint8, device="cuda").fill_(255) if n else None
    o = dict(logprob=torch.full((r,), 7.0, device="cuda"), entropy=torch.full((r,), 7.0, device="cuda"))
    if top:
        o.update(top_ids=torch.full((r, top), 7, dtype=torch.int32, device="cuda"),
                 top_logprobs=torch.full((r, top), 7.0, device="cuda"))
    g.logprobs(x, tokens, o["logprob"], o["entropy"], top_ids=o.get("top_ids"), top_logprobs=o.get("top_logprobs"),
               workspace=ws, stream=stream)
    return o


def want(x, tokens, top):
    y = x.cpu().double()
    y = y - y.amax(-1, keepdim=True).clamp(min=-1e300)    # first, as a row of -3e38 is uniform
    lp = y - torch.log(torch.exp(y).sum(-1, keepdim=True))
    y = x.cpu().double()
    lp = torch.where((y == -INF).all(-1, keepdim=True), torch.full_like(lp, -INF), lp)
    bad = (y.isnan() | (y == INF)).any(-1)
    lp[bad] = float("nan")
    t = tokens.cpu().long()
    inside = (t >= 0) & (t < x.shape[1])
    o = dict(logprob=torch.where(inside, lp.gather(1, t.clamp(0, x.shape[1] - 1)[:, None])[:, 0], -INF))
    o["logprob"][bad] = float("nan")
    o["entropy"] = -torch.where(lp > -INF, torch.exp(lp) * lp, torch.where(lp.isnan(), lp, 0.0)).sum(-1)
    if top:
        ids = torch.sort(y, dim=1, descending=True, stable=True).indices[:, :top]
        o["top_logprobs"] = lp.gather(1, ids)
        o["top_ids"] = torch.where(bad[:, None], -1, ids)
    return o


def check(g, x, tokens, top, **kw):
    """A result rounds once (2^-24 of it); log Z carries a thread's float32 sums of
    terms right to 2^-22 (the exponent's product, exp, the sum): 2^-21 absolute, and
    the entropy a sum weighted by |x - m|, which is below 128 here."""
    got, ref = call(g, x, tokens, top, **kw), want(x, tokens, top)
    for n, y in ref.items():
        z = got[n].cpu()
        if n == "top_ids":
            assert torch.equal(z.long(), y.long()), (z, y)
            continue
        z = z.double()
        assert torch.equal(z.isnan(), y.isnan()) and torch.equal(z == -INF, y == -INF), n
        ok = torch.isfinite(y)
        tol = 2.0 ** -21 * (128 if n == "entropy" else 1) + 2.0 ** -23 * y.abs()
        assert ((z - y).abs() <= tol)[ok].all(), (n, float((z - y).abs()[ok].max()))
    return got


def logits(r, v, dtype, seed, std=2.5):
    gen = torch.Generator().manual_seed(seed)
    return (torch.randn(r, v, generator=gen) * std).to(dtype).cuda(), torch.randint(0, v, (r,), generator=gen, dtype=torch.int32).cuda()


@pytest.mark.parametrize("dtype", TYPES.values(), ids=TYPES)
@pytest.mark.parametrize("r,v,top", [(1, 1, 1), (3, 2, 2), (2, 7, 7), (5, 63, 20), (4, 1000, 64), (2, 4097, 5), (1, 50001, 20),
                                     (3, 131071, 32), (2100, 257, 3), (300, 9001, 0)])
def test_sizes(g, r, v, top, dtype):
    x, t = logits(r, v, dtype, v)
    check(g, x, t, top)


@pytest.mark.parametrize("dtype", TYPES.values(), ids=TYPES)
@pytest.mark.parametrize("v", [100, 20000])
def test_masks(g, dtype, v):
    """A grammar's masks: nearly all -inf, all of it, the type's lowest value."""
    x, t = logits(7, v, dtype, 3)
    x[0, 5:] = -INF
    x[1] = -INF
    x[2, : v - 3] = -INF
    x[3, ::2] = torch.finfo(dtype).min
    x[4] = torch.finfo(dtype).min
    x[5, 1:] = torch.finfo(dtype).min
    x[6] = -INF
    x[6, v // 2] = -3.0
    t[6] = v // 2
    check(g, x, t, 20)


@pytest.mark.parametrize("v", [100, 40000])
def test_not_finite(g, v):
    x, t = logits(5, v, torch.float32, 4)
    x[0, 3] = float("nan")
    x[1, v - 1] = INF
    x[2] = float("nan")
    x[3, 0], x[3, 1] = -INF, float("nan")
    check(g, x, t, 5)


@pytest.mark.parametrize("dtype", TYPES.values(), ids=TYPES)
@pytest.mark.parametrize("v", [600, 30000])
def test_ties(g, dtype, v):
    """Equal values go by the lower id: a constant row, two values, zeros of either sign."""
    x, t = logits(5, v, dtype, 5)
    x[0] = 1.0
    x[1] = (torch.arange(v, device="cuda") % 3 == 0).to(dtype)
    x[2] = torch.where(torch.arange(v, device="cuda") % 2 == 0, -0.0, 0.0).to(dtype)
    x[3] = x[3].round()
    check(g, x, t, 64)


def test_extremes(g):
    """Far offsets, a nearly certain token, the largest values."""
    x, t = logits(5, 5000, torch.float32, 6)
    x[0] += 1e4
    x[1] -= 1e4
    x[2, 77], t[2] = 40.0, 77
    x[3, 0], t[3] = 3.0e38, 0
    x[3, 1] = -3.0e38
    got, ref = call(g, x, t, 3), want(x, t, 3)
    assert abs(float(got["logprob"][2]) - float(ref["logprob"][2])) <= 2.0 ** -24 * 6000 * 2.0 ** -12 + 1e-12
    check(g, x[2:].contiguous(), t[2:].contiguous(), 3)
    # logits of 1e4 are exact inputs; the results are differences of two of them
    check(g, x[:2].contiguous(), t[:2].contiguous(), 3)


def test_tokens_outside(g):
    x, t = logits(4, 300, torch.bfloat16, 7)
    t[0], t[1], t[2] = -1, 300, 1 << 30
    got = check(g, x, t, 2)
    assert got["logprob"][:3].tolist() == [-INF] * 3


@pytest.mark.parametrize("dtype", TYPES.values(), ids=TYPES)
def test_padded_vocabulary(g, dtype):
    """Rows of a slice: what lies behind V is not read."""
    for v, ld in ((1001, 1024), (9000, 9001), (1000, 1003)):
        x, t = logits(6, ld, dtype, 8)
        x[:, v:] = float("nan")
        check(g, x[:, :v], t % v, 9)
        check(g, x[1:, :v], (t % v)[1:].contiguous(), 9)


def test_parts(g):
    """Each output alone has the bits it has with the others."""
    x, t = logits(3, 20000, torch.bfloat16, 9)
    full = call(g, x, t, 5)
    ws = torch.empty(g.logprobs_workspace_bytes(3, 20000, 5), dtype=torch.uint8, device="cuda")
    lp, en = torch.empty(3, device="cuda"), torch.empty(3, device="cuda")
    ids, top = torch.empty(3, 5, dtype=torch.int32, device="cuda"), torch.empty(3, 5, device="cuda")
    g.logprobs(x, t, lp, workspace=ws)
    g.logprobs(x, entropy=en, workspace=ws)
    g.logprobs(x, top_ids=ids, top_logprobs=top, workspace=ws)
    for n, y in (("logprob", lp), ("entropy", en), ("top_ids", ids), ("top_logprobs", top)):
        assert torch.equal(full[n], y), n


def test_graph_stream_threads(g):
    x, t = logits(4, 40000, torch.bfloat16, 10)
    ref = call(g, x, t, 20)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    ws = torch.empty(g.logprobs_workspace_bytes(4, 40000, 20), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    got = call(g, x, t, 20, ws=ws, stream=s)
    torch.cuda.synchronize()
    buf = {n: torch.empty_like(y) for n, y in ref.items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g.logprobs(x, t, **buf, workspace=ws)
    for _ in range(3):
        for y in buf.values():
            y.zero_()
        graph.replay()
        other = call(g, x, t, 20)
        torch.cuda.synchronize()
        for n in ref:
            assert torch.equal(buf[n], ref[n]) and torch.equal(other[n], ref[n]) and torch.equal(got[n], ref[n]), n
    bad = []

    def work():
        st = torch.cuda.Stream()
        with torch.cuda.stream(st):
            for _ in range(5):
                o = call(g, x, t, 20, stream=st)
                st.synchronize()
                bad.extend(n for n in ref if not torch.equal(o[n], ref[n]))
    threads = [threading.Thread(target=work) for _ in range(2)]
    [h.start() for h in threads]
    [h.join() for h in threads]
    assert not bad


def test_after_verify(g):
    """The answer of a speculative step: a verified token's row is its position's."""
    gen = torch.Generator().manual_seed(11)
    B, K, V = 3, 2, 5000
    x = (torch.randn(B, K + 1, V, generator=gen) * 2).cuda()
    target = torch.softmax(x, -1)
    drafts = target[:, :K].argmax(-1).to(torch.int32).contiguous()
    acc, tok = torch.empty(B, dtype=torch.int32, device="cuda"), torch.empty(B, K + 1, dtype=torch.int32, device="cuda")
    ws = torch.empty(g.verify_workspace_bytes(B, V), dtype=torch.uint8, device="cuda")
    ua, us = torch.rand(B, K, generator=gen).cuda() * 0.02, torch.rand(B, generator=gen).cuda()
    g.verify(target, None, drafts, ua, us, acc, tok, workspace=ws)
    got = check(g, x.flatten(0, 1), tok.flatten(), 4)
    lp = got["logprob"].view(B, K + 1).cpu()
    for b in range(B):
        a = int(acc[b])
        assert torch.isfinite(lp[b, :a + 1]).all() and (lp[b, a + 1:] == -INF).all()
