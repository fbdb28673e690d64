"""GPU: the packed operators as one model uses them: a layer's projections from
e4m3 codes, the delta rule over ragged prompts, log probabilities of the next
tokens, and decoded tokens from a captured graph.  Each stage against its formula
in 64 bits, on the inputs that the stage before it really gave."""
import pytest
import torch

import rule_ref as rr

pytestmark = pytest.mark.gpu
D, F8 = rr.D, torch.float8_e4m3fn
HV, HK, H, V = 4, 2, 300, 2000


@pytest.fixture(scope="module")
def g():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import gated_deltanet_decode_amd as g
    return g


class Model:
    def __init__(self, g, dtype):
        gen = torch.Generator().manual_seed(17)
        rnd = lambda *s: torch.randn(*s, generator=gen).cuda()
        self.g, self.dtype, self.dims = g, dtype, g.Dims(HV, HK, D, D)
        self.embed = rnd(V, H).to(dtype)
        self.ns = [HK * D, HK * D, HV * D, 2 * HV]
        self.w_in = self.codes(rnd(sum(self.ns), H) * H ** -0.5, 128)
        self.w_out = self.codes(rnd(V, HV * D) * (HV * D) ** -0.5, 128)

    def codes(self, x, tall=1):
        up = lambda n: (n + 127) // 128
        q = torch.empty(x.shape, dtype=F8, device="cuda")
        scale = torch.empty(x.shape[0] if tall == 1 else up(x.shape[0]), up(x.shape[1]), device="cuda")
        self.g.quantize_f8(x, q, scale, block_rows=tall)
        return q, scale

    def product(self, x, w, ns, dtype):
        outs = [torch.empty(x.shape[0], n, dtype=dtype, device="cuda") for n in ns]
        a = self.codes(x)
        self.g.linear_f8(*a, *w, outs)
        return a, outs

    def tokens(self, ids):
        """q, k, v, beta and gate of the tokens."""
        a, (q, k, v, ba) = self.product(self.embed[ids], self.w_in, self.ns, self.dtype)
        unit = lambda t: torch.nn.functional.normalize(t.float().view(-1, HK, D), dim=-1).to(self.dtype)
        b, alpha = ba.float().view(-1, 2, HV).unbind(1)
        return a, (q, k, v, ba), dict(q=unit(q), k=unit(k), v=v.view(-1, HV, D), beta=torch.sigmoid(b).contiguous(),
                                      gate=(-torch.nn.functional.softplus(alpha)).contiguous())

    def answer(self, out, given, top=8):
        rows = out.shape[0]
        a, (logits,) = self.product(out.reshape(rows, HV * D), self.w_out, [V], torch.float32)
        e = lambda *s, t=torch.float32: torch.empty(*s, dtype=t, device="cuda")
        r = dict(logits=logits, logprob=e(rows), entropy=e(rows), ids=e(rows, top, t=torch.int32), top=e(rows, top))
        ws = e(max(1, self.g.logprobs_workspace_bytes(rows, V, top)), t=torch.uint8)
        self.g.logprobs(logits, given, r["logprob"], r["entropy"], r["ids"], r["top"], workspace=ws)
        return a, r


def wide(codes, rows, n, tall):
    q, s = codes
    return q.cpu().double() * s.cpu().double().repeat_interleave(tall, 0)[:rows].repeat_interleave(128, 1)[:, :n]


def check_product(a, w, got, k):
    """float32: 2^-20 of the norm, some tens of roundings of 2^-24; 16 bits: half a
    step, and 2^-13 for what the 8-bit instructions drop."""
    y = torch.cat([t.cpu().double() for t in got], 1)
    want = wide(a, y.shape[0], k, 1) @ wide(w, y.shape[1], k, 128).t().contiguous()
    t = got[0].dtype
    tol = 2.0 ** -20 if t == torch.float32 else torch.finfo(t).eps / 2 + 2.0 ** -13
    assert float((y - want).norm() / want.norm()) <= tol


def check_answer(a, w, r, given):
    check_product(a, w, [r["logits"]], HV * D)
    p = torch.log_softmax(r["logits"].cpu().double(), -1)
    at = given.cpu().long()[:, None]
    # |log p| below 32: half a step of float32, and 2^-20 for the sums
    assert (r["logprob"].cpu().double() - p.gather(1, at)[:, 0]).abs().max() <= 2.0 ** -19
    assert (r["entropy"].cpu().double() + (p.exp() * p).sum(-1)).abs().max() <= 2.0 ** -19
    top, ids = p.sort(dim=-1, descending=True, stable=True)
    assert torch.equal(r["ids"].cpu().long(), ids[:, :8])
    assert (r["top"].cpu().double() - top[:, :8]).abs().max() <= 2.0 ** -19


@pytest.mark.parametrize("dtype", rr.TYPES.values(), ids=rr.TYPES)
def test_prompt_and_answer(g, dtype):
    m = Model(g, dtype)
    gen = torch.Generator().manual_seed(5)
    lens = [70, 0, 1, 130]
    n, B = sum(lens), len(lens)
    ids = torch.randint(0, V, (n,), generator=gen).cuda()
    given = torch.randint(0, V, (n,), generator=gen).int().cuda()
    slots = torch.tensor([3, 1, 4, 0], dtype=torch.int32, device="cuda")
    pool = 0.1 * torch.randn(6, HV, D, D, generator=gen).cuda()
    a, raw, x = m.tokens(ids)
    check_product(a, m.w_in, raw, H)
    x |= dict(slots=slots, state=pool.clone(),
              offsets=torch.tensor([0, *torch.tensor(lens).cumsum(0).tolist()], dtype=torch.int32, device="cuda"))
    out = torch.empty(n, HV, D, dtype=dtype, device="cuda")
    ws = torch.empty(g.chunk_workspace_bytes(B, n, dtype, m.dims), dtype=torch.uint8, device="cuda")
    g.chunk(x["q"], x["k"], x["v"], x["beta"], x["gate"], out, state=pool, state_out=pool, offsets=x["offsets"],
            slots=slots, workspace=ws)
    y, states, size, psize = rr.forward(x)
    assert ((out.cpu().double() - y).abs() <= rr.out_bound(y, size, dtype)).all()
    assert ((pool.cpu().double() - states).abs() <= rr.state_bound(psize)).all()
    a, r = m.answer(out, given)
    check_answer(a, m.w_out, r, given)

    # decoded tokens: eagerly, then the same from a graph
    first = torch.tensor([11, 12, 13, 14], device="cuda")
    offsets = torch.arange(B + 1, dtype=torch.int32, device="cuda")
    start = pool.clone()

    def step(state, ids):
        x = m.tokens(ids)[2]
        out = torch.empty(B, HV, D, dtype=dtype, device="cuda")
        g.decode(x["q"], x["k"], x["v"], x["beta"], x["gate"], out, state, offsets=offsets, slots=slots)
        a, r = m.answer(out, ids.int())
        return x, out, a, r

    ids, eager = first, []
    for _ in range(4):
        before = pool.clone()
        x, out, a, r = step(pool, ids)
        y, states, size, psize = rr.forward(x | dict(slots=slots, offsets=offsets, state=before))
        assert ((out.cpu().double() - y).abs() <= rr.out_bound(y, size, dtype)).all()
        assert ((pool.cpu().double() - states).abs() <= rr.state_bound(psize)).all()
        check_answer(a, m.w_out, r, ids)
        ids = r["ids"][:, 0].long()
        eager.append((ids.clone(), r["logprob"].clone(), pool.clone()))
    state, now = start.clone(), first.clone()
    graph = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step(state, now)
    torch.cuda.current_stream().wait_stream(s)
    with torch.cuda.graph(graph):
        r = step(state, now)[3]
        now.copy_(r["ids"][:, 0].long())
    state.copy_(start)
    now.copy_(first)
    for ids, logprob, after in eager:
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(now, ids) and torch.equal(r["logprob"], logprob) and torch.equal(state, after)
        m.codes(torch.randn(40, 300, device="cuda"))      # eager work in between
