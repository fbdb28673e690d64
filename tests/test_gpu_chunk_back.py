"""GPU: gdn_chunk_backward against the adjoint recurrence in 64 bits and against
differences of gdn_chunk."""
import pytest
import torch

import rule_ref as rr
from test_gpu_chunk import chunk

pytestmark = pytest.mark.gpu
D = rr.D
NAMES = ("q", "k", "v", "beta", "gate")


@pytest.fixture(scope="module")
def g():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import gated_deltanet_decode_amd as g
    return g


def space(g, x):
    hv, hk = x["v"].shape[1], x["q"].shape[1]
    n = g.chunk_backward_workspace_bytes(x["offsets"].shape[0] - 1, x["q"].shape[0], x["q"].dtype, g.Dims(hv, hk, D, D))
    return torch.empty(n, dtype=torch.uint8, device="cuda").fill_(255)       # NaN wherever nothing was written


def backward(g, x, d_state=True, ws=None, stream=None):
    got = {"d" + n: torch.full_like(x[n], 7.0) for n in NAMES}
    if d_state is True:
        d_state = torch.full((x["offsets"].shape[0] - 1, x["v"].shape[1], D, D), 5.0, device="cuda")
    g.chunk_backward(*(x[n] for n in NAMES), x["d_out"], *got.values(), state=x["state"], d_state_out=x["d_state_out"],
                     d_state=d_state, offsets=x["offsets"], workspace=space(g, x) if ws is None else ws, stream=stream)
    return dict(got, d_state=d_state) if d_state is not None else got


def check(x, got, dtype, more=1):
    """In the 2-norm: 16-bit gradients are rounded once, half a step a value, from
    sums right to 2^-15 of terms that are at most four times as large as their
    sum; float32 ones carry some hundreds of independent roundings of 2^-24.  dgate
    is a sum of up to 64 values c = out . d_out - v . dv, each right to 2^-21 of the
    product of the norms, so eight times their norm counts beside its own."""
    want = rr.backward(x)
    used = x["offsets"][-1].item()
    out = rr.forward(x)[0]
    size = out.norm(dim=-1) * x["d_out"].cpu().double().norm(dim=-1) + want["dv"].norm(dim=-1) * x["v"].cpu().double().norm(dim=-1)
    for n, y in want.items():
        if n not in got:
            continue
        z = got[n].cpu().double()
        if n != "d_state":
            assert (z[used:] == 7.0).all(), n             # rows behind the last sequence
            y, z = y[:used], z[:used]
        wide = dtype == torch.float32 or n in ("dbeta", "dgate", "d_state")
        tol = 2.0 ** -20 if wide else torch.finfo(dtype).eps / 2 + 2.0 ** -13
        limit = more * tol * (y.norm() + (8 * size[:used].norm() if n == "dgate" else 0)) + 1e-30
        err = (z - y).norm()
        assert err <= limit, (n, float(err / (y.norm() + 1e-300)), float(err / limit))


@pytest.mark.parametrize("dtype", rr.TYPES.values(), ids=rr.TYPES)
@pytest.mark.parametrize("lens", [[1], [2, 0, 1], [63], [64], [65], [128, 0, 1, 200, 127], [0], [500]], ids=str)
def test_lengths(g, lens, dtype):
    x = rr.inputs(lens, 4, 2, dtype, 21, tail=3)
    check(x, backward(g, x), dtype)


@pytest.mark.parametrize("dtype", rr.TYPES.values(), ids=rr.TYPES)
@pytest.mark.parametrize("hv,hk", [(1, 1), (3, 1), (6, 2), (5, 5), (16, 4)])
def test_heads(g, hv, hk, dtype):
    """dq and dk are sums over the value heads of a key head."""
    x = rr.inputs([70, 5], hv, hk, dtype, 22, start=False)
    x["d_state_out"] = None
    check(x, backward(g, x, d_state=None), dtype)


@pytest.mark.parametrize("gate", [0.0, -1e-4, -3.0, -50.0, -700.0, float("-inf"), 0.01])
def test_gates(g, gate):
    x = rr.inputs([130], 2, 1, torch.float32, 23, gate=gate)
    if gate == float("-inf"):
        # the formula's own exp(gate) * gradient is 0 there
        want = rr.backward(x)
        assert (want["dgate"] == 0).all()
    check(x, backward(g, x), torch.float32)


def test_slight_decays(g):
    """Gates from nothing at all over what float64 just tells from it beside 1 to strong."""
    x = rr.inputs([130, 64, 1, 70], 4, 2, torch.float32, 31)
    kinds = torch.tensor([0.0, -0.0, -1e-38, -2.0**-60, -2.0**-54, -1e-12, -1e-5, -0.3, -1.0, -50.3], device="cuda")
    x["gate"] = kinds[torch.randint(0, len(kinds), x["gate"].shape, generator=torch.Generator().manual_seed(3)).cuda()]
    x["gate"][:64] = -2.0**-60                            # a chunk of nothing else
    check(x, backward(g, x), torch.float32)


@pytest.mark.parametrize("dtype", rr.TYPES.values(), ids=rr.TYPES)
def test_betas(g, dtype):
    """Tokens that write nothing still have a gradient of beta."""
    x = rr.inputs([100, 30], 4, 2, dtype, 24)
    x["beta"][::3] = 0.0
    x["beta"][1::9] = 1e-25
    x["beta"][2::9] = 1.0
    got = backward(g, x)
    check(x, got, dtype)
    assert (got["dv"][:130:3] == 0).all() and (got["dbeta"][:130:3] != 0).all()


def test_same_key_and_full_writes(g):
    """Every token replaces what the one before it wrote: the corrections are
    Delta_j = v_j - v_(j-1), so a sum over the i before a token, of norm |v|, has i
    terms of norm sqrt(2) |v| whose roundings are independent: sqrt(2 i) as much
    error for its size, 8 at the mean i of 32."""
    x = rr.inputs([128], 2, 1, torch.float32, 25, gate=0.0)
    x["k"][:] = x["k"][0]
    x["beta"][:] = 1.0
    check(x, backward(g, x), torch.float32, more=8)


def test_in_place_and_repeated(g):
    """d_state may be d_state_out; a second call gives the same bits, alone in its
    batch too."""
    x = rr.inputs([70, 200], 4, 2, torch.bfloat16, 26)
    got = backward(g, x)
    y = dict(x, d_state_out=x["d_state_out"].clone())
    again = backward(g, y, d_state=y["d_state_out"])
    for n in got:
        assert torch.equal(got[n], again[n]), n
    one = {n: x[n][70:270].contiguous() for n in NAMES + ("d_out",)}
    one.update(offsets=torch.tensor([0, 200], dtype=torch.int32, device="cuda"), state=x["state"][1:].clone(),
               d_state_out=x["d_state_out"][1:].clone())
    alone = backward(g, one)
    for n in got:
        assert torch.equal(alone[n], got[n][1:] if n == "d_state" else got[n][70:270]), n


def test_against_differences(g):
    """Along random directions of every input, float32: central differences of the
    loss sum(out d_out) + sum(state_out d_state_out), formed in 64 bits.  The step
    2^-6 of unit directions leaves a third-order remainder below 2^-12 of the
    derivative's scale and forward roundings of 2^-21 / 2^-6."""
    x = rr.inputs([90, 33], 4, 2, torch.float32, 27)
    got = backward(g, x)
    gen = torch.Generator().manual_seed(5)

    def loss(y):
        out, so = chunk(g, y)
        return float((out.double() * x["d_out"].double()).sum() + (so.double() * x["d_state_out"].double()).sum())

    for n in NAMES + ("state",):
        d = torch.randn(x[n].shape, generator=gen).cuda()
        # along the gradient, so that the derivative is not a small difference
        grad = got["d_state" if n == "state" else "d" + n]
        d = grad / grad.norm() + 0.1 * d / d.norm()
        h = 2.0 ** -6
        diff = (loss(dict(x, **{n: x[n] + h * d})) - loss(dict(x, **{n: x[n] - h * d}))) / (2 * h)
        want = float((grad.double() * d.double()).sum())
        assert abs(diff - want) <= 2.0 ** -8 * abs(want), (n, diff, want)


def test_foreign_offsets(g):
    x = rr.inputs([20, 30], 2, 1, torch.bfloat16, 28)
    good = backward(g, x)
    y = dict(x, offsets=torch.tensor([-5, 20, 1 << 30], dtype=torch.int32, device="cuda"))
    got = backward(g, y)
    for n in good:
        assert torch.equal(got[n], good[n]), n


def test_graph_and_stream(g):
    x = rr.inputs([130, 40], 8, 4, torch.bfloat16, 29)
    want, ws = backward(g, x), space(g, x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = backward(g, x, ws=ws, stream=s)
    s.synchronize()
    for n in want:
        assert torch.equal(got[n], want[n]), n
    buf = {n: torch.empty_like(t) for n, t in want.items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g.chunk_backward(*(x[n] for n in NAMES), x["d_out"], *(buf["d" + n] for n in NAMES), state=x["state"],
                         d_state_out=x["d_state_out"], d_state=buf["d_state"], offsets=x["offsets"], workspace=ws)
    for _ in range(3):
        for t in buf.values():
            t.zero_()
        graph.replay()
        other = backward(g, x)
        torch.cuda.synchronize()
        for n in want:
            assert torch.equal(buf[n], want[n]) and torch.equal(other[n], want[n]), n


def test_training_step(g):
    """The pair as an autograd function: two layers of the rule one after another,
    their gradients against the recurrence in 64 bits run through torch."""
    dims = g.Dims(4, 2, D, D)

    class Rule(torch.autograd.Function):
        @staticmethod
        def forward(ctx, q, k, v, beta, gate, offsets):
            out = torch.empty_like(v)
            B = offsets.shape[0] - 1
            ws = torch.empty(g.chunk_workspace_bytes(B, q.shape[0], q.dtype, dims), dtype=torch.uint8, device=q.device)
            g.chunk(q, k, v, beta, gate, out, offsets=offsets, workspace=ws)
            ctx.save_for_backward(q, k, v, beta, gate, offsets)
            return out

        @staticmethod
        def backward(ctx, d_out):
            q, k, v, beta, gate, offsets = ctx.saved_tensors
            grads = [torch.empty_like(t) for t in (q, k, v, beta, gate)]
            B = offsets.shape[0] - 1
            ws = torch.empty(g.chunk_backward_workspace_bytes(B, q.shape[0], q.dtype, dims), dtype=torch.uint8, device=q.device)
            g.chunk_backward(q, k, v, beta, gate, d_out.contiguous(), *grads, offsets=offsets, workspace=ws)
            return (*grads, None)

    x = rr.inputs([40, 70], 4, 2, torch.float32, 30, start=False)
    leaves = {n: x[n].clone().requires_grad_() for n in NAMES}
    first = Rule.apply(*leaves.values(), x["offsets"])
    out = Rule.apply(leaves["q"], leaves["k"], first, leaves["beta"], leaves["gate"], x["offsets"])
    (out * x["d_out"]).sum().backward()

    ref = {n: x[n].cpu().double().requires_grad_() for n in NAMES}
    heads = torch.arange(4) % 2

    def rule(v):
        ys = []
        for first_, end, _ in rr._spans(rr._host(x)):
            m = torch.zeros(4, D, D, dtype=torch.float64)
            for t in range(first_, end):
                k, q = ref["k"][t, heads], ref["q"][t, heads]
                m = torch.exp(ref["gate"][t])[:, None, None] * m
                m = m + (ref["beta"][t][:, None] * (v[t] - (m * k[:, None]).sum(-1)))[..., None] * k[:, None]
                ys.append((m * q[:, None]).sum(-1) / D ** 0.5)
        return torch.stack(ys)

    (rule(rule(ref["v"])) * x["d_out"].cpu().double()).sum().backward()
    for n in NAMES:
        # two passes of roundings of 2^-24 in their hundreds; dgate cancels
        assert rr.rel(leaves[n].grad, ref[n].grad) <= (2.0 ** -16 if n == "gate" else 2.0 ** -19), n
