"""GPU: gdn_verify against the definition in 64 bits (whole numbers, equal), and
gdn_pair_commit, a masked copy (bitwise)."""
import numpy as np
import pytest
import torch

import serve_ref as sr

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def g():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import gated_deltanet_decode_amd as g
    return g


def make(B, K, V, dtype, seed, greedy=False, peak=2.0):
    gen = torch.Generator().manual_seed(seed)
    logits = torch.randn(B, K + 1, V, generator=gen) * peak
    target = torch.softmax(logits, -1).to(dtype)
    q = torch.softmax(logits[:, :K] + 0.6 * torch.randn(B, K, V, generator=gen), -1)
    d = q.argmax(-1) if greedy else torch.multinomial(q.reshape(-1, V), 1, generator=gen).reshape(B, K)
    return dict(target=target, draft=None if greedy else q.to(dtype), draft_tokens=d.int(),
                u_accept=torch.rand(B, K, generator=gen), u_sample=torch.rand(B, generator=gen))


def run(g, c, n_draft=None):
    B, K1, V = c["target"].shape
    acc = torch.full((B + 2,), 77, dtype=torch.int32, device="cuda")
    tok = torch.full((B * K1 + 2,), 77, dtype=torch.int32, device="cuda")
    need = g.verify_workspace_bytes(B, V)
    ws = torch.full((need + 64,), 7, dtype=torch.uint8, device="cuda")
    d = {k: None if t is None else t.cuda() for k, t in c.items()}
    g.verify(d["target"], d["draft"], d["draft_tokens"], d["u_accept"], d["u_sample"], acc[1:-1],
             tok[1:-1].view(B, K1), n_draft=None if n_draft is None else n_draft.cuda(),
             workspace=ws[:need])
    torch.cuda.synchronize()
    assert int(acc[0]) == int(acc[-1]) == 77 and int(tok[0]) == int(tok[-1]) == 77
    assert bool((ws[need:] == 7).all())
    return acc[1:-1].cpu().numpy(), tok[1:-1].view(B, K1).cpu().numpy()


def check(g, c, n_draft=None):
    got = run(g, c, n_draft)
    want = sr.verify(c["target"], c["draft"], c["draft_tokens"], c["u_accept"], c["u_sample"], n_draft)
    assert np.array_equal(got[0], want[0]), "accepted"
    assert np.array_equal(got[1], want[1]), "tokens"
    return got


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("greedy", [False, True])
@pytest.mark.parametrize("B,K,V", [(1, 1, 1), (3, 2, 5), (64, 1, 100), (40, 3, 4095), (40, 3, 4096),
                                   (40, 3, 4097), (7, 5, 32000), (5, 1, 131071), (300, 2, 257), (2, 2, 1023),
                                   (2, 2, 1025), (2, 2, 2047), (2, 2, 2049), (3, 1, 262143), (1, 1, 600001),
                                   (1, 1, 1100000)])
def test_against_the_definition(g, dtype, greedy, B, K, V):
    print(f"\n  verify B={B} K={K} V={V} {dtype} greedy={greedy}", flush=True)
    check(g, make(B, K, V, dtype, B + K + V, greedy))


@pytest.mark.parametrize("K", [1, 2, 63, 64, 65, 130])
def test_long_runs(g, K):
    """Runs past a wave's 64 positions; every length of the drafts, and lengths
    outside [0, K], which count as the nearer end."""
    print(f"\n  verify K={K}", flush=True)
    B, V = 40, 50
    c = make(B, K, V, torch.float32, K)
    c["u_accept"] *= 0.02                      # most drafts pass
    n = torch.randint(0, K + 1, (B,), generator=torch.Generator().manual_seed(K), dtype=torch.int32)
    n[:4] = torch.tensor([-5, K + 9, 0, K])
    check(g, c, n)
    c["u_accept"].zero_()                      # all pass: 0 * q < p
    a, _ = check(g, c, n)
    assert np.array_equal(a, np.clip(n.numpy(), 0, K))


def test_borders_are_exact(g):
    """Dyadic probabilities: u q = p refuses, the next binary32 below accepts;
    a cumulative sum equal to the goal does not pass it."""
    print("\n  verify: borders", flush=True)
    V = 8
    p = torch.tensor([0.25, 0.0, 0.125, 0.125, 0.0, 0.25, 0.25, 0.0])
    q = torch.tensor([0.5, 0.0, 0.25, 0.0, 0.0, 0.25, 0.0, 0.0])
    u = torch.tensor([0.5, np.nextafter(np.float32(0.5), np.float32(0)), 0.0, 0.999])
    c = dict(target=p.repeat(4, 2, 1), draft=q.repeat(4, 1, 1), draft_tokens=torch.zeros(4, 1).int(),
             u_accept=u[:, None].contiguous(), u_sample=torch.tensor([0.0, 0.0, 0.25, 0.5]))
    a, t = check(g, c)
    assert a.tolist() == [0, 1, 1, 0]
    # rest = [0 0 0 1/8 0 0 1/4 0]; its third equals 1/3, so u = 0.5 falls in entry 6
    assert t.tolist() == [[3, -1], [0, 0], [0, 2], [6, -1]]
    # goals on the borders of p's cumulative sum
    for us, want in ((0.0, 0), (0.25, 2), (0.375, 3), (0.5, 5), (0.75, 6), (0.99999994, 6), (1.0, 6),
                     (float("nan"), 6), (-1.0, 0)):
        c2 = dict(c, u_sample=torch.full((4,), us))
        _, t = check(g, c2, torch.zeros(4, dtype=torch.int32))
        assert t[:, 0].tolist() == [want] * 4, us


@pytest.mark.parametrize("V", [3, 100, 5000, 20000])
def test_rows_with_nothing_left(g, V):
    """p = q (no rest: drawn from p), all-zero rows (-1), NaN, infinite and
    negative entries (count as 0), a single live entry, drafts outside [0, V)."""
    print(f"\n  verify: degenerate rows V={V}", flush=True)
    B = 10
    c = make(B, 2, V, torch.float32, V)
    c["u_accept"].fill_(0.9999)
    c["draft"][0] = c["target"][0, :2]
    c["u_accept"][0] = 1.0                     # refuses although p = q
    c["target"][1] = 0.0
    c["target"][2] = float("nan")
    c["target"][3] = -1.0
    c["target"][4] = 0.0
    c["target"][4, :, V - 1] = 1e-30
    c["target"][5, :, 0] = float("inf")
    c["draft"][6] = float("nan")
    c["draft_tokens"][7, 0] = -1
    c["draft_tokens"][8, 0] = V
    c["draft_tokens"][9, 0] = 2 ** 31 - 1
    check(g, c)
    check(g, dict(c, draft=None))
    c["u_accept"][6] = float("nan")
    check(g, c)


@pytest.mark.parametrize("dtype,step", [(torch.float32, 2.0 ** -149), (torch.bfloat16, 2.0 ** -133),
                                        (torch.float16, 2.0 ** -24)])
def test_subnormal_probabilities(g, dtype, step):
    """Whole multiples of the type's smallest value: products, differences and
    sums are exact in binary64, so nothing may be flushed to zero."""
    print(f"\n  verify: subnormal probabilities {dtype}", flush=True)
    gen = torch.Generator().manual_seed(11)
    B, K, V = 24, 2, 777
    target = (torch.randint(0, 4, (B, K + 1, V), generator=gen).double() * step).to(dtype)
    draft = (torch.randint(0, 4, (B, K, V), generator=gen).double() * step).to(dtype)
    assert float(target.double().max()) == 3 * step
    c = dict(target=target, draft=draft,
             draft_tokens=torch.randint(0, V, (B, K), generator=gen).int(),
             u_accept=torch.rand(B, K, generator=gen), u_sample=torch.rand(B, generator=gen))
    a, t = check(g, c)
    assert 0 < a.sum() < B * K and (t[np.arange(B), a] >= 0).all()


def test_peaked_rows(g):
    """Rows where one entry holds nearly everything, at every place of a vector and
    of a unit, so that the goal falls next to it."""
    print("\n  verify: peaked rows", flush=True)
    V = 5000
    places = list(range(0, 20)) + [63, 64, 255, 256, 1023, 1024, 1025, 2047, 2048, 4095, 4096, 4990, 4999]
    B = len(places)
    gen = torch.Generator().manual_seed(5)
    target = torch.rand(B, 2, V, generator=gen) * 1e-9
    draft = torch.rand(B, 1, V, generator=gen) * 1e-9
    for b, v in enumerate(places):
        target[b, :, v] = 1.0
    for u in (0.0, 1e-7, 0.5, 0.9999999):
        c = dict(target=target, draft=draft, draft_tokens=torch.zeros(B, 1).int() + 7,
                 u_accept=torch.full((B, 1), 0.7), u_sample=torch.full((B,), u))
        for dt in (torch.float32, torch.bfloat16):
            check(g, dict(c, target=target.to(dt), draft=draft.to(dt)))
            check(g, dict(c, target=target.to(dt), draft=None))


def test_offsets_past_31_bits(g):
    """A target of 2.7e9 entries: the last sequence, alone and in the batch."""
    print("\n  verify: offsets past 2^31", flush=True)
    B, K, V = 512, 20, 250001
    c = make(1, K, V, torch.float32, 3)
    c["u_accept"] *= 0.2
    target = torch.zeros(B, K + 1, V, dtype=torch.float16, device="cuda")
    draft = torch.zeros(B, K, V, dtype=torch.float16, device="cuda")
    c["target"], c["draft"] = c["target"].half(), c["draft"].half()
    target[-1], draft[-1] = c["target"][0].cuda(), c["draft"][0].cuda()
    d = torch.zeros(B, K, dtype=torch.int32, device="cuda")
    d[-1] = c["draft_tokens"][0].cuda()
    ua, us = torch.zeros(B, K, device="cuda"), torch.zeros(B, device="cuda")
    ua[-1], us[-1] = c["u_accept"][0].cuda(), c["u_sample"][0].cuda()
    acc = torch.empty(B, dtype=torch.int32, device="cuda")
    tok = torch.empty(B, K + 1, dtype=torch.int32, device="cuda")
    ws = torch.empty(g.verify_workspace_bytes(B, V), dtype=torch.uint8, device="cuda")
    g.verify(target, draft, d, ua, us, acc, tok, workspace=ws)
    want = sr.verify(c["target"], c["draft"], c["draft_tokens"], c["u_accept"], c["u_sample"])
    torch.cuda.synchronize()
    assert int(acc[-1]) == want[0][0] and tok[-1].tolist() == want[1][0].tolist()
    assert not bool(acc[:-1].any()) and bool((tok[:-1] == -1).all())


@pytest.mark.parametrize("layers,B,Hv,ring", [(1, 1, 32, None), (1, 5, 32, (3, 8192)), (3, 4, 16, (3, 4096)),
                                              (2, 3, 1, (1, 100)), (1, 33, 2, (7, 4))])
def test_commit(g, layers, B, Hv, ring):
    print(f"\n  pair_commit layers={layers} B={B} Hv={Hv} ring={ring}", flush=True)
    gen = torch.Generator().manual_seed(B)
    rand = lambda *s: torch.randn(*s, generator=gen)
    M, N = rand(layers, B, Hv, 128, 128), rand(layers, B, Hv, 128, 128)
    C = rand(layers, B, *ring) if ring else None
    Cn = rand(layers, B, *ring) if ring else None
    for acc in (torch.zeros(B), torch.ones(B), torch.randint(-2, 4, (B,), generator=gen)):
        acc = acc.int()
        m, n = M.cuda(), N.cuda()
        c, cn = (C.cuda(), Cn.cuda()) if ring else (None, None)
        if layers == 1:
            g.pair_commit(acc.cuda(), m[0], n[0], c[0] if ring else None, cn[0] if ring else None)
        else:
            g.pair_commit(acc.cuda(), m, n, c, cn)
        torch.cuda.synchronize()
        keep = (acc >= 1).view(1, B, 1, 1)
        assert torch.equal(m.cpu(), torch.where(keep[..., None], N, M)) and torch.equal(n.cpu(), N)
        if ring:
            assert torch.equal(c.cpu(), torch.where(keep, Cn, C)) and torch.equal(cn.cpu(), Cn)


def test_commit_past_31_bits(g):
    """States of 2.2e9 floats: the last sequence of the last layer."""
    print("\n  pair_commit: offsets past 2^31", flush=True)
    layers, B = 2, 2050
    m = torch.zeros(layers, B, 32, 128, 128, device="cuda")
    n = torch.zeros_like(m)
    n[:, -2:] = 1.0
    acc = torch.zeros(B, dtype=torch.int32, device="cuda")
    acc[-1] = 1
    g.pair_commit(acc, m, n)
    torch.cuda.synchronize()
    assert bool((m[:, -1] == 1).all()) and not bool(m[:, :-1].any())


def test_refusals_on_the_gpu(g):
    c = {k: t.cuda() for k, t in make(3, 2, 50, torch.float32, 1).items()}
    acc = torch.full((3,), 9, dtype=torch.int32, device="cuda")
    tok = torch.full((3, 3), 9, dtype=torch.int32, device="cuda")
    ws = torch.empty(g.verify_workspace_bytes(3, 50), dtype=torch.uint8, device="cuda")

    def f(**over):
        x = dict(c, accepted=acc, tokens=tok, workspace=ws)
        x.update(over)
        g.verify(**x)

    for bad in (dict(target=c["target"].double()), dict(draft=c["draft"].half()),
                dict(draft=c["draft"][:, :1]), dict(draft_tokens=c["draft_tokens"].long()),
                dict(u_accept=c["u_accept"].double()), dict(tokens=tok[:, :2]), dict(workspace=None),
                dict(workspace=ws[:-1]), dict(workspace=ws.cpu()), dict(accepted=tok.view(-1)[:3]),
                dict(n_draft=acc), dict(n_draft=acc.long()), dict(target=c["target"][:, :1]),
                dict(target=None)):
        with pytest.raises((g.GdnError, TypeError, ValueError)):
            f(**bad)
    m = torch.full((3, 2, 128, 128), 4.0, device="cuda")
    n, ring = torch.zeros_like(m), torch.zeros(3, 3, 100, device="cuda")
    for bad in (lambda: g.pair_commit(acc, m, m), lambda: g.pair_commit(acc[:2], m, n),
                lambda: g.pair_commit(acc.long(), m, n), lambda: g.pair_commit(acc, m, n[:2]),
                lambda: g.pair_commit(acc, m[..., :64], n[..., :64]),
                lambda: g.pair_commit(acc, m, n, ring, None), lambda: g.pair_commit(acc, m, n, None, ring),
                lambda: g.pair_commit(acc, m, n, ring, ring),
                lambda: g.pair_commit(acc, m, n, ring[..., :1].contiguous(), ring[..., 1:2].contiguous())):
        with pytest.raises((g.GdnError, TypeError, ValueError)):
            bad()
    torch.cuda.synchronize()
    assert bool((acc == 9).all()) and bool((tok == 9).all()) and bool((m == 4.0).all())
