"""GPU: gdn_chunk and gdn_decode over packed sequences against the recurrence in
64 bits."""
import threading

import pytest
import torch

import rule_ref as rr

pytestmark = pytest.mark.gpu
D = rr.D


@pytest.fixture(scope="module")
def g():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import gated_deltanet_decode_amd as g
    return g


def chunk(g, x, state_out="new", stream=None, ws=None):
    hv, hk = x["v"].shape[1], x["q"].shape[1]
    B = x["offsets"].shape[0] - 1
    dims = g.Dims(hv, hk, D, D)
    if ws is None:
        ws = torch.empty(g.chunk_workspace_bytes(B, x["q"].shape[0], x["q"].dtype, dims), dtype=torch.uint8, device="cuda")
        ws.fill_(255)                                     # NaN wherever nothing was written
    out = torch.full(x["v"].shape, 7.0, dtype=x["v"].dtype, device="cuda")
    n = x["state"].shape[0] if x["state"] is not None else B
    so = torch.full((n, hv, D, D), 5.0, device="cuda") if state_out == "new" else state_out
    g.chunk(x["q"], x["k"], x["v"], x["beta"], x["gate"], out, state=x["state"], state_out=so, offsets=x["offsets"],
            slots=x["slots"], workspace=ws, stream=stream)
    return out, so


def decode(g, x, state_out="new"):
    out = torch.full(x["v"].shape, 7.0, dtype=x["v"].dtype, device="cuda")
    so = torch.full(x["state"].shape, 5.0, device="cuda") if state_out == "new" else state_out
    g.decode(x["q"], x["k"], x["v"], x["beta"], x["gate"], out, x["state"], state_out=so, offsets=x["offsets"],
             slots=x["slots"])
    return out, x["state"] if so is None else so


def check(x, out, so, dtype, more=1):
    y, pool, size, psize = rr.forward(x)
    used = x["offsets"][-1].item()
    o = out.cpu().double()
    bound = rr.out_bound(y, size, dtype)
    assert ((o - y).abs()[:used] <= bound[:used]).all(), float(((o - y).abs() / bound)[:used].max())
    assert (o[used:] == 7.0).all()                        # rows behind the last sequence
    live = torch.zeros(pool.shape[0], dtype=torch.bool)
    live[torch.tensor([s for _, _, s in rr._spans(rr._host(x)) if 0 <= s < pool.shape[0]], dtype=torch.long)] = True
    s = so.cpu().double()
    bound = rr.state_bound(psize)
    assert ((s - pool).abs() <= bound)[live].all(), float(((s - pool).abs() / bound)[live].max())
    if live.any():
        assert rr.rel(s[live], pool[live]) <= more * 2.0 ** -20   # roundings of 2^-24, some hundreds, independent
    assert (s[~live] == 5.0).all()                        # slots of no sequence


LENS = [[1], [2, 0, 1], [63], [64], [65], [128, 0, 0, 1, 200, 127], [0], [1000]]


@pytest.mark.parametrize("dtype", rr.TYPES.values(), ids=rr.TYPES)
@pytest.mark.parametrize("lens", LENS, ids=str)
def test_chunk_lengths(g, lens, dtype):
    x = rr.inputs(lens, 4, 2, dtype, 1, tail=3)
    check(x, *chunk(g, x), dtype)


@pytest.mark.parametrize("hv,hk", [(1, 1), (3, 1), (6, 2), (5, 5), (16, 4)])
def test_chunk_heads(g, hv, hk):
    x = rr.inputs([70, 5], hv, hk, torch.bfloat16, 2, start=False)
    check(x, *chunk(g, x), torch.bfloat16)


@pytest.mark.parametrize("dtype", rr.TYPES.values(), ids=rr.TYPES)
@pytest.mark.parametrize("gate", [0.0, -1e-4, -3.0, -50.0, -700.0, -1e30, float("-inf"), 0.01])
def test_chunk_gates(g, gate, dtype):
    x = rr.inputs([130], 2, 1, dtype, 3, gate=gate)
    check(x, *chunk(g, x), dtype)


@pytest.mark.parametrize("dtype", rr.TYPES.values(), ids=rr.TYPES)
def test_chunk_one_strong_decay(g, dtype):
    """The tokens after a token that forgets everything keep their accuracy."""
    x = rr.inputs([200], 2, 2, dtype, 4, gate=-0.001)
    x["gate"][5], x["gate"][70], x["gate"][133] = -1e4, -1e35, float("-inf")
    check(x, *chunk(g, x), dtype)


def test_chunk_slight_decays(g):
    """Gates from nothing at all over what float64 just tells from it beside 1 to strong."""
    x = rr.inputs([130, 64, 1, 70], 4, 2, torch.float32, 31)
    kinds = torch.tensor([0.0, -0.0, -1e-38, -2.0**-60, -2.0**-54, -1e-12, -1e-5, -0.3, -1.0, -50.3], device="cuda")
    x["gate"] = kinds[torch.randint(0, len(kinds), x["gate"].shape, generator=torch.Generator().manual_seed(3)).cuda()]
    x["gate"][:64] = -2.0**-60                            # a chunk of nothing else
    check(x, *chunk(g, x), torch.float32)


def test_chunk_same_key_and_full_writes(g):
    """Keys that are all alike and beta 1: the triangular system is as full as it
    gets, every token replaces what the one before it wrote.  The corrections are
    v_j - v_(j-1), of norm sqrt(2) |v|, and their sum over 128 tokens, of norm |v|,
    carries the independent roundings of all of them: sqrt(2 * 128) = 16 times one's
    where a sum that does not cancel has its own size."""
    x = rr.inputs([128], 2, 1, torch.float32, 5, gate=0.0)
    x["k"][:] = x["k"][0]
    x["beta"][:] = 1.0
    check(x, *chunk(g, x), torch.float32, more=16)


@pytest.mark.parametrize("call", ["chunk", "decode"])
def test_slots(g, call):
    """States anywhere in a pool, and sequences that are left out."""
    x = rr.inputs([3, 70, 0, 9, 4], 4, 2, torch.bfloat16, 6, tail=2, pool=11)
    run = chunk if call == "chunk" else decode
    check(x, *run(g, x), torch.bfloat16)
    x["slots"][1], x["slots"][4] = -1, 11
    out, so = run(g, x)
    o = x["offsets"].tolist()
    for b in (1, 4):
        assert (out[o[b]:o[b + 1]] == 7.0).all()
    keep = [t for b in (0, 3) for t in range(o[b], o[b + 1])]
    y, pool, size, _ = rr.forward(x)
    assert ((out.cpu().double() - y).abs() <= rr.out_bound(y, size, torch.bfloat16))[keep].all()
    named = x["slots"][[0, 2, 3]].tolist()
    for s in range(11):
        if s in named:
            assert rr.rel(so[s], pool[s]) <= 2.0 ** -20
        else:
            assert (so[s] == 5.0).all()


@pytest.mark.parametrize("dtype", rr.TYPES.values(), ids=rr.TYPES)
@pytest.mark.parametrize("lens", [[1], [1, 0, 1, 1], [4, 1, 7], [40]], ids=str)
def test_decode(g, lens, dtype):
    x = rr.inputs(lens, 4, 2, dtype, 7, tail=2)
    check(x, *decode(g, x), dtype)


def test_decode_is_step(g):
    """float32: the bits of gdn_step."""
    x = rr.inputs([1] * 9, 32, 16, torch.float32, 8)
    out, so = decode(g, x)
    want = torch.empty_like(x["v"])
    state = x["state"].clone()
    g.step(x["q"], x["k"], x["v"], x["beta"], x["gate"], state, want)
    assert torch.equal(out, want) and torch.equal(so, state)


@pytest.mark.parametrize("call", ["chunk", "decode"])
def test_in_place_and_dense(g, call):
    """state_out may be state, and [B][T] without offsets is offsets of T."""
    x = rr.inputs([66, 66], 4, 2, torch.bfloat16, 9)
    run = chunk if call == "chunk" else decode
    out, so = run(g, x)
    y = dict(x, state=x["state"].clone())
    out2, so2 = run(g, y, state_out=y["state"])
    assert torch.equal(out, out2) and torch.equal(so, so2) and so2 is y["state"]
    two = lambda t: t.unflatten(0, (2, 66))
    out3, st = torch.empty_like(two(x["v"])), x["state"].clone()
    if call == "chunk":
        ws = torch.empty(g.chunk_workspace_bytes(2, 132, torch.bfloat16, g.Dims(4, 2, D, D)), dtype=torch.uint8, device="cuda")
        g.chunk(*(two(x[n]) for n in ("q", "k", "v", "beta", "gate")), out3, state=st, state_out=st, workspace=ws)
    else:
        g.decode(*(two(x[n]) for n in ("q", "k", "v", "beta", "gate")), out3, st)
    assert torch.equal(out3.flatten(0, 1), out) and torch.equal(st, so)


def test_no_state_wanted(g):
    x = rr.inputs([100], 2, 1, torch.bfloat16, 10, start=False)
    out, _ = chunk(g, x, state_out=None)
    assert torch.equal(out, chunk(g, x)[0])


def test_independent_of_the_batch(g):
    """A sequence alone gives the bits it has among others, and a second call
    gives them again."""
    x = rr.inputs([70, 300, 5], 4, 2, torch.bfloat16, 11)
    out, so = chunk(g, x)
    again, so2 = chunk(g, x)
    assert torch.equal(out, again) and torch.equal(so, so2)
    cut = lambda t: t[70:370].contiguous()
    one = {n: cut(x[n]) for n in ("q", "k", "v", "beta", "gate")}
    one.update(offsets=torch.tensor([0, 300], dtype=torch.int32, device="cuda"), slots=None, state=x["state"][1:2].clone())
    out1, so1 = chunk(g, one)
    assert torch.equal(out1, out[70:370]) and torch.equal(so1[0], so[1])


def test_chunk_then_decode(g):
    """A prompt in chunks and the tokens after it one by one are the sequence."""
    x = rr.inputs([75], 4, 2, torch.float32, 12)
    y, pool, size, psize = rr.forward(x)
    head = {n: x[n][:70].contiguous() for n in ("q", "k", "v", "beta", "gate")}
    off = lambda n: torch.tensor([0, n], dtype=torch.int32, device="cuda")
    out, so = chunk(g, dict(head, offsets=off(70), slots=None, state=x["state"]))
    outs = [out]
    for t in range(70, 75):
        tok = {n: x[n][t:t + 1].contiguous() for n in ("q", "k", "v", "beta", "gate")}
        o, _ = decode(g, dict(tok, offsets=off(1), slots=None, state=so), state_out=None)
        outs.append(o)
    o = torch.cat(outs).cpu().double()
    assert ((o - y).abs() <= rr.out_bound(y, size, torch.float32)).all()
    assert rr.rel(so, pool) <= 2.0 ** -20


def test_foreign_offsets(g):
    """Offsets outside the tensors count as their ends; nothing else is touched."""
    x = rr.inputs([20, 30], 2, 1, torch.bfloat16, 13)
    good, so = chunk(g, x)
    y = dict(x, offsets=torch.tensor([-5, 20, 1 << 30], dtype=torch.int32, device="cuda"))
    out, so2 = chunk(g, y)
    assert torch.equal(out, good) and torch.equal(so, so2)
    out, so3 = decode(g, y)
    assert torch.equal(out, decode(g, x)[0])
    y = dict(x, offsets=torch.tensor([30, 10, 50], dtype=torch.int32, device="cuda"))    # the first is empty
    out, so4 = chunk(g, y)
    assert torch.equal(so4[0], x["state"][0])


def test_nan_stays_with_its_sequence(g):
    x = rr.inputs([100, 100], 2, 1, torch.bfloat16, 14)
    good, so = chunk(g, x)
    y = dict(x, v=x["v"].clone(), k=x["k"].clone())
    y["v"][90] = float("nan")
    y["k"][95] = float("inf")
    out, so2 = chunk(g, y)
    assert torch.equal(out[:64], good[:64]) and torch.equal(out[100:], good[100:]) and torch.equal(so2[1], so[1])
    assert out[95:100].isnan().all() and so2[0].isnan().any()


def test_graph_stream_threads(g):
    """Captured and replayed between eager work, on another stream, and from two
    threads with a workspace each."""
    x = rr.inputs([130, 40], 8, 4, torch.bfloat16, 15)
    dims = g.Dims(8, 4, D, D)
    ws = [torch.empty(g.chunk_workspace_bytes(2, 170, torch.bfloat16, dims), dtype=torch.uint8, device="cuda") for _ in range(3)]
    want, so = chunk(g, x, ws=ws[0])
    out, st = torch.empty_like(want), torch.empty_like(so)
    call = lambda w: g.chunk(x["q"], x["k"], x["v"], x["beta"], x["gate"], out, state=x["state"], state_out=st,
                             offsets=x["offsets"], workspace=w)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call(ws[1])
    s.synchronize()
    assert torch.equal(out, want) and torch.equal(st, so)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(ws[1])
    for _ in range(3):
        out.zero_()
        st.zero_()
        graph.replay()
        other, _ = chunk(g, x, ws=ws[0])
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(st, so) and torch.equal(other, want)
    bad = []

    def work(w):
        st_ = torch.cuda.Stream()
        with torch.cuda.stream(st_):
            for _ in range(5):
                o, _ = chunk(g, x, ws=w, stream=st_)
                st_.synchronize()
                if not torch.equal(o, want):
                    bad.append(w)
    torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=(ws[i],)) for i in (1, 2)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not bad
