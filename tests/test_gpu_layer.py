"""GPU: the quantised norm, the 8-bit projections, the recurrent tail, the
verification and the commit together, as a decode loop uses them: a layer of the
page's geometry (hidden 2048) for single tokens and for the speculative pair.
Every stage is checked on the inputs that the stage before it left on the GPU;
the whole chain is replayed from a graph, issued on another stream and from two
threads, with the bits of eager calls."""
import threading

import numpy as np
import pytest
import torch

import gdn_inputs as gi
import serve_ref as sr

pytestmark = pytest.mark.gpu

HIDDEN, C, NV, HV = 2048, 8192, 4096, 32


@pytest.fixture(scope="module")
def g():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import gated_deltanet_decode_amd as g
    return g


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def weights(seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    codes = lambda *s: (torch.randn(*s, device="cuda", generator=gen) * 32).round_().clamp_(-127, 127).to(torch.int8)
    scale = lambda n: (0.5 + torch.rand(n, device="cuda", generator=gen)) / (32 * HIDDEN ** 0.5)
    ti = gi.tail_inputs(seed, 1)
    gin = gi.gate_inputs(seed, 1)
    return dict(norm=1.0 + 0.02 * torch.randn(HIDDEN, device="cuda", generator=gen),
                w_in=codes(C + NV + 2 * HV, HIDDEN), s_in=scale(C + NV + 2 * HV),
                w_out=codes(HIDDEN, NV), s_out=scale(HIDDEN), conv_w=dev(ti["conv_w"]),
                norm_w=dev(ti["norm_w"]), a_log=dev(gin["a_log"]), dt_bias=dev(gin["dt_bias"]))


def buffers(B, positions, seed):
    """The streams, states and scratch of B sequences, `positions` tokens each."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    R = B * positions
    e = lambda *s, dtype=torch.float32: torch.empty(*s, device="cuda", dtype=dtype)
    ti = gi.tail_inputs(seed, B)
    b = dict(branch=torch.randn(R, HIDDEN, device="cuda", generator=gen).bfloat16(),
             stream=torch.randn(R, HIDDEN, device="cuda", generator=gen) * 3,
             q=e(R, HIDDEN, dtype=torch.int8), qs=e(R), x=e(R, C), z=e(R, NV), ba=e(R, 2 * HV), beta=e(R, HV),
             gate=e(R, HV), y=e(R, NV), yq=e(R, NV, dtype=torch.int8), ys=e(R),
             out=e(R, HIDDEN, dtype=torch.bfloat16), ring=dev(ti["conv_state"]), state=dev(gi.state(seed, 0, B)))
    if positions == 2:
        V = 1000
        logits = torch.randn(B, 2, V, device="cuda", generator=gen) * 2
        b.update(ring_next=e(*b["ring"].shape), state_next=e(*b["state"].shape),
                 target=torch.softmax(logits, -1),
                 draft=torch.softmax(logits[:, :1] + 0.5 * torch.randn(B, 1, V, device="cuda", generator=gen), -1),
                 u_accept=torch.rand(B, 1, device="cuda", generator=gen) * 0.9,
                 u_sample=torch.rand(B, device="cuda", generator=gen), accepted=e(B, dtype=torch.int32),
                 tokens=e(B, 2, dtype=torch.int32))
        b["drafted"] = b["draft"].argmax(-1).int()
    return b


def layer(g, w, b, ws=None, stream=None):
    """One layer; with a pair also the decision about the draft and what follows."""
    pair = "ring_next" in b
    R = b["x"].shape[0]
    g.add_rmsnorm_q8(b["branch"], b["stream"], b["stream"], w["norm"], b["q"], b["qs"], stream=stream)
    g.linear_q8(b["q"], b["qs"], w["w_in"], w["s_in"], [b["x"], b["z"], b["ba"]], stream=stream)
    if pair:
        B = R // 2
        g.gate_transform(b["ba"], w["a_log"], w["dt_bias"], b["beta"], b["gate"], stream=stream)
        g.layer_tail_pair(b["x"].view(B, 2, C), w["conv_w"], b["ring"], b["ring_next"], b["beta"].view(B, 2, HV),
                          b["gate"].view(B, 2, HV), b["state"], b["state_next"], b["z"].view(B, 2, NV),
                          w["norm_w"], b["y"].view(B, 2, NV), stream=stream)
    else:
        g.layer_tail_ba(b["x"], w["conv_w"], b["ring"], b["ba"], w["a_log"], w["dt_bias"], b["state"], b["z"],
                        w["norm_w"], b["y"], stream=stream)
    g.quantize_q8(b["y"], b["yq"], b["ys"], stream=stream)
    g.linear_q8(b["yq"], b["ys"], w["w_out"], w["s_out"], b["out"], stream=stream)
    if pair:
        g.verify(b["target"], b["draft"], b["drafted"], b["u_accept"], b["u_sample"], b["accepted"], b["tokens"],
                 workspace=ws, stream=stream)
        g.pair_commit(b["accepted"], b["state"], b["state_next"], b["ring"], b["ring_next"], stream=stream)


def scratch(g, B):
    return torch.empty(g.verify_workspace_bytes(B, 1000), dtype=torch.uint8, device="cuda")


def close(got, want, tol):
    err = np.abs(sr.f64(got) - want)
    assert np.all(err <= tol), float((err - tol).max())


@pytest.mark.parametrize("B", [1, 7, 32])
def test_decoded_layer_stage_by_stage(g, orc, B):
    print(f"\n  decoded layer, B={B}", flush=True)
    w, b = weights(8100), buffers(B, 1, 8200 + B)
    for token in range(3):
        before = {k: t.clone() for k, t in b.items()}
        layer(g, w, b)
        torch.cuda.synchronize()
        h = sr.stored_sum(before["branch"], before["stream"])
        assert torch.equal(b["stream"].cpu(), h)
        q, s = sr.rmsnorm_q8(h, w["norm"], 1e-6)
        assert np.array_equal(b["q"].cpu().numpy(), q)
        assert np.all(np.abs(sr.f64(b["qs"]) - s) <= s * 2.0 ** -22)
        y, tol = sr.linear_q8(b["q"], b["qs"], w["w_in"], w["s_in"], None, torch.float32)
        close(torch.cat([b["x"], b["z"], b["ba"]], 1), y, tol)
        n = lambda t: t.cpu().numpy()
        beta, gate = orc.gate_transform(n(b["ba"]), n(w["a_log"]), n(w["dt_bias"]))
        ring, M = n(before["ring"]).copy(), n(before["state"]).copy()
        yo, _, _ = orc.layer_tail(n(b["x"]), n(w["conv_w"]), ring, beta, gate, M, n(b["z"]), n(w["norm_w"]),
                                  16, 128)
        assert np.array_equal(n(b["ring"]), ring)
        assert np.abs(n(b["state"]) - M).max() <= 1e-6
        assert np.abs(n(b["y"]) - yo).max() <= 1e-5
        q, s = sr.quantize_q8(b["y"])
        assert np.array_equal(n(b["yq"]), q)
        assert np.all(np.abs(sr.f64(b["ys"]) - s) <= s * 2.0 ** -23)
        y, tol = sr.linear_q8(b["yq"], b["ys"], w["w_out"], w["s_out"], None, torch.bfloat16)
        close(b["out"], y, tol)
        b["branch"].copy_(b["out"])


@pytest.mark.parametrize("B", [1, 6])
def test_speculative_pair_with_verification_and_commit(g, B):
    """The pair's committed and tentative buffers are those of two single layers;
    the commit keeps position 2 exactly where the draft was accepted."""
    print(f"\n  speculative layer, B={B}", flush=True)
    w, b = weights(8100), buffers(B, 2, 8300 + B)
    b["u_accept"][: (B + 1) // 2] = 0.0          # accepted
    b["u_accept"][(B + 1) // 2:] = 1.0           # refused where q >= p
    b["draft"][(B + 1) // 2:, 0] = b["target"][(B + 1) // 2:, 0]
    ring0, state0 = b["ring"].clone(), b["state"].clone()
    layer(g, w, b, scratch(g, B))
    torch.cuda.synchronize()
    want = sr.verify(b["target"], b["draft"], b["drafted"], b["u_accept"], b["u_sample"])
    assert np.array_equal(b["accepted"].cpu().numpy(), want[0])
    assert np.array_equal(b["tokens"].cpu().numpy(), want[1])
    assert b["accepted"].tolist() == [1] * ((B + 1) // 2) + [0] * (B // 2)
    ring, state = ring0, state0
    y = torch.empty(B, NV, device="cuda")
    at = lambda t, p: t.view(B, 2, -1)[:, p].contiguous()
    for p in range(2):
        r, s = ring.clone(), state.clone()
        g.layer_tail(at(b["x"], p), w["conv_w"], r, at(b["beta"], p), at(b["gate"], p), s, at(b["z"], p),
                     w["norm_w"], y)
        torch.cuda.synchronize()
        assert torch.equal(y, at(b["y"], p))
        for k in range(B):
            if int(b["accepted"][k]) == p:
                assert torch.equal(b["ring"][k], r[k]) and torch.equal(b["state"][k], s[k])
        ring, state = r, s


@pytest.mark.parametrize("B,positions", [(3, 1), (3, 2), (40, 1)])
def test_graph_replays_are_eager_calls(g, B, positions):
    print(f"\n  layer in a graph, B={B} positions={positions}", flush=True)
    w, eager, ws = weights(8100), buffers(B, positions, 8400 + B), scratch(g, B)
    graph = {k: t.clone() for k, t in eager.items()}
    second = {k: t.clone() for k, t in eager.items()}
    layer(g, w, {k: t.clone() for k, t in eager.items()}, ws)
    side = torch.cuda.Stream()
    graphs = []
    for bufs in (graph, second):                  # two graphs that share the workspace
        gr = torch.cuda.CUDAGraph()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(gr, stream=side):
            layer(g, w, bufs, ws)
        graphs.append(gr)
    torch.cuda.synchronize()
    for rep in range(4):
        graphs[0].replay()
        layer(g, w, eager, ws)
        graphs[1].replay()
        torch.cuda.synchronize()
        for k in eager:
            assert torch.equal(graph[k], eager[k]), f"replay {rep}: {k}"
            assert torch.equal(second[k], eager[k]), f"replay {rep}: {k} (second graph)"
        for b in (eager, graph, second):
            b["branch"].copy_(b["out"])


def test_another_stream_and_two_threads(g):
    print("\n  layer on other streams and threads", flush=True)
    w = weights(8100)
    want, mine = [], []
    for i, (B, positions) in enumerate(((5, 2), (9, 1))):
        b = buffers(B, positions, 8500 + i)
        mine.append({k: t.clone() for k, t in b.items()})
        layer(g, w, b, scratch(g, B))
        want.append(b)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    spaces = [scratch(g, 5), scratch(g, 9)]
    once = [{k: t.clone() for k, t in b.items()} for b in mine]
    torch.cuda.synchronize()
    for b, s, ws in zip(once, streams, spaces):
        layer(g, w, b, ws, stream=s)
    torch.cuda.synchronize()
    for b, c in zip(once, want):
        assert all(torch.equal(b[k], c[k]) for k in c)
    failed = []

    def work(i):
        try:
            for _ in range(20):
                b = {k: t.clone() for k, t in mine[i].items()}
                streams[i].wait_stream(torch.cuda.current_stream())
                with torch.cuda.stream(streams[i]):
                    layer(g, w, b, spaces[i])
                streams[i].synchronize()
                for k in want[i]:
                    if not torch.equal(b[k], want[i][k]):
                        failed.append((i, k))
        except Exception as e:                    # shown below, in the main thread
            failed.append((i, repr(e)))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed[:3]


def test_messages_stay_with_their_call(g):
    """A refused call names its reason and the next call is unaffected."""
    q = torch.full((2, 16), 3, dtype=torch.int8, device="cuda")
    s = torch.zeros(2, device="cuda")
    x = torch.randn(2, 16, device="cuda")
    with pytest.raises(g.GdnError, match="GDN_ERR_ALIAS"):
        g.add_rmsnorm_q8(x, x, x, torch.ones(16, device="cuda"), q, s)
    g.quantize_q8(x, q, s)
    torch.cuda.synchronize()
    assert g.last_error() == "" and int(q.abs().max()) == 127


def test_sizes_past_32_bits_are_refused(g):
    """The C arguments are 32 bits wide: a dimension that would wrap around to a
    small one (here of expanded tensors, that take no memory) is refused."""
    wide = 2 ** 32 + 3
    one = lambda dtype, *s: torch.zeros(*[1] * len(s), dtype=dtype, device="cuda").expand(*s)
    v = torch.zeros(3, device="cuda")
    i8 = torch.int8
    for shape in ((wide, 2), (2, wide)):
        with pytest.raises(ValueError, match="no dimension may pass"):
            g.quantize_q8(one(torch.float16, *shape), one(i8, *shape), v)
        with pytest.raises(ValueError, match="no dimension may pass"):
            g.add_rmsnorm_q8(one(torch.float32, *shape), None, None, v, one(i8, *shape), v)
        with pytest.raises(ValueError, match="no dimension may pass"):
            g.linear_q8(one(i8, *shape), v, one(i8, 3, 2), v, one(torch.float32, 2, 3))
    with pytest.raises(ValueError, match="no dimension may pass"):
        g.linear_q8(one(i8, 2, 16), v, one(i8, wide + 2, 16), v,
                    [torch.zeros(2, 2, device="cuda"), one(torch.float32, 2, wide)])
    i32 = torch.zeros(2, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="no dimension may pass"):
        g.verify(one(torch.float32, 1, 2, wide), None, i32[:1].view(1, 1), v[:1].view(1, 1), v[:1], i32[:1],
                 i32.view(1, 2), workspace=torch.empty(4096, dtype=torch.uint8, device="cuda"))
    state = torch.zeros(1, 1, 128, 128, device="cuda")
    ring = one(torch.float32, 1, 2 ** 16, 2 ** 16 + 4)
    with pytest.raises(ValueError, match="floats a sequence"):
        g.pair_commit(i32[:1], state, state.clone(), ring, ring)
