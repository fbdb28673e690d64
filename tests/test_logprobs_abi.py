"""CPU: gdn_logprobs rejects bad arguments with the documented codes before it
touches the GPU."""
import pytest
import torch

BASE = 1 << 40
STEP = 1 << 36
NAMES = ("logits", "tokens", "logprob", "entropy", "ids", "lps", "ws")


@pytest.fixture(scope="module")
def g():
    import gated_deltanet_decode_amd as g
    return g


def expect(g, rc, code, needle):
    assert rc == code, f"rc={rc} ({g.ERRORS.get(rc)}), expected {g.ERRORS[code]}: {g.last_error()}"
    assert needle in g.last_error(), g.last_error()


def test_refusals(g):
    base = {n: BASE + i * STEP for i, n in enumerate(NAMES)}

    def f(rows=4, V=50000, ld=None, t=0, top=5, bytes=None, **over):
        a = dict(base, **over)
        if bytes is None:
            bytes = g.logprobs_workspace_bytes(rows, V, top)
        return g.lib.gdn_logprobs(rows, V, V if ld is None else ld, t, a["logits"], a["tokens"], a["logprob"], a["entropy"],
                                  top, a["ids"], a["lps"], a["ws"], bytes, None)

    for n in ("logits", "tokens", "logprob"):
        expect(g, f(**{n: None}), -1, n)
    expect(g, f(ids=None), -1, "top_ids")
    expect(g, f(lps=None), -1, "top_logprobs")
    expect(g, f(tokens=None, logprob=None, entropy=None, top=0), -1, "nothing else")
    expect(g, f(rows=0), -2, "rows")
    expect(g, f(rows=4194304), -2, "rows")
    expect(g, f(V=0), -2, "V must")
    expect(g, f(V=(1 << 30) + 1), -2, "V must")
    expect(g, f(top=65), -2, "top")
    expect(g, f(top=-1), -2, "top")
    expect(g, f(V=4, top=5), -2, "top")
    expect(g, f(ld=49999), -2, "ld")
    expect(g, f(t=3), -2, "logit_type")
    expect(g, f(logits=base["logits"] + 2), -3, "logits")
    expect(g, f(t=1, logits=base["logits"] + 1), -3, "logits")
    for n in ("tokens", "logprob", "entropy", "ids", "lps"):
        expect(g, f(**{n: base[n] + 2}), -3, "aligned")
    expect(g, f(ws=None), -5, "NULL")
    expect(g, f(bytes=8), -5, "needed")
    expect(g, f(ws=base["ws"] + 8), -3, "workspace")
    expect(g, f(logprob=base["tokens"]), -4, "logprob")
    expect(g, f(entropy=base["logits"] + 4 * 50000 * 4 - 4), -4, "entropy")
    expect(g, f(ids=base["lps"] + 16), -4, "top_ids")
    expect(g, f(ws=base["logits"]), -4, "workspace")


def test_workspace(g):
    f = g.logprobs_workspace_bytes
    assert f(1, 131072, 20) > f(1, 131072, 0) > 0 and f(1, 100, 5) == 0 and f(100000, 131072, 5) == 0
    assert f(0, 5, 0) == 0 and f(1, 0, 0) == 0 and f(1 << 40, 5, 0) == 0 and f(5, 5, 6) == 0


def test_binding_refusals(g):
    with pytest.raises(ValueError, match="GPU"):
        g.logprobs(torch.zeros(2, 5))
    with pytest.raises(TypeError, match="float32, bfloat16"):
        g.logprobs(torch.zeros(2, 5, dtype=torch.float64))
