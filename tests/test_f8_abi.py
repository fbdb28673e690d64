"""CPU: the 8-bit floating point operators reject bad arguments with the
documented codes before they touch the GPU."""
import pytest
import torch

BASE = 1 << 40
STEP = 1 << 36


@pytest.fixture(scope="module")
def g():
    import gated_deltanet_decode_amd as g
    return g


def expect(g, rc, code, needle):
    assert rc == code, f"rc={rc} ({g.ERRORS.get(rc)}), expected {g.ERRORS[code]}: {g.last_error()}"
    assert needle in g.last_error(), g.last_error()


def slots(names):
    return {n: BASE + i * STEP for i, n in enumerate(names)}


def test_quantize(g):
    base = slots(("x", "q", "scale"))

    def f(rows=4, n=300, br=1, t=0, **over):
        a = dict(base, **over)
        return g.lib.gdn_quantize_f8(rows, n, br, t, a["x"], a["q"], a["scale"], None)

    for n in base:
        expect(g, f(**{n: None}), -1, n)
    expect(g, f(rows=0), -2, "rows")
    expect(g, f(n=0), -2, "n must")
    expect(g, f(n=1 << 30), -2, "n must")
    expect(g, f(br=2), -2, "block_rows")
    expect(g, f(br=0), -2, "block_rows")
    expect(g, f(t=3), -2, "x_type")
    expect(g, f(rows=(1 << 29) - 31, n=1), -2, "scales")
    expect(g, f(rows=1 << 21, n=1 << 18, br=128), -2, "scales")
    expect(g, f(x=base["x"] + 8), -3, "aligned")
    expect(g, f(q=base["q"] + 8), -3, "aligned")
    expect(g, f(scale=base["scale"] + 2), -3, "aligned")
    expect(g, f(q=base["x"]), -4, "q overlaps")
    expect(g, f(scale=base["q"] + 4 * 300 - 4), -4, "overlaps")


def test_linear(g):
    base = slots(("a", "sa", "w", "sw", "bias", "o0", "o1", "o2", "o3"))

    def f(M=4, K=300, t=0, ns=(130, 8), n_outs=None, null=False, **over):
        a = dict(base, **over)
        outs = (g.LinearOut * 4)()
        for i, n in enumerate(ns):
            outs[i].out, outs[i].n = a[f"o{i}"], n
        return g.lib.gdn_linear_f8(M, K, a["a"], a["sa"], a["w"], a["sw"], a["bias"], t, None if null else outs,
                                   len(ns) if n_outs is None else n_outs, None)

    for n, s in (("a", "a"), ("w", "w"), ("sa", "a_scale"), ("sw", "w_scale"), ("o1", "outs[1]")):
        expect(g, f(**{n: None}), -1, s)
    expect(g, f(null=True), -1, "outs")
    expect(g, f(M=0), -2, "M must")
    expect(g, f(K=0), -2, "K must")
    expect(g, f(K=4194304), -2, "K must")
    expect(g, f(t=-1), -2, "out_type")
    expect(g, f(n_outs=0), -2, "n_outs")
    expect(g, f(n_outs=5), -2, "n_outs")
    expect(g, f(ns=(8, 0)), -2, "outs[1].n")
    expect(g, f(ns=(1 << 27,)), -2, "too large")
    expect(g, f(M=1 << 26, ns=(1 << 10,)), -2, "too large")
    for n in ("a", "w", "o0"):
        expect(g, f(**{n: base[n] + 8}), -3, "aligned")
    for n in ("sa", "sw", "bias"):
        expect(g, f(**{n: base[n] + 2}), -3, "aligned")
    expect(g, f(o0=base["a"]), -4, "outs[0] overlaps a")
    expect(g, f(o1=base["o0"]), -4, "outs[0]")
    expect(g, f(o0=base["sa"] + 4 * 3 * 4 - 4 - (4 * 3 * 4 - 4) % 16), -4, "a_scale")
    expect(g, f(o0=base["sw"] + 16), -4, "w_scale")


def test_binding(g):
    with pytest.raises(ValueError, match="GPU"):
        g.quantize_f8(torch.zeros(2, 5), None, None)
    with pytest.raises(ValueError, match="GPU"):
        g.linear_f8(torch.zeros(2, 5).to(torch.float8_e4m3fn), None, None, None, None)
