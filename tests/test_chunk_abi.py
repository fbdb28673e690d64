"""CPU: the delta rule over packed sequences rejects bad arguments with the
documented codes before it touches the GPU."""
import ctypes

import pytest
import torch

BASE = 1 << 40
STEP = 1 << 36
NAMES = ("q", "k", "v", "beta", "gate", "offsets", "slots", "state", "state_out", "out", "ws")


@pytest.fixture(scope="module")
def g():
    import gated_deltanet_decode_amd as g
    return g


def expect(g, rc, code, needle):
    assert rc == code, f"rc={rc} ({g.ERRORS.get(rc)}), expected {g.ERRORS[code]}: {g.last_error()}"
    assert needle in g.last_error(), g.last_error()


def caller(g, decode):
    base = {n: BASE + i * STEP for i, n in enumerate(NAMES)}

    def f(hv=4, hk=2, dk=128, dv=128, B=3, tokens=100, type=1, n_slots=7, bytes=None, **over):
        a = dict(base, **over)
        d = g.Dims(hv, hk, dk, dv)
        args = [ctypes.byref(d), B, tokens, type, *(a[n] for n in NAMES[:7]), n_slots, a["state"], a["state_out"], a["out"]]
        if decode:
            return g.lib.gdn_decode(*args, None)
        if bytes is None:
            bytes = g.lib.gdn_chunk_workspace_bytes(ctypes.byref(d), B, tokens, type)
        return g.lib.gdn_chunk(*args, a["ws"], bytes, None)
    f.base = base
    return f


@pytest.mark.parametrize("decode", [False, True])
def test_refusals(g, decode):
    f = caller(g, decode)
    base = f.base
    for n in ("q", "k", "v", "beta", "gate", "out") + (("state", "state_out") if decode else ()):
        expect(g, f(**{n: None}), -1, n)
    expect(g, f(hv=0), -2, "head counts")
    expect(g, f(hv=3), -2, "multiple")
    expect(g, f(dk=64), -2, "d_k")
    expect(g, f(dv=256), -2, "d_v")
    expect(g, f(hv=65536, hk=1), -2, "65535")
    expect(g, f(B=0), -2, "B must")
    expect(g, f(tokens=0), -2, "tokens must")
    expect(g, f(tokens=-4), -2, "tokens must")
    expect(g, f(type=3), -2, "type")
    expect(g, f(type=-1), -2, "type")
    expect(g, f(B=3000000), -2, "n_v_heads")
    expect(g, f(offsets=None), -2, "multiple of B")
    expect(g, f(n_slots=0), -2, "n_slots")
    expect(g, f(slots=None), -2, "n_slots")
    for n in ("q", "k", "v", "out", "state", "state_out"):
        expect(g, f(**{n: base[n] + 8}), -3, "aligned")
    for n in ("beta", "gate", "offsets", "slots"):
        expect(g, f(**{n: base[n] + 2}), -3, "aligned")
    nk, nv, ns = 100 * 2 * 128 * 2, 100 * 4 * 128 * 2, 7 * 4 * 128 * 128 * 4
    for n, size in (("q", nk), ("k", nk), ("v", nv), ("beta", 1600), ("gate", 1600), ("offsets", 16), ("slots", 12),
                    ("state", ns)):
        expect(g, f(out=(base[n] + size - 4) // 16 * 16), -4, "out overlaps")
        expect(g, f(state_out=(base[n] + size - 4) // 16 * 16), -4, "state_out overlaps")
    expect(g, f(state_out=base["out"] + nv - 16), -4, "overlaps")
    expect(g, f(state_out=base["state"] + 16), -4, "state")
    if not decode:
        expect(g, f(ws=None), -5, "NULL")
        expect(g, f(bytes=64), -5, "needed")
        expect(g, f(ws=base["ws"] + 8), -3, "workspace")
        expect(g, f(ws=base["state"]), -4, "overlaps")
        expect(g, f(ws=base["q"] + nk - 16), -4, "overlaps")
        expect(g, f(tokens=(1 << 31) - 1, bytes=1 << 60), -2, "tokens")
        expect(g, f(hv=1024, hk=1, tokens=1 << 20, bytes=1 << 60), -2, "64")
    else:
        expect(g, f(B=4194303 // 4 + 1), -2, "n_v_heads")


def test_workspace_bytes(g):
    f = g.chunk_workspace_bytes
    d = g.Dims(4, 2, 128, 128)
    assert 0 < f(1, 1, torch.bfloat16, d) < f(1, 200, torch.bfloat16, d) < f(1, 200, torch.float16, d) < f(1, 200, torch.float32, d)
    assert f(0, 1, torch.bfloat16, d) == 0 and f(1, 0, torch.bfloat16, d) == 0 and f(1, 1, torch.int8, d) == 0
    assert f(1, 1, torch.bfloat16, g.Dims(4, 3, 128, 128)) == 0
    assert f(1 << 40, 1, torch.bfloat16, d) == 0 and f(1, 1 << 40, torch.bfloat16, d) == 0


def test_binding_refusals(g):
    z = lambda *s, dtype=torch.bfloat16: torch.zeros(*s, dtype=dtype)
    q, v, b = z(4, 2, 128), z(4, 4, 128), z(4, 4, dtype=torch.float32)
    with pytest.raises(ValueError, match="GPU"):
        g.chunk(q, q, v, b, b, v)
    with pytest.raises(TypeError, match="float32, bfloat16"):
        g.decode(q.int(), q, v, b, b, v, None)
    with pytest.raises(ValueError, match="required"):
        g.decode(None, q, v, b, b, v, None)


BACK = ("q", "k", "v", "beta", "gate", "offsets", "state", "d_out", "d_state_out", "dq", "dk", "dv", "dbeta", "dgate",
        "d_state")


def test_backward_refusals(g):
    base = {n: BASE + i * STEP for i, n in enumerate(BACK + ("ws",))}

    def f(hv=4, hk=2, dk_=128, B=3, tokens=100, type=1, bytes=None, **over):
        a = dict(base, **over)
        d = g.Dims(hv, hk, dk_, 128)
        if bytes is None:
            bytes = g.lib.gdn_chunk_backward_workspace_bytes(ctypes.byref(d), B, tokens, type)
        return g.lib.gdn_chunk_backward(ctypes.byref(d), B, tokens, type, *(a[n] for n in BACK), a["ws"], bytes, None)

    for n in BACK:
        if n not in ("offsets", "state", "d_state_out", "d_state"):
            expect(g, f(**{n: None}), -1, n)
    expect(g, f(hv=3), -2, "multiple")
    expect(g, f(dk_=64), -2, "d_k")
    expect(g, f(B=0), -2, "B must")
    expect(g, f(tokens=0), -2, "tokens must")
    expect(g, f(type=5), -2, "type")
    expect(g, f(offsets=None), -2, "multiple of B")
    expect(g, f(hv=1024, hk=1, tokens=1 << 20, bytes=1 << 60), -2, "64")
    for n in ("q", "k", "v", "state", "d_out", "d_state_out", "dq", "dk", "dv", "d_state"):
        expect(g, f(**{n: base[n] + 8}), -3, "aligned")
    for n in ("beta", "gate", "offsets", "dbeta", "dgate"):
        expect(g, f(**{n: base[n] + 2}), -3, "aligned")
    expect(g, f(ws=None), -5, "NULL")
    expect(g, f(bytes=1 << 20), -5, "needed")
    expect(g, f(ws=base["ws"] + 4), -3, "workspace")
    for n in ("dq", "dk", "dv", "dbeta", "dgate", "d_state"):
        for m in BACK:
            if m != n and (n, m) != ("d_state", "d_state_out"):
                expect(g, f(**{n: base[m]}), -4, "overlaps")
        expect(g, f(**{n: base["ws"] + 1024}), -4, "overlaps")
    expect(g, f(d_state=base["d_state_out"] + 16), -4, "d_state")


def test_backward_workspace_bytes(g):
    f = g.chunk_backward_workspace_bytes
    d = g.Dims(4, 2, 128, 128)
    assert 0 < f(1, 1, torch.bfloat16, d) < f(1, 200, torch.bfloat16, d) < f(1, 200, torch.float32, d)
    assert f(0, 1, torch.bfloat16, d) == 0 and f(1, 1, torch.int8, d) == 0
