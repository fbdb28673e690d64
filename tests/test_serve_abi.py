"""CPU: the operators around the recurrent branch reject bad arguments with the
documented codes before they touch the GPU (no call here reaches a launch), and
their C-ABI layer runs clean under the sanitizers."""
import ctypes
import os
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
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


def test_norm_and_quantize_validation(g):
    base = slots(("x", "residual", "out", "w", "q", "scale"))

    def f(rows=4, n=64, xt=0, rt=1, eps=1e-6, **over):
        a = dict(base, **over)
        return g.lib.gdn_add_rmsnorm_q8(rows, n, xt, a["x"], rt, a["residual"], a["out"], a["w"], eps,
                                        a["q"], a["scale"], None)

    for n in ("x", "residual", "out", "w", "q", "scale"):
        expect(g, f(**{n: None}), -1, {"w": "norm_w", "out": "residual_out"}.get(n, n))
    expect(g, f(rows=0), -2, "rows")
    expect(g, f(rows=-1), -2, "rows")
    expect(g, f(rows=(1 << 32) // 1024), -2, "rows")
    expect(g, f(n=0), -2, "n must")
    expect(g, f(xt=3), -2, "x_type")
    expect(g, f(xt=-1), -2, "x_type")
    expect(g, f(rt=7), -2, "residual_type")
    expect(g, f(rt=-1), -2, "GDN_NONE")
    expect(g, f(eps=-1e-6), -2, "eps")
    expect(g, f(eps=float("nan")), -2, "eps")
    expect(g, f(eps=float("inf")), -2, "eps")
    for n in ("x", "residual", "out", "q"):
        expect(g, f(**{n: base[n] + 8}), -3, "aligned")
    for n in ("w", "scale"):
        expect(g, f(**{n: base[n] + 2}), -3, "aligned")
    expect(g, f(out=base["residual"] + 16), -4, "residual")      # neither in place nor apart
    expect(g, f(out=base["x"]), -4, "x")
    expect(g, f(q=base["x"] + 4 * 64 * 4 - 16), -4, "x")
    expect(g, f(scale=base["w"]), -4, "norm_w")
    expect(g, f(q=base["out"]), -4, "q")

    def h(rows=4, n=64, xt=0, **over):
        a = dict(base, **over)
        return g.lib.gdn_quantize_q8(rows, n, xt, a["x"], a["q"], a["scale"], None)

    for n in ("x", "q", "scale"):
        expect(g, h(**{n: None}), -1, n)
    expect(g, h(rows=0), -2, "rows")
    expect(g, h(n=-3), -2, "n must")
    expect(g, h(xt=9), -2, "x_type")
    expect(g, h(q=base["x"]), -4, "q")
    expect(g, h(scale=base["q"] + 4), -4, "q")


def test_linear_validation(g):
    base = slots(("a", "sa", "w", "sw", "bias", "o0", "o1", "o2", "o3"))

    def f(M=4, K=64, ot=0, ns=(32, 8), n_outs=None, null_outs=False, **over):
        a = dict(base, **over)
        outs = (g.LinearOut * 4)()
        for i, n in enumerate(ns):
            outs[i].out, outs[i].n = a[f"o{i}"], n
        return g.lib.gdn_linear_q8(M, K, a["a"], a["sa"], a["w"], a["sw"], a["bias"], ot,
                                   None if null_outs else outs, len(ns) if n_outs is None else n_outs,
                                   None)

    for n, name in (("a", "a"), ("w", "w"), ("sa", "a_scale"), ("sw", "w_scale"), ("o0", "outs[0]"),
                    ("o1", "outs[1]")):
        expect(g, f(**{n: None}), -1, name)
    expect(g, f(null_outs=True), -1, "outs")
    expect(g, f(M=0), -2, "M")
    expect(g, f(K=0), -2, "K")
    expect(g, f(K=131072), -2, "K")
    expect(g, f(ot=3), -2, "out_type")
    expect(g, f(n_outs=0), -2, "n_outs")
    expect(g, f(n_outs=5), -2, "n_outs")
    expect(g, f(ns=(32, 0)), -2, "outs[1].n")
    expect(g, f(ns=((1 << 27),)), -2, "too large")
    expect(g, f(ns=(2 ** 31 - 1,) * 4), -2, "too large")
    expect(g, f(M=64 * 4194303 + 1, ns=(1,)), -2, "too large")
    for n in ("a", "w", "o0", "o1"):
        expect(g, f(**{n: base[n] + 8}), -3, "aligned")
    for n in ("sa", "sw", "bias"):
        expect(g, f(**{n: base[n] + 2}), -3, "aligned")
    expect(g, f(o1=base["o0"] + 16), -4, "outs")
    expect(g, f(o0=base["w"]), -4, "w")
    expect(g, f(o0=base["bias"]), -4, "bias")
    expect(g, f(o1=base["a"]), -4, "a")


def test_verify_validation(g):
    base = slots(("target", "draft", "d", "n", "ua", "us", "acc", "tok", "ws"))
    assert g.verify_workspace_bytes(2, 5000) > 0
    for bad in ((0, 5), (-1, 5), (65536, 5), (2, 0), (2, -4)):
        assert g.verify_workspace_bytes(*bad) == 0

    def f(B=2, K=3, V=5000, t=0, ws_bytes=None, **over):
        a = dict(base, **over)
        return g.lib.gdn_verify(B, K, V, t, a["target"], a["draft"], a["d"], a["n"], a["ua"], a["us"],
                                a["acc"], a["tok"], a["ws"],
                                g.verify_workspace_bytes(2, 5000) if ws_bytes is None else ws_bytes, None)

    for n, name in (("target", "target"), ("d", "draft_tokens"), ("ua", "u_accept"),
                    ("us", "u_sample"), ("acc", "accepted"), ("tok", "tokens")):
        expect(g, f(**{n: None}), -1, name)
    for over in (dict(B=0), dict(B=65536), dict(K=0), dict(K=1025), dict(V=0), dict(t=4)):
        expect(g, f(**over), -2, "")
    expect(g, f(ws=None), -5, "workspace")
    expect(g, f(ws_bytes=g.verify_workspace_bytes(2, 5000) - 1), -5, "workspace")
    expect(g, f(ws=base["ws"] + 8), -3, "workspace")
    for n in ("target", "draft"):
        expect(g, f(**{n: base[n] + 8}), -3, "aligned")
    for n in ("d", "n", "ua", "us", "acc", "tok"):
        expect(g, f(**{n: base[n] + 2}), -3, "aligned")
    expect(g, f(acc=base["n"]), -4, "n_draft")
    expect(g, f(tok=base["d"] + 8), -4, "draft_tokens")
    expect(g, f(tok=base["acc"] + 4), -4, "accepted")
    expect(g, f(ws=base["target"] + 16), -4, "target")
    expect(g, f(B=3), -5, "needed")


def test_commit_validation(g):
    base = slots(("acc", "m", "n", "c", "cn"))
    d = g.Dims(32, 16, 128, 128)

    def f(dd=d, layers=2, B=3, ring=8192 * 3, **over):
        a = dict(base, **over)
        return g.lib.gdn_pair_commit(ctypes.byref(dd) if dd is not None else None, layers, B, a["acc"],
                                     a["m"], a["n"], ring, a["c"], a["cn"], None)

    expect(g, f(dd=None), -1, "dims")
    for n, name in (("acc", "accepted"), ("m", "state"), ("n", "state_next"), ("c", "conv_state"),
                    ("cn", "conv_state_next")):
        expect(g, f(**{n: None}), -1, name)
    expect(g, f(dd=g.Dims(32, 16, 64, 128)), -2, "d_k")
    expect(g, f(layers=0), -2, "layers")
    expect(g, f(B=0), -2, "B")
    expect(g, f(layers=1 << 12, B=1 << 12), -2, "too large")
    expect(g, f(layers=2 ** 31 - 1, B=134213631 // 32), -2, "too large")
    expect(g, f(ring=0), -2, "conv_floats")
    expect(g, f(ring=-4), -2, "conv_floats")
    expect(g, f(ring=6), -2, "conv_floats")
    expect(g, f(m=base["m"] + 8), -3, "state")
    expect(g, f(cn=base["cn"] + 4), -3, "conv_state_next")
    expect(g, f(acc=base["acc"] + 2), -3, "accepted")
    expect(g, f(n=base["m"]), -4, "state")
    expect(g, f(cn=base["c"] + 16), -4, "conv_state")
    expect(g, f(m=base["acc"]), -4, "accepted")


def test_binding_rejects_cpu_tensors(g):
    x = torch.zeros(4, 64)
    q, s, w = torch.zeros(4, 64, dtype=torch.int8), torch.zeros(4), torch.zeros(64)
    i = torch.zeros(4, dtype=torch.int32)
    for f in (lambda: g.quantize_q8(x, q, s), lambda: g.add_rmsnorm_q8(x, None, None, w, q, s),
              lambda: g.linear_q8(q, s, q, s, x), lambda: g.pair_commit(i, x[:, :, None, None], x),
              lambda: g.verify(x[None], None, i, s, s, i, i)):
        with pytest.raises(ValueError, match="GPU"):
            f()
    with pytest.raises(TypeError, match="float32, bfloat16 or float16"):
        g.quantize_q8(x.double(), q, s)
    with pytest.raises(TypeError, match="torch tensor"):
        g.quantize_q8([1.0], q, s)


def test_abi_layer_under_asan_ubsan(tmp_path):
    """gdn_serve_api.cpp (with gdn_api.cpp) built for the host under ASan and
    UBSan, its launchers replaced by recording stubs."""
    csrc = os.path.join(ROOT, "gated_deltanet_decode_amd", "csrc")
    cdir = os.path.join(ROOT, "tests", "c")
    cmd = ["g++", "-std=c++17", "-Wall", "-D__HIP_PLATFORM_AMD__", "-I", "/opt/rocm/include", "-O1", "-g",
           "-fno-omit-frame-pointer", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
           "-I", os.path.join(ROOT, "include"), "-I", csrc, "-I", cdir]
    exe = str(tmp_path / "gdn_serve_check")
    subprocess.run(cmd + [os.path.join(csrc, "gdn_api.cpp"), os.path.join(csrc, "gdn_serve_api.cpp"),
                          os.path.join(cdir, "gdn_api_stubs.cpp"),
                          os.path.join(cdir, "gdn_serve_check.cpp"), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout + r.stderr
    assert "serve ABI host check ok" in r.stdout
