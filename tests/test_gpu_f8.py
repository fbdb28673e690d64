"""GPU: e4m3 codes with block scales and their product against the formulas in
64 bits."""
import pytest
import torch

pytestmark = pytest.mark.gpu
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
F8 = torch.float8_e4m3fn
B = 128


@pytest.fixture(scope="module")
def g():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import gated_deltanet_decode_amd as g
    return g


def up(n):
    return (n + B - 1) // B


def spread(scale, tall, rows, n):
    return scale.repeat_interleave(tall, 0)[:rows].repeat_interleave(B, 1)[:, :n]


# ------------------------------------------------------------------- codes
def e4m3(y):
    """The nearest e4m3 values of the binary64 y, |y| <= 448, ties to even: found
    among all of them."""
    values = torch.arange(127, dtype=torch.uint8).view(F8).double()          # ascending, code by code
    a = y.abs()
    hi = torch.searchsorted(values, a.contiguous()).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    below, above = a - values[lo], values[hi] - a
    pick = torch.where((below < above) | ((below == above) & (lo % 2 == 0)), lo, hi)
    return torch.where(values[hi] == a, values[hi], values[pick]) * torch.sign(y)


def want(x, tall):
    x = x.cpu().double()
    rows, n = x.shape
    pad = torch.zeros(up(rows) * B if tall == B else rows, up(n) * B, dtype=torch.float64)
    pad[:rows, :n] = x
    t = pad.view(-1, tall, up(n), B)
    bad = ~torch.isfinite(t).all(3).all(1)
    top = t.abs().amax((1, 3))
    wide = spread(top, tall, rows, n)
    q = torch.where(wide > 0, 448.0 * x / wide, 0.0)
    q = torch.where(spread(bad.double(), tall, rows, n) > 0, 0.0, q)
    scale = (top / 448.0).float()
    scale[bad] = float("nan")
    return e4m3(torch.nan_to_num(q)), scale


def check(g, x, tall):
    rows, n = x.shape
    q = torch.full((rows, n), 1.0, device="cuda").to(F8)
    scale = torch.full((rows if tall == 1 else up(rows), up(n)), 7.0, device="cuda")
    g.quantize_f8(x, q, scale, block_rows=tall)
    wq, ws = want(x, tall)
    assert torch.equal(q.cpu().double(), wq)              # every code, ties included
    s = scale.cpu()
    assert torch.equal(s.isnan(), ws.isnan()) and torch.equal(s.nan_to_num(), ws.nan_to_num())


@pytest.mark.parametrize("dtype", TYPES.values(), ids=TYPES)
@pytest.mark.parametrize("tall", [1, B])
@pytest.mark.parametrize("rows,n", [(1, 1), (3, 127), (2, 128), (5, 129), (130, 300), (129, 1111), (1, 20000), (300, 16), (700, 2048)])
def test_codes(g, rows, n, tall, dtype):
    gen = torch.Generator().manual_seed(rows * n)
    check(g, torch.randn(rows, n, generator=gen).to(dtype).cuda(), tall)


@pytest.mark.parametrize("tall", [1, B])
def test_code_borders(g, tall):
    """Values on and next to the borders between codes, for several largest values."""
    values = torch.arange(127, dtype=torch.uint8).view(F8).double()
    mid = (values[1:] + values[:-1]) / 2
    for top in (448.0, 1.0, 3.0, 0.7, 1e-20, 5e30, 1.1754944e-38, 2.0 ** -130, 3.0e38):
        t = torch.tensor([top], dtype=torch.float32).double()
        x = (torch.cat([mid, values]) * t / 448.0).float()
        x = torch.cat([x, torch.nextafter(x, torch.tensor(float("inf"))), torch.nextafter(x, torch.tensor(0.0)), -x])
        x = x[x.abs() <= float(t)]
        rows = [torch.cat([t.float(), x[i:i + 127]]) for i in range(0, len(x), 127)]
        for r in rows:
            check(g, r[None].cuda(), tall)


@pytest.mark.parametrize("dtype,bits", [(torch.bfloat16, 8), (torch.float16, 11)], ids=["bf16", "f16"])
def test_code_borders_16_bit(g, dtype, bits):
    """Every value of ten binades under a block's largest magnitude, which runs through
    its mantissas (64 of them for float16): each tie and what lies next to one."""
    half = 2 ** (bits - 1)
    mantissas = torch.arange(half, 2 * half, dtype=torch.float64)
    tops = mantissas if bits == 8 else mantissas[torch.randperm(half, generator=torch.Generator().manual_seed(1))[:64]]
    x = torch.cat([mantissas * 2.0**-s for s in range(1, 12)])
    x = torch.cat([x, x.new_zeros(-len(x) % (B - 1))]).view(1, -1, B - 1).repeat(len(tops), 1, 1)
    x[:, :, 1::2] *= -1
    x = torch.cat([tops.view(-1, 1, 1).expand(-1, x.shape[1], 1), x], 2).reshape(len(tops), -1) * 16
    assert torch.equal(x.to(dtype).double(), x)
    check(g, x.to(dtype).cuda(), 1)


@pytest.mark.parametrize("tall", [1, B])
def test_codes_not_finite(g, tall):
    x = torch.randn(260, 400, generator=torch.Generator().manual_seed(1)).cuda()
    x[0, 5], x[1, 200], x[2, 399], x[200, 130] = float("nan"), float("inf"), -float("inf"), float("nan")
    x[10, :128] = 0.0
    x[11, :128] = -0.0
    check(g, x, tall)
    check(g, torch.zeros(3, 200, device="cuda"), tall)
    check(g, torch.full((3, 200), 1e-45, device="cuda"), tall)


# ------------------------------------------------------------------- product
def operands(M, N, K, seed, std=100.0):
    gen = torch.Generator().manual_seed(seed)
    codes = lambda *s: (torch.randn(*s, generator=gen) * std).clamp(-448, 448).to(F8)
    return dict(a=codes(M, K), w=codes(N, K), sa=0.01 + torch.rand(M, up(K), generator=gen),
                sw=0.01 + torch.rand(up(N), up(K), generator=gen), bias=torch.randn(N, generator=gen))


def product(g, d, ns, dtype, bias=True, stream=None):
    M = d["a"].shape[0]
    outs = [torch.full((M, n), 7.0, dtype=dtype, device="cuda") for n in ns]
    c = {k: v.cuda() for k, v in d.items()}
    g.linear_f8(c["a"], c["sa"], c["w"], c["sw"], outs, bias=c["bias"] if bias else None, stream=stream)
    return outs


def off(got, y, tol, dtype):
    """Further off than tol; a value past the type's largest is an infinity."""
    past = y.abs() + tol > torch.finfo(dtype).max
    return ((got - y).abs() > tol) & ~(past & (got == torch.sign(y) * float("inf")))


def check_product(d, outs, dtype, bias=True):
    """float32: per block 128 products summed in float32 (each of at most 7 roundings
    of 2^-24 in a tree, 128 in the worst order), one fused step a block, the scales'
    product and the bias.  16 bits: a block's instruction drops 2^-16 of its
    largest product at most 128 times over four steps of 32, so 2^-13 of the largest
    products, and the result rounds once."""
    M, K = d["a"].shape
    N = d["w"].shape[0]
    a, w = d["a"].double(), d["w"].double()
    y = torch.zeros(M, N, dtype=torch.float64)
    size, most = torch.zeros_like(y), torch.zeros_like(y)
    for b in range(up(K)):
        k = slice(b * B, min(K, b * B + B))
        s = d["sa"][:, b:b + 1].double() * d["sw"][:, b].double().repeat_interleave(B)[:N]
        y += a[:, k] @ w[:, k].T * s
        size += a[:, k].abs() @ w[:, k].abs().T * s
        most += a[:, k].abs().amax(1)[:, None] * w[:, k].abs().amax(1) * s
    if bias:
        y += d["bias"].double()
        size += d["bias"].double().abs()
    u = 2.0 ** -24
    tol = (128 + 2 * up(K) + 4) * u * size + 1e-30
    if dtype != torch.float32:
        tol = tol + 2.0 ** -13 * most + torch.finfo(dtype).eps / 2 * (y.abs() + 2.0 ** -13 * most) + 2.0 ** -24
    got = torch.cat([o.cpu().double() for o in outs], 1)
    bad = off(got, y, tol, dtype)
    assert not bad.any(), (int(bad.sum()), float(((got - y).abs() / tol).max()))
    ok = torch.isfinite(got)
    rel = float((got - y)[ok].norm() / y[ok].norm()) if ok.any() else 0.0
    # random roundings: half a step of the type, or some of 2^-24
    assert rel <= {torch.float32: 1e-6, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}[dtype], rel


@pytest.mark.parametrize("dtype", TYPES.values(), ids=TYPES)
@pytest.mark.parametrize("M,ns,K", [(1, (1,), 1), (1, (130,), 128), (2, (17, 3), 129), (16, (64, 64, 5, 7), 256), (33, (100,), 4000),
                                    (5, (1000,), 112), (77, (1003,), 1111), (130, (300, 84), 2064), (300, (520,), 384),
                                    (129, (4100,), 272), (1, (12352,), 2048), (64, (2048,), 4096), (700, (1500,), 640)])
def test_product(g, M, ns, K, dtype):
    d = operands(M, sum(ns), K, M + K)
    check_product(d, product(g, d, ns, dtype), dtype)


@pytest.mark.parametrize("dtype", TYPES.values(), ids=TYPES)
@pytest.mark.parametrize("M,N,K", [(2500, 2300, 512), (4100, 4100, 144), (2048, 4096, 1024), (3000, 2000, 777)])
def test_large_product(g, M, N, K, dtype):
    """All tile shapes, whole and ragged; every element against a product in 64 bits
    on the GPU."""
    d = operands(M, N, K, 5)
    outs = product(g, d, (N,), dtype, bias=False)
    c = {k: v.cuda() for k, v in d.items()}
    y = (c["a"].double() * spread(c["sa"].double(), 1, M, K)) @ (c["w"].double() * spread(c["sw"].double(), B, N, K)).t().contiguous()
    size = (c["a"].double().abs() * spread(c["sa"].double(), 1, M, K)) @ (c["w"].double().abs() * spread(c["sw"].double(), B, N, K)).t().contiguous()
    tol = (128 + 2 * up(K) + 4) * 2.0 ** -24 * size
    if dtype != torch.float32:
        tol = tol + 2.0 ** -13 * size + torch.finfo(dtype).eps / 2 * y.abs() * (1 + 2.0 ** -10) + 2.0 ** -24
    assert not off(outs[0].double(), y, tol, dtype).any()


def test_stray_codes(g):
    """What lies behind a row's last k, in the next row, is not multiplied: NaN
    codes there change nothing."""
    for K, dtype in ((144, torch.bfloat16), (100, torch.float32), (16, torch.float16)):
        d = operands(40, 70, K, 9)
        nan = torch.full((1,), 0x7f, dtype=torch.uint8).view(F8)
        ref = product(g, d, (70,), dtype)
        d["a"][20], d["w"][30] = nan, nan
        got = product(g, d, (70,), dtype)
        keep_m, keep_n = torch.arange(40) != 20, torch.arange(70) != 30
        assert torch.equal(got[0].cpu()[keep_m][:, keep_n], ref[0].cpu()[keep_m][:, keep_n])
        assert got[0][20].isnan().all() and got[0][:, 30].isnan().all()


def test_layer_chain(g):
    """Weights and activations quantised here, multiplied, the result's rows
    quantised again; repeated from a graph and on another stream."""
    gen = torch.Generator().manual_seed(3)
    x = torch.randn(50, 300, generator=gen).cuda().bfloat16()
    w = (torch.randn(400, 300, generator=gen) * 0.05).cuda()
    e = lambda *s, t=torch.float32: torch.empty(*s, device="cuda", dtype=t)
    wq, ws = e(400, 300, t=F8), e(4, 3)
    g.quantize_f8(w, wq, ws, block_rows=128)
    xq, xs, z, y, yq, ys = e(50, 300, t=F8), e(50, 3), e(50, 144), e(50, 256), e(50, 256, t=F8), e(50, 2)

    def chain():
        g.quantize_f8(x, xq, xs)
        g.linear_f8(xq, xs, wq, ws, [y, z])
        g.quantize_f8(y, yq, ys)
    chain()
    want_ = (xq.double() * spread(xs.double(), 1, 50, 300)) @ (wq.double() * spread(ws.double(), B, 400, 300)).t().contiguous()
    assert float((torch.cat([y, z], 1).double() - want_).norm() / want_.norm()) <= 1e-6
    full = x.double() @ w.double().t().contiguous()
    # two roundings of at most 2^-4 a value, independent over 300 products
    assert float((want_ - full).norm() / full.norm()) <= 2.0 ** -4
    wy, ws_ = want(y, 1)
    assert torch.equal(yq.cpu().double(), wy) and torch.equal(ys.cpu(), ws_)
    keep = [t.clone() for t in (xq.view(torch.uint8), xs, y, z, yq.view(torch.uint8), ys)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        chain()
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        chain()
    for _ in range(3):
        for t in (xs, y, z, ys):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        now = (xq.view(torch.uint8), xs, y, z, yq.view(torch.uint8), ys)
        assert all(torch.equal(a, b) for a, b in zip(now, keep))
