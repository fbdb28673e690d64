"""GPU: gdn_add_rmsnorm_q8 and gdn_quantize_q8 against the formulas in 64 bits.
The codes have to be the formula's exactly: they are functions of products that
binary64 holds exactly, and the library divides out every quotient that comes
near a border.  The scale is one rounding to binary32 of a binary64 value whose
own error is that of the sum of squares: at most four roundings of 2^-24 while
eight squares are added in pairs (squaring, three additions), binary64 above
that; the square root halves them."""
import itertools

import numpy as np
import pytest
import torch

import serve_ref as sr

pytestmark = pytest.mark.gpu

GUARD = 64


@pytest.fixture(scope="module")
def g():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import gated_deltanet_decode_amd as g
    return g


def guarded(shape, dtype, fill=77):
    """A GPU tensor inside a larger one whose borders must stay as they are."""
    n = int(np.prod(shape))
    whole = torch.full((n + 2 * GUARD,), fill, dtype=dtype, device="cuda")
    return whole[GUARD:GUARD + n].view(shape), whole


def untouched(whole, fill=77):
    return bool((whole[:GUARD] == fill).all()) and bool((whole[-GUARD:] == fill).all())


def check_scale(got, want, norm):
    got = got.cpu().double().numpy()
    nan = np.isnan(want)
    assert np.array_equal(np.isnan(got), nan)
    got, want = got[~nan], want[~nan]
    # half a binary32 step (2^-150 below the normal range), and half of the sum's
    # four where there is one
    lim = np.maximum(want * 2.0 ** -24 * (1 + (2 if norm else 0)) * (1 + 1e-4), 2.0 ** -150)
    assert np.all(np.abs(got - want) <= lim), np.max(np.abs(got - want) / np.maximum(want, 1e-300))


def make(rows, n, dtype, seed, std=1.0):
    gen = torch.Generator().manual_seed(seed)
    return (torch.randn(rows, n, generator=gen) * std).to(dtype)


def run_norm(g, x, res, w, eps=1e-6, in_place=False):
    rows, n = x.shape
    q, qw = guarded((rows, n), torch.int8)
    s, sw = guarded((rows,), torch.float32)
    rd = None if res is None else res.cuda()
    out, ow = (None, None)
    if res is not None:
        if in_place:
            out = rd
        else:
            out, ow = guarded((rows, n), res.dtype)
    g.add_rmsnorm_q8(x.cuda(), rd, out, w.cuda(), q, s, eps=eps)
    torch.cuda.synchronize()
    assert untouched(qw) and untouched(sw) and (ow is None or untouched(ow))
    if res is not None and not in_place:
        assert torch.equal(rd.cpu().view(torch.uint8), res.view(torch.uint8)), "the residual input was written"
    return q, s, out


def check_norm(g, x, res, w, eps=1e-6, in_place=False):
    q, s, out = run_norm(g, x, res, w, eps, in_place)
    h = sr.stored_sum(x, res)
    if res is not None:
        a, b = out.cpu(), h
        same = (a == b) | (a.isnan() & b.isnan())
        assert bool(same.all()), "stored residual"
    wq, ws = sr.rmsnorm_q8(h, w, eps)
    assert np.array_equal(q.cpu().numpy(), wq), "codes"
    check_scale(s, ws, True)


def check_quant(g, x):
    rows, n = x.shape
    q, qw = guarded((rows, n), torch.int8)
    s, sw = guarded((rows,), torch.float32)
    g.quantize_q8(x.cuda(), q, s)
    torch.cuda.synchronize()
    assert untouched(qw) and untouched(sw)
    wq, ws = sr.quantize_q8(x)
    assert np.array_equal(q.cpu().numpy(), wq), "codes"
    check_scale(s, ws, False)


WIDTHS = [1, 2, 7, 8, 63, 64, 65, 255, 256, 257, 511, 513, 1000, 1024, 1025, 2048, 2049, 4096, 4097,
          6001, 6144, 8191, 8192, 8200, 12288, 16384, 16390, 20001, 32768, 32769, 40000]


@pytest.mark.parametrize("n", WIDTHS)
def test_norm_widths(g, n):
    print(f"\n  add_rmsnorm_q8 n={n}", flush=True)
    rows = 5
    w = 1.0 + 0.02 * make(1, n, torch.float32, n + 1)[0]
    check_norm(g, make(rows, n, torch.float32, n), make(rows, n, torch.float32, n + 2, 3.0), w)
    check_norm(g, make(rows, n, torch.bfloat16, n), make(rows, n, torch.bfloat16, n + 2, 3.0), w)


@pytest.mark.parametrize("xt,rt", itertools.product(sr.TYPES, [*sr.TYPES, None]))
@pytest.mark.parametrize("rows,n", [(1, 2048), (33, 513), (300, 2048), (3, 9000)])
def test_norm_types(g, xt, rt, rows, n):
    print(f"\n  add_rmsnorm_q8 x={xt} residual={rt} rows={rows} n={n}", flush=True)
    x = make(rows, n, sr.TYPES[xt], 11)
    res = None if rt is None else make(rows, n, sr.TYPES[rt], 12, 3.0)
    w = 1.0 + 0.02 * make(1, n, torch.float32, 13)[0]
    check_norm(g, x, res, w)
    if res is not None:
        check_norm(g, x, res, w, in_place=True)


@pytest.mark.parametrize("t", list(sr.TYPES))
@pytest.mark.parametrize("rows,n", [(1, 1), (2, 7), (32, 4096), (300, 4097), (5, 20001), (2000, 130)])
def test_quantize(g, t, rows, n):
    print(f"\n  quantize_q8 {t} rows={rows} n={n}", flush=True)
    check_quant(g, make(rows, n, sr.TYPES[t], 21))


@pytest.mark.parametrize("xt,rt", [("f32", "f32"), ("bf16", "bf16"), ("f16", "f32"), ("f32", "bf16"), ("f16", None)])
@pytest.mark.parametrize("n", [1, 3, 17, 100, 128, 129, 135, 136, 200, 256, 263, 264])
def test_narrow_rows(g, xt, rt, n):
    """Several rows to a wave: ordinary rows beside rows of zeros, of NaN and of
    magnitudes that take the other path, and a number of rows that ends anywhere."""
    print(f"\n  narrow rows n={n} x={xt} residual={rt}", flush=True)
    w = 1.0 + 0.02 * make(1, n, torch.float32, 73)[0]
    for rows in (1, 15, 16, 17, 1003):
        x = make(rows, n, sr.TYPES[xt], 71)
        res = None if rt is None else make(rows, n, sr.TYPES[rt], 72, 3.0)
        for t in (x,) if res is None else (x, res):
            t[3::7] *= 1e-30 if t.dtype != torch.float16 else 1e-6
            t[5::11] = 0.0
            t[6::13, 0] = float("nan")
        check_norm(g, x, res, w)
        check_quant(g, x)


@pytest.mark.parametrize("t", list(sr.TYPES))
@pytest.mark.parametrize("n", [4100, 8192, 8199, 8200, 8201, 12345, 16384, 16391, 16392])
def test_quantize_long_rows(g, t, n):
    print(f"\n  quantize_q8 {t} n={n}", flush=True)
    x = make(9, n, sr.TYPES[t], 22)
    x[4] *= 1e-30 if t != "f16" else 1e-6
    x[6, n - 1] = float("inf")
    check_quant(g, x)


@pytest.mark.parametrize("n", [16, 100, 2048, 4099, 20000])
def test_ties_go_to_even(g, n):
    """127 g / 254 = g / 2 is a tie for every odd g."""
    print(f"\n  ties n={n}", flush=True)
    x = torch.randint(-253, 254, (7, n), generator=torch.Generator().manual_seed(n)).float()
    x[:, 0] = 254.0
    check_quant(g, x)
    check_norm(g, x, None, torch.ones(n))
    # next to a tie: one binary32 step to either side
    y = torch.where(torch.rand(7, n, generator=torch.Generator().manual_seed(1)) < 0.5,
                    torch.nextafter(x, torch.tensor(1e9)), torch.nextafter(x, torch.tensor(-1e9)))
    y[:, 0] = 254.0
    check_quant(g, y)


@pytest.mark.parametrize("n", [5, 64, 1000, 2048, 9001, 20001])
def test_extreme_rows(g, n):
    """Zero rows, rows with NaN and infinities, the largest and smallest
    magnitudes, one entry that is not zero."""
    print(f"\n  extreme rows n={n}", flush=True)
    x = make(12, n, torch.float32, 31)
    x[0] = 0.0
    x[1, n // 2] = float("nan")
    x[2, 0] = float("inf")
    x[3, n - 1] = float("-inf")
    x[4] = x[4].sign() * 3.4028234e38
    x[5] *= 1e-38
    x[6] *= 1e-44
    x[7] = 0.0
    x[7, n - 1] = -1e-45
    x[8] = -0.0
    x[9, 0], x[9, n - 1] = float("nan"), float("inf")
    x[10] = 1.0
    w = 1.0 + 0.02 * make(1, n, torch.float32, 33)[0]
    check_quant(g, x)
    check_norm(g, x, None, w)
    check_norm(g, x, None, w, eps=0.0)
    check_norm(g, x, make(12, n, torch.bfloat16, 32), w)
    wz = w.clone()
    wz[: n // 2 + 1] = 0.0          # a weight of zero beside an infinite entry: 0 * inf is NaN
    check_norm(g, x, None, wz)
    wz[n - 1] = float("inf")
    check_norm(g, x, None, wz)


@pytest.mark.parametrize("n", [3, 200, 1024, 2048, 5000, 20000])
def test_rows_of_every_magnitude(g, n):
    """Rows scaled by every power of two that binary32 holds, with weights of
    ordinary size and of 2^40 and 2^-40: products, squares and sums that pass
    through both ends of the range."""
    print(f"\n  every magnitude n={n}", flush=True)
    e = torch.arange(-149, 126, 5 if n < 5000 else 13)
    x = make(len(e), n, torch.float32, 61).clamp_(-1.9, 1.9) * torch.exp2(e.double()).float()[:, None]
    w = 1.0 + 0.02 * make(1, n, torch.float32, 62)[0]
    check_quant(g, x)
    for s in (1.0, 2.0 ** 40, 2.0 ** -40, 2.0 ** -120):
        check_norm(g, x, None, w * s)
        check_norm(g, x, None, w * s, eps=0.0)
    check_norm(g, x, make(len(e), n, torch.float16, 63) * 1e-3, w)


def test_products_that_round_alike(g):
    """Largest products that differ only beyond binary32: the scale and the codes
    follow the exact one."""
    print("\n  products that round alike", flush=True)
    n = 4096
    gen = torch.Generator().manual_seed(64)
    for k in range(6):
        # h w = (1 + a 2^-12)(1 + b 2^-12) with a + b fixed: equal to 2^-24 or so
        a = torch.randint(0, 2048, (16, n), generator=gen)
        h = 1.0 + a.float() * 2.0 ** -12
        x = h * torch.where(torch.rand(16, n, generator=gen) < 0.5, -1.0, 1.0)
        w = 1.0 + (2048 - a[0]).float() * 2.0 ** -12
        x[1:, ::2] *= 0.5
        x[0] = h[0]
        check_norm(g, x, None, w)
        x = torch.full((5, n), 1.0 + k * 2.0 ** -20)        # every element is the largest
        check_quant(g, x)
        check_norm(g, x, None, torch.ones(n))


def test_rows_do_not_depend_on_the_batch(g):
    print("\n  batch independence", flush=True)
    for n in (100, 200, 700, 2048, 4096, 5000, 9000, 20000):
        x, w = make(700, n, torch.float32, 41), torch.ones(n)
        r = make(700, n, torch.float32, 42)
        q, s, _ = run_norm(g, x, r, w)
        for rows in (1, 3, 64):
            q1, s1, _ = run_norm(g, x[:rows].contiguous(), r[:rows].contiguous(), w)
            assert torch.equal(q[:rows], q1) and torch.equal(s[:rows], s1)


def test_large_row_offsets(g):
    """Rows past 2^31 elements: the last rows of a tensor of 2.2e9 bytes of
    codes, against the same rows alone."""
    print("\n  offsets past 2^31", flush=True)
    n, rows = 65536, 33000
    x = torch.zeros(rows, n, dtype=torch.bfloat16, device="cuda")
    tail = make(4, n, torch.bfloat16, 51).cuda()
    x[-4:] = tail
    q = torch.empty(rows, n, dtype=torch.int8, device="cuda")
    s = torch.empty(rows, device="cuda")
    g.quantize_q8(x, q, s)
    q1, s1 = torch.empty(4, n, dtype=torch.int8, device="cuda"), torch.empty(4, device="cuda")
    g.quantize_q8(tail, q1, s1)
    torch.cuda.synchronize()
    assert torch.equal(q[-4:], q1) and torch.equal(s[-4:], s1)
    assert not bool(q[:-4].any()) and not bool(s[:-4].any())


def test_refusals_on_the_gpu(g):
    x = torch.zeros(4, 64, device="cuda")
    q = torch.full((4, 64), 5, dtype=torch.int8, device="cuda")
    s = torch.full((4,), 6.0, device="cuda")
    w = torch.ones(64, device="cuda")
    for bad in (lambda: g.quantize_q8(x.double(), q, s),
                lambda: g.quantize_q8(x.t(), q.t(), s),
                lambda: g.quantize_q8(x[:, ::2], q[:, :32], s),
                lambda: g.quantize_q8(x, q.float(), s),
                lambda: g.quantize_q8(x, q[:3], s),
                lambda: g.quantize_q8(x[0], q, s),
                lambda: g.quantize_q8(x[:0], q[:0], s[:0]),
                lambda: g.quantize_q8(None, q, s),
                lambda: g.quantize_q8(x.cpu(), q, s),
                lambda: g.quantize_q8(x, q.cpu(), s),
                lambda: g.add_rmsnorm_q8(x, None, x, w, q, s),
                lambda: g.add_rmsnorm_q8(x, x, None, w, q, s),
                lambda: g.add_rmsnorm_q8(x, x, x, w, q, s),
                lambda: g.add_rmsnorm_q8(x, s, s, w, q, s),
                lambda: g.add_rmsnorm_q8(x, None, None, w, q, s, eps=-1.0),
                lambda: g.add_rmsnorm_q8(x, None, None, w, q, s, eps=float("nan"))):
        with pytest.raises((g.GdnError, TypeError, ValueError)):
            bad()
    torch.cuda.synchronize()
    assert bool((q == 5).all()) and bool((s == 6.0).all()) and bool((x == 0).all())
