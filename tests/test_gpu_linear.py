"""GPU: gdn_linear_q8 against the product in 64 bits (tests/serve_ref.py derives
the bound of the scaling; the integer sum is exact)."""
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


def make(M, N, K, seed, full=False):
    gen = torch.Generator().manual_seed(seed)
    lo = -128 if full else -127
    a = torch.randint(lo, 128, (M, K), generator=gen, dtype=torch.int8)
    w = torch.randint(lo, 128, (N, K), generator=gen, dtype=torch.int8)
    return (a, 0.01 + torch.rand(M, generator=gen), w, 0.001 + 0.01 * torch.rand(N, generator=gen),
            torch.randn(N, generator=gen) * 10)


def run(g, a, sa, w, sw, bias, splits, dtype):
    M = a.shape[0]
    wholes = [torch.full((M * n + 2 * GUARD,), 77.0, dtype=dtype, device="cuda") for n in splits]
    outs = [t[GUARD:GUARD + M * n].view(M, n) for t, n in zip(wholes, splits)]
    g.linear_q8(a.cuda(), sa.cuda(), w.cuda(), sw.cuda(), outs if len(outs) > 1 else outs[0],
                bias=None if bias is None else bias.cuda())
    torch.cuda.synchronize()
    for t in wholes:
        assert bool((t[:GUARD] == 77).all()) and bool((t[-GUARD:] == 77).all()), "written outside"
    return torch.cat(outs, 1)


def check(g, M, splits, K, dtype, bias, seed=0, full=False):
    print(f"\n  linear_q8 M={M} N={splits} K={K} {dtype} bias={bias}", flush=True)
    a, sa, w, sw, b = make(M, sum(splits), K, seed + M + K, full)
    b = b if bias else None
    got = sr.f64(run(g, a, sa, w, sw, b, splits, dtype))
    want, tol = sr.linear_q8(a, sa, w, sw, b, dtype)
    err = np.abs(got - want)
    i = int(np.argmax(err - tol))
    assert np.all(err <= tol), f"at {divmod(i, want.shape[1])}: {got.flat[i]} for {want.flat[i]}"


@pytest.mark.parametrize("M", [1, 2, 3, 8, 15, 16, 17, 31, 32, 33, 48, 64, 65, 77, 128, 129, 200, 256,
                               257, 500])
@pytest.mark.parametrize("N,K", [(64, 64), (256, 512), (1003, 1111), (130, 2048)])
def test_sizes(g, M, N, K):
    check(g, M, [N], K, torch.float32, False)


@pytest.mark.parametrize("K", [1, 2, 15, 16, 17, 31, 63, 64, 65, 127, 128, 129, 191, 192, 255, 256, 257,
                               1000, 1024, 1040, 4096, 8208])
@pytest.mark.parametrize("M", [1, 40, 300])
def test_inner_lengths(g, M, K):
    check(g, M, [80], K, torch.float32, False)


@pytest.mark.parametrize("N", [1, 2, 3, 4, 5, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 257, 513])
@pytest.mark.parametrize("M", [1, 20, 270])
def test_channel_counts(g, M, N):
    check(g, M, [N], 160, torch.float32, True)


# Shapes that reach each kernel and tile on a GPU of 256 compute units, with
# tokens and channels that end inside a tile and groups that end inside one.
VARIANTS = [(13, [12289, 31]), (30, [6100, 57, 43]), (30, [12300, 50]), (200, [1999, 51]),
            (500, [1025, 1025]), (1000, [2050]), (1990, [1000, 40, 1010]), (4100, [2000, 1000, 1999, 1])]


@pytest.mark.parametrize("K", [1, 16, 100, 112, 128, 130, 144, 256, 272, 384, 400, 527, 640, 1040])
@pytest.mark.parametrize("M,splits", VARIANTS)
def test_every_kernel_over_inner_lengths(g, M, splits, K):
    check(g, M, splits, K, torch.float32, K % 3 == 0)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("K", [527, 1280])
@pytest.mark.parametrize("M,splits", VARIANTS)
def test_every_kernel_over_types(g, M, splits, K, dtype):
    check(g, M, splits, K, dtype, True, full=True)


# One round of 128 x 128 tiles, one and several rounds of 256 x 128, rounds of
# 256 x 256, and tile counts that do not divide among the XCDs.
ROUNDS = [(1500, [1025, 1025]), (1290, [2000, 500, 13]), (640, [8192, 4096, 64]), (4100, [5000]),
          (300, [12352]), (130, [8300])]


@pytest.mark.parametrize("K", [16, 128, 240, 256, 384, 512, 656, 2064])
@pytest.mark.parametrize("M,splits", ROUNDS)
def test_rounds_of_tiles(g, M, splits, K):
    check(g, M, splits, K, torch.float32 if K % 256 else torch.bfloat16, K < 300)


# Just enough tiles for each kernel, from 16 x 16 to one round and more of 256 x
# 256, with k of no, one and several blocks, whole and not.
@pytest.mark.parametrize("dtype", [torch.float32, torch.float16])
@pytest.mark.parametrize("K", [48, 256, 400, 512, 768, 1040, 1280])
@pytest.mark.parametrize("M,splits", [(13, [2000]), (13, [8300]), (30, [4100, 55]), (30, [8300]), (200, [1203]),
                                      (190, [3000]), (500, [2000, 100]), (1200, [1801]), (4100, [2500, 2477])])
def test_smallest_of_each_kernel(g, dtype, M, splits, K):
    check(g, M, splits, K, dtype, K % 512 == 0)


# k that is no multiple of 16: the bytes past a row's end belong to the next row,
# or lie past the matrix behind the last one.
@pytest.mark.parametrize("K", [1, 3, 7, 13, 18, 31, 47, 111, 127, 129, 143, 250, 391])
@pytest.mark.parametrize("M,splits", [(1, [1]), (2, [3]), (17, [100]), (320, [2048]), (700, [82, 429, 26]),
                                      (1500, [1000]), (5953, [144])])
def test_rows_that_end_anywhere(g, M, splits, K):
    check(g, M, splits, K, torch.float32, K % 2 == 1, full=True)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("M,splits,K", [(5953, [144], 64), (10729, [80], 64), (3000, [1000, 1999, 1], 192),
                                        (1500, [2050], 240), (320, [2048], 400), (640, [2047], 272)])
def test_short_inner_lengths(g, dtype, M, splits, K):
    check(g, M, splits, K, dtype, True)


@pytest.mark.parametrize("M,N,K", [(40000, 5, 200), (3, 40000, 33), (9000, 17, 64), (5000, 5000, 48)])
def test_narrow_and_wide(g, M, N, K):
    check(g, M, [N], K, torch.float32, False)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("M,splits,K", [(1, [8192, 4096, 64], 2048), (5, [33, 1, 7, 100], 100),
                                        (64, [256, 128, 64], 256), (100, [130, 62], 384),
                                        (300, [256, 3, 253], 512), (513, [512, 256, 64], 320)])
def test_types_and_groups(g, dtype, bias, M, splits, K):
    check(g, M, splits, K, dtype, bias)


@pytest.mark.parametrize("M,N,K", [(4, 48, 131071), (40, 48, 131056), (260, 300, 131071)])
def test_largest_sums(g, M, N, K):
    """Every product 2^14: the integer sum reaches 2^31 - 2^14 and must not wrap."""
    print(f"\n  linear_q8 M={M} N={N} K={K} largest sums", flush=True)
    a = torch.full((M, K), -128, dtype=torch.int8)
    w = torch.full((N, K), -128, dtype=torch.int8)
    one_m, one_n = torch.ones(M), torch.ones(N)
    got = run(g, a, one_m, w, one_n, None, [N], torch.float32)
    assert bool((got.double() == float(np.float32(K * 16384))).all())


@pytest.mark.parametrize("M,N,K", [(1, 2048, 4096), (256, 2048, 4096), (2048, 8192, 2048),
                                   (1500, 1111, 777)])
def test_larger(g, M, N, K):
    check(g, M, [N], K, torch.float32, False, full=True)


def test_scales_that_are_not_finite_stay_in_their_row_and_channel(g):
    print("\n  NaN and infinite scales", flush=True)
    for M in (3, 70, 300):
        a, sa, w, sw, _ = make(M, 90, 128, 5)
        sa[1], sw[7], sw[89] = float("nan"), float("inf"), 0.0
        got = run(g, a, sa, w, sw, None, [90], torch.float32)
        keep_m = torch.arange(M, device="cuda") != 1
        keep_n = torch.ones(90, dtype=torch.bool, device="cuda")
        keep_n[7] = False
        assert bool(got[1].isnan().all())
        assert bool(got[keep_m][:, keep_n].isfinite().all())
        assert bool((got[keep_m][:, 89] == 0).all())


def test_rows_do_not_depend_on_the_batch(g):
    print("\n  batch independence", flush=True)
    a, sa, w, sw, b = make(600, 200, 1000, 9)
    full = run(g, a, sa, w, sw, b, [200], torch.bfloat16)
    for M in (1, 2, 16, 17, 40, 64, 100, 257):
        part = run(g, a[:M], sa[:M], w, sw, b, [200], torch.bfloat16)
        assert torch.equal(full[:M], part), M


def test_offsets_past_31_bits(g):
    """Weights and outputs beyond 2^31 elements: the last channels and tokens."""
    print("\n  offsets past 2^31", flush=True)
    K, N = 16384, 140000                     # 2.3e9 bytes of weights
    w = torch.zeros(N, K, dtype=torch.int8, device="cuda")
    w[-3:] = 1
    a = torch.ones(2, K, dtype=torch.int8, device="cuda")
    out = torch.empty(2, N, device="cuda")
    g.linear_q8(a, torch.ones(2, device="cuda"), w, torch.ones(N, device="cuda"), out)
    torch.cuda.synchronize()
    assert bool((out[:, -3:] == K).all()) and not bool(out[:, :-3].any())
    del w, a, out
    M, N, K = 70000, 32768, 64               # 2.3e9 outputs
    a = torch.zeros(M, K, dtype=torch.int8, device="cuda")
    a[-2:] = 1
    w = torch.ones(N, K, dtype=torch.int8, device="cuda")
    out = torch.full((M, N), 9.0, dtype=torch.bfloat16, device="cuda")
    g.linear_q8(a, torch.ones(M, device="cuda"), w, torch.ones(N, device="cuda"), out)
    torch.cuda.synchronize()
    assert bool((out[-2:] == K).all())
    for r in range(0, M - 2, 10000):
        assert not bool(out[r:min(r + 10000, M - 2)].any())


def test_refusals_on_the_gpu(g):
    a = torch.zeros(4, 64, dtype=torch.int8, device="cuda")
    w = torch.zeros(32, 64, dtype=torch.int8, device="cuda")
    sa, sw = torch.ones(4, device="cuda"), torch.ones(32, device="cuda")
    out = torch.full((4, 32), 3.0, device="cuda")
    for bad in (lambda: g.linear_q8(a.float(), sa, w, sw, out),
                lambda: g.linear_q8(a, sa, w.t(), sw, out),
                lambda: g.linear_q8(a, sa, w[:, :32], sw, out),
                lambda: g.linear_q8(a, sa[:3], w, sw, out),
                lambda: g.linear_q8(a, sa, w, sw, out.double()),
                lambda: g.linear_q8(a, sa, w, sw, out[:, :31]),
                lambda: g.linear_q8(a, sa, w, sw, []),
                lambda: g.linear_q8(a, sa, w, sw, [out[:, :16].contiguous(),
                                                   out[:, 16:].contiguous().half()]),
                lambda: g.linear_q8(a, sa, w, sw, [torch.empty(4, 32, device="cuda")] * 5),
                lambda: g.linear_q8(a, sa, w, sw, [out.view(8, 16)[:4], out.view(8, 16)[:4]]),
                lambda: g.linear_q8(a, sa, w, sw, out, bias=sw.half()),
                lambda: g.linear_q8(a, sa, w.cpu(), sw, out),
                lambda: g.linear_q8(a[:0], sa[:0], w, sw, out[:0])):
        with pytest.raises((g.GdnError, TypeError, ValueError)):
            bad()
    torch.cuda.synchronize()
    assert bool((out == 3.0).all())
