"""GPU: the codes of gdn_add_rmsnorm_q8 where 127 g / G lies on or next to a
border and g is a product of two full binary32 numbers: 127 g then takes up to 55
bits, and a quotient rounded to binary64 falls on the wrong side.  The reference
compares whole numbers."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

# (a, b, c, d, k): 254 a b is 1 to 4 off (2 k + 1) c d
NEAR = [(11732069, 15600007, 13229291, 14580738, 120), (12060317, 15426295, 13610231, 16300802, 106),
        (9045447, 11524151, 10753856, 15884618, 77), (10044827, 11624117, 10572843, 15497648, 90),
        (9041273, 10586379, 11132623, 16419563, 66), (10660427, 11892239, 12020585, 13196243, 101),
        (8750241, 16769331, 8977544, 16409351, 126), (16301799, 9726087, 15042632, 16424644, 81),
        (10801205, 11619521, 11563526, 15401068, 89), (8717173, 10650437, 11672918, 16424504, 61),
        (10799955, 16079451, 12970444, 14228992, 119), (11487659, 9875683, 13155520, 16720647, 65),
        (9179037, 14466555, 14748257, 16219451, 70),
        (8158185, 8875831, 7674737, 17751662, 67)]          # a tie


def code(g, top):
    """rint(127 g / top) of whole numbers, ties to even."""
    q, r = divmod(127 * abs(g), top)
    q += 2 * r > top or (2 * r == top and q & 1)
    return q if g >= 0 else -q


def check(g, x, w, e):
    """Whole numbers x [rows][n] and w [n], scaled by 2^e each (nothing rounds)."""
    rows, n = len(x), len(w)
    xt = torch.tensor(x, dtype=torch.float64).float() * 2.0 ** e
    wt = torch.tensor(w, dtype=torch.float64).float() * 2.0 ** e
    assert (xt.double() * 2.0 ** -e).tolist() == x and (wt.double() * 2.0 ** -e).tolist() == w
    q = torch.empty(rows, n, dtype=torch.int8, device="cuda")
    scale = torch.empty(rows, device="cuda")
    g.add_rmsnorm_q8(xt.cuda(), None, None, wt.cuda(), q, scale)
    torch.cuda.synchronize()
    for i, row in enumerate(x):
        p = [u * v for u, v in zip(row, w)]
        top = max(map(abs, p))
        want = [code(v, top) for v in p]
        got = q[i].tolist()
        assert got == want, [(j, p[j], top, got[j], want[j]) for j in range(n) if got[j] != want[j]][:4]


@pytest.fixture(scope="module")
def g():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import gated_deltanet_decode_amd as g
    return g


# one row of every kernel (16 lanes, a wave, 256 to 1024 threads, the long rows), and
# magnitudes that take the binary32 and the binary64 path
SIZES = [(4, -24), (200, -24), (700, -24), (2048, -24), (5000, -24), (9001, -24), (20000, -24), (300, -70), (300, 40)]


@pytest.mark.parametrize("n,e", SIZES)
def test_next_to_a_border(g, n, e):
    print(f"\n  codes next to a border, n={n} 2^{e}", flush=True)
    for a, b, c, d, k in NEAR:
        x, w = [1] * n, [1] * n
        x[0], w[0], x[n // 2], w[n // 2], x[n - 1], w[n - 1] = a, b, -c, d, -a, b
        assert math.floor(127 * a * b / (c * d)) == k
        check(g, [x, [-v for v in x]], w, e)


@pytest.mark.parametrize("n,e", SIZES)
def test_ties_of_full_products(g, n, e):
    """a = (2 k + 1) s and c = 127 s: 127 a b = (k + 1/2) c (2 b) for every b."""
    print(f"\n  ties of full products, n={n} 2^{e}", flush=True)
    gen = torch.Generator().manual_seed(n)
    rows, w = [], [int(v) for v in torch.randint(1 << 22, 1 << 23, (n,), generator=gen)]
    w[n - 1] = 2 * max(w[:n - 1])
    for r in range(4 if n <= 2048 else 2):
        s = int(torch.randint(32768, 65793, (1,), generator=gen))
        at = torch.randint(0, 127, (n,), generator=gen).tolist()
        sign = (2 * torch.randint(0, 2, (n,), generator=gen) - 1).tolist()
        row = [(2 * k + 1) * s * f for k, f in zip(at, sign)]
        row[n - 1] = 127 * s
        rows.append(row)
    # the largest weight's entries are ties; the others lie anywhere
    b = w[n - 1] // 2
    w = [b if j % 3 else v for j, v in enumerate(w[:n - 1])] + [2 * b]
    check(g, rows, w, e)
