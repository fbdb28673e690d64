"""GPU: gdn_logprobs where logits are far from 0: masks of a large finite value, and
rows, tokens and offsets of any magnitude, against log_softmax in 64 bits."""
import pytest
import torch

from test_gpu_logprobs import INF, check

pytestmark = pytest.mark.gpu
# Magnitudes on both sides of 2^20 and 2^31, masks in use, and beside the largest.
FAR = [2.0**19, 1048575.0, 2.0**20, 2.0**21, 1e7, 1e9, 2.0**31, 1e10, 1e12, 1e15, 1e20, 1e30, 2.0**100, 1e38]
# fp16 has none of them.
VALUES = {torch.float32: FAR, torch.bfloat16: FAR, torch.float16: [3e4, 65504.0]}


@pytest.fixture(scope="module")
def g():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import gated_deltanet_decode_amd as g
    return g


def rows(v, dtype):
    """For each value: a whole row of it, one with all but three entries masked by it, one
    whose first half is, a single entry of it, and a row around it.  And rows of all."""
    gen = torch.Generator().manual_seed(v)
    rnd = lambda: torch.randn(v, generator=gen) * 2.5
    some = torch.tensor([f * s for f in VALUES[dtype] for s in (1.0, -1.0)])
    xs, tokens = [], []
    for f in some.tolist():
        few, half, one = rnd(), rnd(), rnd()
        keep = torch.randperm(v, generator=gen)[:3]
        few[torch.isin(torch.arange(v), keep, invert=True)] = f
        half[:v // 2] = f
        one[keep[0]] = f
        xs += [torch.full((v,), f), few, half, one, f + rnd()]
        tokens += [v - 1, int(keep[1]), v - 1, int(keep[0]), 5]
    for _ in range(3):
        xs.append(some[torch.randint(0, len(some), (v,), generator=gen)] * (torch.rand(v, generator=gen) < 0.5))
        xs[-1][torch.rand(v, generator=gen) < 0.2] = -INF
        tokens.append(9)
    xs.append(-some.abs()[torch.randint(0, len(some), (v,), generator=gen)])
    tokens.append(0)
    # past the largest: the type's own infinity, which has rows of its own elsewhere
    x = torch.stack(xs).to(dtype)
    return torch.where(torch.isinf(x) & torch.isfinite(torch.stack(xs)), torch.finfo(dtype).max, x).cuda(), \
        torch.tensor(tokens, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("dtype", VALUES, ids=lambda t: str(t)[6:])
@pytest.mark.parametrize("v", [100, 3000, 30000, 120001])
def test_far(g, v, dtype):
    """Threads with an entry at a time, one unit a row, several units a row, and units
    of many vectors a thread (with fewer rows a call, so more units)."""
    x, t = rows(v, dtype)
    check(g, x, t, 20)
    if v == 120001:
        check(g, x[-9:].contiguous(), t[-9:].contiguous(), 3)
