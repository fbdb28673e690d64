"""GPU: gdn_chunk and gdn_chunk_backward with more heads than half the compute units,
where a workgroup has a whole head (eight waves); the other files' batches are
smaller, and have two workgroups a head."""
import pytest
import torch

import rule_ref as rr
from test_gpu_chunk import check as check_chunk, chunk
from test_gpu_chunk_back import NAMES, backward, check as check_back

pytestmark = pytest.mark.gpu
LENS = [130, 0, 65, 1, 200, 63, 64, 128, 3]               # 9 x 16 heads, 36 units of a key head


@pytest.fixture(scope="module")
def g():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import gated_deltanet_decode_amd as g
    assert 2 * len(LENS) * 16 > torch.cuda.get_device_properties(0).multi_processor_count
    return g


def alone(x, b):
    """Sequence b of x as a call of its own (16 heads: two workgroups each)."""
    o = x["offsets"].tolist()
    one = {n: x[n][o[b]:o[b + 1]].contiguous() for n in NAMES + ("d_out",)}
    one.update(offsets=torch.tensor([0, o[b + 1] - o[b]], dtype=torch.int32, device="cuda"), slots=None)
    one.update({n: None if x[n] is None else x[n][b:b + 1].clone() for n in ("state", "d_state_out")})
    return one, slice(o[b], o[b + 1])


@pytest.mark.parametrize("dtype", rr.TYPES.values(), ids=rr.TYPES)
def test_chunk(g, dtype):
    x = rr.inputs(LENS, 16, 4, dtype, 41, tail=3)
    out, so = chunk(g, x)
    check_chunk(x, out, so, dtype)
    for b in (0, 3, 4, 7):
        one, at = alone(x, b)
        o, s = chunk(g, one)
        assert torch.equal(o, out[at]) and torch.equal(s[0], so[b]), b


@pytest.mark.parametrize("dtype", rr.TYPES.values(), ids=rr.TYPES)
def test_backward(g, dtype):
    x = rr.inputs(LENS, 16, 4, dtype, 42, tail=3)
    got = backward(g, x)
    check_back(x, got, dtype)
    for b in (0, 3, 4, 7):
        one, at = alone(x, b)
        for n, y in backward(g, one).items():
            assert torch.equal(y, got[n][b:b + 1] if n == "d_state" else got[n][at]), (b, n)
