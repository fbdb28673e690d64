"""GPU: sequences of many chunks, whose operands' buffers in LDS change hands as often:
one buffer for float32 and fp16, two for bf16."""
import pytest
import torch

import rule_ref as rr
from test_gpu_chunk import check as check_chunk, chunk
from test_gpu_chunk_back import backward
from test_gpu_chunk_wide import alone

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def g():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import gated_deltanet_decode_amd as g
    return g


@pytest.mark.parametrize("dtype", rr.TYPES.values(), ids=rr.TYPES)
def test_many_chunks(g, dtype):
    """Twenty chunks and a piece, eight waves a workgroup: again, the same bits, and those of
    a sequence alone (four waves), which is checked against the recurrence."""
    x = rr.inputs([1290] * 3 + [700] * 6, 16, 4, dtype, 43)
    out, so = chunk(g, x)
    again, so2 = chunk(g, x)
    assert torch.equal(out, again) and torch.equal(so, so2)
    got, more = backward(g, x), backward(g, x)
    assert all(torch.equal(got[n], more[n]) for n in got)
    one, at = alone(x, 1)
    o, s = chunk(g, one)
    check_chunk(one, o, s, dtype)
    assert torch.equal(o, out[at]) and torch.equal(s[0], so[1])
    for n, y in backward(g, one).items():
        assert torch.equal(y, got[n][1:2] if n == "d_state" else got[n][at]), n
