"""GPU: gdn_pair_commit where one sequence's state passes 2^31 float4s (a masked
copy, bitwise)."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def test_one_state_past_2_31_float4s():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import gated_deltanet_decode_amd as g
    print("\n  pair_commit: 524289 heads", flush=True)
    heads = 524289
    m = torch.zeros(1, heads, 128, 128, device="cuda")
    n = torch.rand(1, heads, 128, 128, device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    ring = torch.zeros(1, 3, 100, device="cuda")
    ring_next = torch.ones_like(ring)
    acc = torch.zeros(1, dtype=torch.int32, device="cuda")
    g.pair_commit(acc, m, n, ring, ring_next)
    torch.cuda.synchronize()
    assert not bool(m[:, ::4097].any()) and not bool(m[:, -2:].any()) and not bool(ring.any())
    g.pair_commit(acc + 1, m, n, ring, ring_next)
    torch.cuda.synchronize()
    for i in range(0, heads, 65536):
        assert torch.equal(m[:, i:i + 65536], n[:, i:i + 65536]), f"heads from {i}"
    assert torch.equal(ring, ring_next)
    del m, n
    torch.cuda.empty_cache()
