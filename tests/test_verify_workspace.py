"""CPU: verify_workspace_bytes is 0 for sizes past the C arguments' 32 bits, which
would otherwise wrap around to small ones."""
import pytest


@pytest.mark.parametrize("B,V", [(2 ** 32 + 1, 5), (2 ** 32 + 65535, 5), (1, 2 ** 32 + 5), (2 ** 31, 5), (1, 2 ** 31),
                                 (2 ** 64 + 1, 5), (1 - 2 ** 32, 5), (1, 5 - 2 ** 32), (0, 5), (1, 0)])
def test_sizes_past_32_bits(B, V):
    import gated_deltanet_decode_amd as g
    assert g.verify_workspace_bytes(B, V) == 0
    assert g.verify_workspace_bytes(65535, 2 ** 31 - 1) == 65535 * g.verify_workspace_bytes(1, 1)
