"""CPU: the 64-bit reference's gradient of the delta rule against differences of
its forward pass."""
import pytest
import torch

import rule_ref as rr


@pytest.mark.parametrize("name", ["q", "k", "v", "beta", "gate", "state"])
def test_adjoint_against_differences(name):
    x = rr.inputs([5, 0, 3], 2, 1, torch.float32, 1, device="cpu")
    x = {n: t.double() if t is not None and t.is_floating_point() else t for n, t in x.items()}
    want = rr.backward(x)["d_state" if name == "state" else "d" + name]
    d = torch.randn(x[name].shape, generator=torch.Generator().manual_seed(2)).double()

    def loss(y):
        out, so, _, _ = rr.forward(y)
        return float((out * x["d_out"]).sum() + (so * x["d_state_out"]).sum())

    h = 1e-4
    diff = (loss(dict(x, **{name: x[name] + h * d})) - loss(dict(x, **{name: x[name] - h * d}))) / (2 * h)
    got = float((want * d).sum())
    assert abs(diff - got) <= 1e-6 * (1 + abs(got))       # h^2 of the third derivative's scale
