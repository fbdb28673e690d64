"""GPU: the scale of gdn_add_rmsnorm_q8 is the formula's, rounded once to binary32:
half a step off.  The binary64 sums on both sides take at most 64 roundings on a
path (a lane's elements and the joins here, numpy's pairs there), the root halves
them, and a few follow: below 1e-14 of the scale, against the 6e-14 that 1e-6 of
half a step allows."""
import numpy as np
import pytest
import torch

import serve_ref as sr

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("xt,rt", [("f32", None), ("f32", "f32"), ("bf16", "bf16"), ("f16", "f16"), ("bf16", "f32"),
                                   ("f16", None)])
@pytest.mark.parametrize("rows,n", [(2000, 8), (2000, 100), (1000, 256), (1000, 513), (500, 1024), (500, 2048),
                                    (300, 4096), (200, 8192), (100, 9001), (100, 16384), (50, 20001)])
def test_scale_rounds_once(xt, rt, rows, n):
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import gated_deltanet_decode_amd as g
    print(f"\n  scale x={xt} residual={rt} rows={rows} n={n}", flush=True)
    gen = torch.Generator().manual_seed(n)
    x = torch.randn(rows, n, generator=gen).to(sr.TYPES[xt])
    res = None if rt is None else (3 * torch.randn(rows, n, generator=gen)).to(sr.TYPES[rt])
    w = 1.0 + 0.02 * torch.randn(n, generator=gen)
    q = torch.empty(rows, n, dtype=torch.int8, device="cuda")
    scale = torch.empty(rows, device="cuda")
    rd = None if res is None else res.cuda()
    g.add_rmsnorm_q8(x.cuda(), rd, rd, w.cuda(), q, scale)
    torch.cuda.synchronize()
    _, want = sr.rmsnorm_q8(sr.stored_sum(x, res), w, 1e-6)
    half = np.spacing(want.astype(np.float32)).astype(np.float64) / 2
    off = np.abs(scale.cpu().double().numpy() - want) / half
    assert off.max() <= 1 + 1e-6, off.max()
